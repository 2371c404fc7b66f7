"""An empty batch through paged_attention: nothing to do, and no refusal."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dvl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from draft_vocab_lm_gb300 import build
    build.build()
    import draft_vocab_lm_gb300 as d
    return d


@pytest.mark.parametrize("dim", [3, 4])
def test_attention_without_sequences(dvl, dim):
    cache = dvl.KVCache(*(torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    q = torch.empty((0, 1, 4, 64) if dim == 4 else (0, 4, 64), dtype=torch.bfloat16, device="cuda")
    table = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    lengths = torch.empty(0, dtype=torch.int32, device="cuda")
    for kw in (dict(), dict(want_lse=False), dict(ws=dvl.attention_workspace(cache, 1, 1, 4))):
        out, lse = dvl.paged_attention(cache, q, table, lengths, **kw)
        assert out.shape == q.shape and (lse is None if "want_lse" in kw else lse.shape == q.shape[:-1])
