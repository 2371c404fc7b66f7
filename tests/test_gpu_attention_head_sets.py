"""dvl_paged_attention with more cached heads than a grid has lanes (eight)."""
import pytest

from test_gpu_attention import Case

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


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads", [9, 11, 12, 16, 32])
@pytest.mark.parametrize("T", [1, 3])
def test_attention_more_heads_than_lanes(dvl, T, heads, fp8):
    # several sets of heads follow one another in a block's share
    for lengths in ([700, 1, 0, 64, 333, 5, 128], [9000, 40]):
        c = Case(heads + T, lengths, T, 2 * heads, heads, 64, 16, fp8)
        c.verify(c.call(dvl))
