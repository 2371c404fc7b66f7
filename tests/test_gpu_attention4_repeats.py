"""Attention over an NVFP4 cache gives the same bits every time: alone, next to
other work that shifts its blocks, with another workspace, and replayed."""
import pytest

from test_gpu_attention4 import Case

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


@pytest.mark.parametrize("lengths,T,Hq,heads,D", [
    ([731], 1, 20, 4, 128), ([4101, 0, 1553, 3898], 3, 40, 8, 128), ([60001], 1, 16, 2, 256), ([9000, 3, 30000], 5, 8, 1, 64),
    ([200] * 70, 1, 4, 2, 192), ([2000, 1], 8, 16, 2, 128),
])
def test_attention4_repeats_itself(dvl, lengths, T, Hq, heads, D):
    c = Case(len(lengths) + D, lengths, T, Hq, heads, D, 32)
    want = [x.clone() for x in c.call(dvl)]
    q, side = c.q.cuda(), torch.cuda.Stream()
    a = torch.randn(2048, 2048, device="cuda")
    ws = dvl.attention_workspace(c.cache, len(lengths), T, Hq)
    for i in range(24):
        if i % 3 == 1:
            with torch.cuda.stream(side):
                torch.mm(a, a)
        got = c.call(dvl, q=q, ws=ws if i % 2 else None)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), i
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        dvl.paged_attention(c.cache, q, c.table, c.lengths, out=out, lse=lse, ws=ws)
    for _ in range(5):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
