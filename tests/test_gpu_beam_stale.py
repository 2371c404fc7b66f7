"""dvl_beam_select on a workspace that a call cut short could leave: its results
say nothing, but it stays inside its tensors, and initialising the workspace
mends it."""
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


def test_keys_of_a_longer_call_do_not_index_d2t(dvl):
    g = torch.Generator(device="cuda").manual_seed(1)
    long = torch.randn(1, 2, 248320, generator=g, device="cuda") + 50.0
    short = torch.randn(1, 2, 9000, generator=g, device="cuda")
    scores = torch.zeros(1, 2, device="cuda")
    d2t = (torch.arange(9000, dtype=torch.int32, device="cuda") * 3 + 7).contiguous()
    ws = dvl.beam_workspace(1, 2, 248320)
    want = dvl.beam_select(short, scores, 8, d2t=d2t)
    kept = [torch.full_like(t, -1) for t in want]
    for left in range(1, 6):
        dvl.beam_select(long, scores, 8, ws=ws)        # keys of rows far past 9,000
        ws[512:516] = torch.tensor([left, 0, 0, 0], dtype=torch.uint8)  # as many blocks as counted already
        dvl.beam_select(short, scores, 8, d2t=d2t, ws=ws, out_scores=kept[0], parents=kept[1], tokens=kept[2])
        known = torch.isin(kept[2], d2t) | (kept[2] == -1)
        assert known.all()
        dvl.workspace_init(ws)
        for a, b in zip(dvl.beam_select(short, scores, 8, d2t=d2t, ws=ws), want):
            assert torch.equal(a, b)
