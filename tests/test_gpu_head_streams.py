"""The head's entry points on another stream than the current one: what they
make for themselves is that stream's, and comes out the same."""
import pytest

from test_gpu_step_streams import dvl, overwrite, owner  # noqa: F401  (dvl is a fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def calls(dvl):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(3)
    w = (torch.randn(4096, 2560, generator=g, device="cuda") * 0.02).bfloat16()
    h = torch.randn(3, 2560, generator=g, device="cuda").bfloat16()
    cand = torch.randint(0, 4096, (3, 16), generator=g, device="cuda", dtype=torch.int32)
    ranks = list(range(5, 3000, 3))
    head = dvl.Head(w)

    def shortlist(s):
        sl = dvl.Shortlist(w, ranks, len(ranks) + 8, stream=s)
        return [sl.w[:len(ranks)], sl.d2t[:len(ranks)]]

    return {
        "argmax": lambda s: dvl.draft_argmax(head, h, stream=s),
        "topk": lambda s: dvl.draft_topk(head, h, 4, stream=s),
        "score": lambda s: [dvl.score_ids(head, h, cand, stream=s)],
        "trim": lambda s: [t for t in dvl.trim_head(w, ranks, stream=s) if torch.is_tensor(t)],
        "nvfp4": lambda s: list(dvl.quantize_head(w, "nvfp4", stream=s)[:2]),
        "fp8": lambda s: [dvl.quantize_head(w, "fp8", stream=s)[0]],
        "shortlist": shortlist,
    }


@pytest.mark.parametrize("name", ["argmax", "topk", "score", "trim", "nvfp4", "fp8", "shortlist"])
@pytest.mark.parametrize("handle", [False, True])
def test_results_on_another_stream(dvl, name, handle):  # noqa: F811
    call = calls(dvl)[name]
    here = torch.cuda.current_stream().cuda_stream
    want = [t.clone() for t in call(None)]
    assert all(owner(t) == here for t in call(None))
    st = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            torch.cuda._sleep(20_000_000)
        got = call(st.cuda_stream if handle else st)
        held = overwrite([t.numel() * t.element_size() for t in want] + [dvl.workspace_bytes(3, k) for k in (1, 4)])
        st.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert all(owner(t) == st.cuda_stream for t in got)
        del held, got
    torch.cuda.synchronize()
    assert owner(dvl.make_workspace(3, 4, stream=st)) == st.cuda_stream
    torch.cuda.synchronize()
