"""The drafting step's operators on another stream than the current one, with
nothing of their own passed in: what the current stream allocates and writes
right after the call does not reach it."""
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


def calls(dvl):
    """name -> a call that takes the stream and returns its results."""
    g = torch.Generator(device="cuda").manual_seed(2)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    kv = [rand(200, 16, 2, 128).bfloat16() for _ in range(2)]
    cache = dvl.KVCache(*kv)
    q, table = rand(4, 1, 8, 128).bfloat16(), torch.arange(200, dtype=torch.int32, device="cuda").view(4, 50)
    lengths = torch.tensor([800, 3, 0, 555], dtype=torch.int32, device="cuda")
    x, w, r = rand(64, 2560).bfloat16(), rand(2560).bfloat16(), rand(64, 2560)
    logits, scores = rand(2, 4, 30000), rand(2, 4)
    parents, state = torch.tensor([[3, 0, 0, 2]], dtype=torch.int32, device="cuda"), rand(1, 4, 5000)
    return {
        "norm": lambda s: dvl.add_rmsnorm(x, w, r, fp8_group=128, stream=s),
        "attention": lambda s: dvl.paged_attention(cache, q, table, lengths, stream=s),
        "select": lambda s: dvl.beam_select(logits, scores, 6, stream=s),
        "reorder": lambda s: dvl.beam_reorder(parents, [state], stream=s)[0],
    }


def overwrite(sizes):
    """New blocks of these sizes on the current stream, filled at once."""
    held = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    return held


@pytest.mark.parametrize("name", ["norm", "attention", "select", "reorder"])
@pytest.mark.parametrize("handle", [False, True])
def test_other_streams_memory_is_left_alone(dvl, name, handle):
    call = calls(dvl)[name]
    want = [t.clone() for t in call(None)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    sizes = [512 + 16384 + n for n in (0, 160_512)] + [t.numel() * t.element_size() for t in want]
    cache = dvl.KVCache(*(torch.zeros(1, 16, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    sizes += [dvl.attention_workspace(cache, 4, 1, 8).numel(), dvl.beam_workspace(2, 4, 30000).numel()]
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            torch.cuda._sleep(20_000_000)  # the call waits behind it
        got = call(st.cuda_stream if handle else st)
        held = overwrite(sizes)
        torch.cuda.current_stream().synchronize()
        st.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        del held


def owner(t):
    """The stream whose memory a tensor lies in."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the allocator's memory")


def test_results_and_workspaces_belong_to_the_stream_they_are_made_for(dvl):
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for name, call in calls(dvl).items():
        torch.cuda.synchronize()
        here = torch.cuda.current_stream().cuda_stream
        assert all(owner(t) == here for t in call(None)), name
        assert all(owner(t) == st.cuda_stream for t in call(st)), name
        torch.cuda.synchronize()
    cache = dvl.KVCache(*(torch.zeros(1, 16, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    for s in (st, st.cuda_stream):
        assert owner(dvl.attention_workspace(cache, 1, 1, 8, stream=s)) == st.cuda_stream
        assert owner(dvl.beam_workspace(1, 4, 1000, stream=s)) == st.cuda_stream
    torch.cuda.synchronize()
