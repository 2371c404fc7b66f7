"""The cache's operators on a stream that has yet to make their inputs: a call that
ran anywhere else would read what lay there before, and what a call allocates
belongs to that stream until its work has ended."""
import pytest

from test_gpu_cache_step import Loop, snapshot

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


def late(dvl, kind, on, calls):
    """calls(loop, lengths, stream) while the stream still sleeps in front of the
    copies that make the inputs; returns its results, the caches and lengths of a
    twin's step in time, and the blocks the current stream filled meanwhile."""
    here, there = Loop(dvl, kind, seed=4), Loop(dvl, kind, seed=4)
    want = [x.clone() for x in here.step()]
    real = [x.clone() for x in (there.qkv, there.before, there.keep, there.counts)]
    lengths = there.before + there.T
    real.append(lengths.clone())
    inputs = (there.qkv, there.before, there.keep, there.counts, lengths)
    # in order, but another step's: other values, shorter sequences, nothing kept
    there.qkv.copy_(there.qkv.flip(0) * 0.5)
    there.before.copy_(there.before // 2)
    lengths.copy_(there.before + there.T)
    there.counts.zero_()
    sizes = [x.numel() * x.element_size() for x in want for _ in range(4)]
    # loading a kernel or asking the driver for memory may wait for the device:
    # everything runs once before
    st = torch.cuda.Stream()
    first = Loop(dvl, kind, seed=4)
    calls(first, first.before + first.T, on(st))
    warm = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes]
    del warm, first
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(400_000_000)
        for x, y in zip(inputs, real):
            x.copy_(y)
    got = calls(there, lengths, on(st))
    held = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes]
    torch.cuda.current_stream().synchronize()
    assert not st.query()  # all of it came while the stream slept
    st.synchronize()
    return got, want, here, there, held


def same(got, want, here, there, held):
    ok = all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want[1:]))
    ok &= all(torch.equal(a, b) for a, b in zip(snapshot(here), snapshot(there)))
    return ok, all(bool(torch.all(x == 0x55)) for x in held)


def step(loop, lengths, stream):
    """A step whose rotated queries live only as long as the host needs them."""
    dvl = loop.dvl
    q, k, v = loop.qkv.split([loop.Hq, loop.H, loop.H], dim=2)
    qo, _ = dvl.qk_norm_rope(q, k, v, rope=loop.rope, q_weight=loop.wq, k_weight=loop.wk, cache=loop.cache,
                             table=loop.table, lengths=lengths, stream=stream)
    out, lse = dvl.paged_attention(loop.cache, qo, loop.table, lengths, ws=loop.ws, stream=stream)
    after = dvl.cache_keep(loop.cache, loop.table, lengths, loop.before, loop.keep, loop.counts, stream=stream)
    return out, lse, after


@pytest.mark.parametrize("kind", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("handle", [False, True])
def test_a_step_behind_its_inputs(dvl, kind, handle):
    results, blocks = same(*late(dvl, kind, lambda st: st.cuda_stream if handle else st, step))
    assert results and blocks
