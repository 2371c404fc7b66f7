"""dvl_beam_reorder where rows of one tensor lie between another's, and its
refusals of calls in place."""
import ctypes

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


def test_interleaved_rows_are_no_overlap(dvl):
    # one buffer, 256 bytes per beam: state a, state b, then their copies
    from draft_vocab_lm_gb300._native import DvlState, lib
    buf = torch.randint(0, 255, (2, 3, 256), dtype=torch.uint8, device="cuda")
    want = buf.clone()
    parents = torch.tensor([[2, 0, 0], [1, -1, 2]], dtype=torch.int32, device="cuda")
    for r in range(2):
        for i, p in enumerate(parents[r].tolist()):
            want[r, i, 128:] = want[r, p, :128] if p >= 0 else 0
    at = buf.data_ptr()
    states = (DvlState * 2)(DvlState(at, at + 128, 48, 256, 256), DvlState(at + 48, at + 176, 80, 256, 256))
    st = torch.cuda.current_stream().cuda_stream
    assert lib().dvl_beam_reorder(states, 2, None, None, parents.data_ptr(), 2, 3, 3, ctypes.c_void_p(st)) == 0
    torch.cuda.synchronize()
    assert torch.equal(buf, want)


def test_reordering_in_place_is_refused(dvl):
    a, b = torch.randn(2, 3, 8, device="cuda"), torch.randn(2, 3, 8, device="cuda")
    p = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    table, lengths = torch.zeros(2, 3, 2, dtype=torch.int32, device="cuda"), torch.ones_like(p)
    cache = dvl.KVCache(*(torch.zeros(9, 4, 1, 16, dtype=torch.bfloat16, device="cuda") for _ in range(2)))
    ok = dict(cache=cache, table=table, lengths=lengths, spare=torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3))
    for bad in [dict(states=[a, b], states_out=[b, a]), dict(states=[a], states_out=[a]), dict(ok, table_out=table),
                dict(ok, lengths_out=lengths), dict(ok, lengths_out=ok["spare"]), dict(ok, lengths_out=p),
                dict(states=[a, b], states_out=[torch.empty_like(a)] * 2)]:
        with pytest.raises(dvl.DvlError) as e:
            dvl.beam_reorder(p, **bad)
        assert e.value.status == 1
    t, n = torch.empty_like(table), torch.empty_like(lengths)
    assert dvl.beam_reorder(p, [a, a], states_out=[b, torch.empty_like(a)], **ok, table_out=t, lengths_out=n)[1] is t
