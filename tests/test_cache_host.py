"""qk_norm_rope, cache_keep and NVFP4 caches refuse bad arguments on the host,
before anything is enqueued (no GPU here: the pointers are never dereferenced),
and the tests' own references tell planted mistakes."""
import concurrent.futures as cf
import ctypes

import numpy as np
import pytest

import cache_reference as C
from test_step_host import attend, cache, reorder


@pytest.fixture(scope="module")
def L():
    from draft_vocab_lm_gb300 import build
    build.build()
    from draft_vocab_lm_gb300 import _native
    return _native.lib()


def nvfp4(**kw):
    a = dict(dtype=1, k_blocks=0x8000, v_blocks=0x9000)
    a.update(kw)
    return cache(**a)


@pytest.mark.parametrize("bad", [
    dict(k_blocks=None), dict(v_blocks=None), dict(k_blocks=0x8008), dict(v_blocks=0x9004), dict(D=32), dict(D=48),
    dict(D=80), dict(D=96), dict(k_head_stride=32), dict(v_token_stride=96), dict(k_page_stride=2080), dict(k=0x1008),
    dict(D=128), dict(k_scale=float("nan")), dict(pages=0), dict(reserved=1), dict(v_head_stride=-64),
])
def test_nvfp4_cache_checks(L, bad):
    c = nvfp4(**bad)
    if bad == dict(D=128):  # strides of 64 are no multiple of it
        assert c.k_head_stride % c.D
    assert attend(L, c) == 1
    assert L.dvl_attention_workspace_bytes(c, 1, 4) == 0
    assert reorder(L, cache=c) == 1
    assert keep(L, c) == 1
    assert L.dvl_qk_norm_rope(ctypes.byref(qk(cache=c)), None) == 1


def qk(cache=None, **kw):
    """Two heads of 64 of a key-value cache, four query heads, six rows."""
    from draft_vocab_lm_gb300._native import DvlQk
    a = dict(rows=6, Hq=4, H=2, D=64, rot=64, interleaved=0, eps=1e-6, q=0x100000, k=0x110000, q_stride=256,
             q_head_stride=64, k_stride=128, k_head_stride=64, v_stride=128, v_head_stride=64, freq=0x1000,
             q_out=0x130000, q_out_stride=256, q_out_head_stride=64, k_out_stride=128, k_out_head_stride=64)
    if cache is not None:
        a.update(v=0x120000, cache=ctypes.pointer(cache), table=0x2000, table_stride=4, table_width=4, B=3,
                 lengths=0x3000)
    else:
        a.update(k_out=0x140000, positions=0x4000)
    a.update(kw)
    return DvlQk(**a)


def rope(L, **kw):
    return L.dvl_qk_norm_rope(ctypes.byref(qk(**kw)), None)


@pytest.mark.parametrize("with_cache", [False, True])
@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=1 << 31), dict(Hq=0), dict(H=0), dict(Hq=65537), dict(D=8), dict(D=72), dict(D=272),
    dict(rot=-16), dict(rot=24), dict(rot=80), dict(interleaved=2), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(q=None), dict(k=None), dict(q=0x100008), dict(k=0x110002), dict(q_stride=252),
    dict(q_head_stride=68), dict(k_stride=-128), dict(q_out=None), dict(q_out=0x130004), dict(q_weight=0x5002),
    dict(k_weight=0x5008), dict(freq=None), dict(freq=0x1004), dict(positions=0x4001),
    # outputs whose values overlap each other's, an input's or the other output's
    dict(q_out_stride=248), dict(q_out_head_stride=56), dict(q_out=0x100010), dict(q_out=0x110000),
    dict(k_out=0x130000), dict(k_out=0x100000), dict(k_out=0x110080), dict(k_out=0x150008),
    dict(k_out=0x150000, k_out_stride=64),
])
def test_rope_checks(L, bad, with_cache):
    assert rope(L, cache=cache() if with_cache else None, **bad) == 1
    assert L.dvl_qk_norm_rope(None, None) == 1


@pytest.mark.parametrize("bad", [
    dict(v=None), dict(v=0x120008), dict(v_stride=4), dict(H=4), dict(D=128), dict(B=-1), dict(B=4), dict(B=0),
    dict(table=None), dict(table=0x2002), dict(table_stride=-1), dict(table_width=0), dict(table_width=1 << 27),
    dict(lengths=None), dict(lengths=0x3001), dict(starts=0x6002),
])
def test_rope_cache_checks(L, bad):
    assert rope(L, cache=cache(), **bad) == 1


def test_rope_needs_a_place_to_write_and_positions(L):
    assert rope(L, v=0x120000) == 1
    assert rope(L, k_out=None) == 1
    assert rope(L, positions=None) == 1
    for scale in (0.0, -1.0, 1e-38, 1e38, float("nan")):
        assert rope(L, cache=cache(dtype=2, k_scale=scale)) == 1
        assert rope(L, cache=nvfp4(v_scale=scale)) == 1


@pytest.mark.parametrize("kw", [dict(rows=0), dict(rows=0, B=0), dict(B=0, starts=0x6000, table=None, lengths=None),
                                dict(rows=0, q_out=0x100000)])
def test_rope_nothing_to_do(L, kw):
    assert rope(L, cache=cache(), **kw) == 0


# (with every argument in order a call reaches the device, which is not here)
NO_DEVICE = 5


@pytest.mark.parametrize("kw", [
    dict(), dict(q_out=0x100000), dict(k_out=0x110000), dict(k_out=0x110000, q_out=0x100000),
    # queries, keys and values of one projection, normed in place
    dict(q=0x100000, k=0x100200, v=0x100300, q_stride=512, k_stride=512, v_stride=512, q_out=0x100000, q_out_stride=512,
         k_out=0x100200, k_out_stride=512),
    # heads first
    dict(q_out_stride=64, q_out_head_stride=6 * 64), dict(rot=0, freq=None), dict(interleaved=1, rot=32),
])
def test_rope_allowed(L, kw):
    import torch
    if torch.cuda.is_available():
        pytest.skip("no pointers to give a device")
    # (on a thread of its own: the failure's description is the thread's)
    with cf.ThreadPoolExecutor(1) as one:
        assert one.submit(rope, L, cache=cache(), **kw).result() == NO_DEVICE
        assert one.submit(rope, L, cache=nvfp4(), **kw).result() == NO_DEVICE


def test_rope_in_place_of_a_neighbour_is_refused(L):
    fused = dict(q=0x100000, k=0x100200, v=0x100300, q_stride=512, k_stride=512, v_stride=512, q_out_stride=512,
                 k_out_stride=512)
    assert rope(L, cache=cache(), **fused, q_out=0x100080) == 1  # heads 1 .. 4 of q and a key
    assert rope(L, cache=cache(), **fused, q_out=0x100000, k_out=0x100300) == 1  # over the values
    assert rope(L, cache=cache(), **fused, q_out=0x100400 - 512) == 1


def keep(L, c, **kw):
    a = dict(table=0x2000, ts=4, width=4, lengths=0x3000, first=0x4000, keep=0x5000, ks=8, counts=0x6000, B=3, M=8,
             out=0x7000)
    a.update(kw)
    return L.dvl_cache_keep(c, *a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(table=None), dict(table=0x2002), dict(ts=-1), dict(width=0), dict(width=1 << 27), dict(lengths=None),
    dict(lengths=0x3001), dict(first=None), dict(first=0x4002), dict(keep=None), dict(keep=0x5001), dict(ks=-1),
    dict(counts=None), dict(counts=0x6003), dict(B=-1), dict(M=-1), dict(M=0x7fffffff), dict(out=0x7002),
    # the new lengths over an input
    dict(out=0x3000), dict(out=0x4008), dict(out=0x6000), dict(out=0x5040), dict(out=0x2010),
])
def test_keep_checks(L, bad):
    assert keep(L, cache(), **bad) == 1
    assert keep(L, nvfp4(), **bad) == 1
    assert keep(L, None) == 1


def test_keep_nothing_to_do(L):
    assert keep(L, cache(), B=0) == 0


def test_references_and_planted_mistakes():
    rng = np.random.default_rng(0)
    x, w = rng.normal(size=(3, 2, 64)), 1 + 0.1 * rng.normal(size=64)
    freqs = [10000.0 ** (-2 * i / 32) for i in range(16)]
    z, err = C.turned(x, w, 1e-6, [5, 70000, -3], freqs, False)
    # a rotation keeps lengths, and position 0 keeps the values
    normed, _ = C.turned(x, w, 1e-6, [0, 0, 0], freqs, False)
    assert np.allclose((z ** 2).sum(-1), (normed ** 2).sum(-1))
    assert np.array_equal(normed, C.turned(x, w, 1e-6, None, None, False)[0])
    tol = C.bf16_bound(z, err)
    for wrong in (C.turned(x, w, 1e-6, [5, 70001, -3], freqs, False)[0], C.turned(x, w, 1e-6, [5, 70000, 3], freqs, False)[0],
                  C.turned(x, w, 1e-6, [5, 70000, -3], freqs, True)[0], C.turned(x, None, 0, [5, 70000, -3], freqs, False)[0]):
        assert np.any(np.abs(wrong - z) > tol)
    # a block of known values
    codes = np.array([[0x10, 0x32, 0x54, 0x76, 0x98, 0xba, 0xdc, 0xfe]], dtype=np.uint8)
    one = np.array([[0x38]], dtype=np.uint8)
    got = C.decode(codes, one, 2.0)
    assert np.array_equal(got[0], 2 * C.E2M1)
    C.check_nvfp4(codes, one, got, np.zeros_like(got), 2.0)
    for wrong in (codes ^ 0x70, codes[:, ::-1]):
        with pytest.raises(AssertionError):
            C.check_nvfp4(wrong, one, got, np.zeros_like(got), 2.0)
    with pytest.raises(AssertionError):
        C.check_nvfp4(codes, one + 2, got, np.zeros_like(got), 2.0)
    e = np.array([0x38, 0x7e, 0x01], dtype=np.uint8)
    C.check_e4m3(e, np.array([1.03, 600.0, 0.002]), np.zeros(3), 1.0)
    with pytest.raises(AssertionError):
        C.check_e4m3(e, np.array([1.07, 600.0, 0.002]), np.zeros(3), 1.0)
    # kept tokens: tokens 2 and 5 of the nodes follow token 0
    pool = np.arange(32).reshape(8, 4, 1)
    table = np.array([[3, 1, 0]])
    out = C.kept(pool, table, [9], [2], np.array([[0, 2, 5, -1]]), [3])
    flat = out[table[0]].reshape(-1)
    was = pool[table[0]].reshape(-1)
    assert flat[:5].tolist() == [was[0], was[1], was[2], was[4], was[7]] and np.array_equal(flat[5:], was[5:])
