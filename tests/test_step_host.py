"""The drafting step's entry points refuse bad arguments on the host, before
anything is enqueued (no GPU here: the pointers are never dereferenced)."""
import ctypes

import numpy as np
import pytest

import step_reference as R


@pytest.fixture(scope="module")
def L():
    from draft_vocab_lm_gb300 import build
    build.build()
    from draft_vocab_lm_gb300 import _native
    return _native.lib()


def norm(**kw):
    from draft_vocab_lm_gb300._native import DvlNorm
    a = dict(rows=4, K=64, residual_dtype=0, group=0, eps=1e-6, x=0x1000, x_stride=64, weight=0x2000,
             out=0x3000, out_stride=64)
    a.update(kw)
    return DvlNorm(**a)


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=1 << 31), dict(K=0), dict(K=24577), dict(residual_dtype=1), dict(group=8),
    dict(group=48), dict(group=512), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None),
    dict(weight=None), dict(out=None), dict(x=0x1001), dict(weight=0x2001), dict(out=0x3001), dict(x_stride=-1),
    dict(out_stride=63), dict(codes=0x4000, codes_stride=64), dict(scales=0x5000),
    dict(codes=0x4000, codes_stride=63, scales=0x5000), dict(codes=0x4000, codes_stride=64, scales=0x5002),
    dict(residual=0x6000, residual_stride=64), dict(residual_out=0x6000, residual_out_stride=64),
    dict(residual=0x6002, residual_stride=64, residual_out=0x7000, residual_out_stride=64, residual_dtype=3),
    dict(residual=0x6000, residual_stride=64, residual_out=0x7000, residual_out_stride=32),
])
def test_norm_checks(L, bad):
    assert L.dvl_add_rmsnorm(ctypes.byref(norm(**bad)), None) == 1
    assert L.dvl_add_rmsnorm(None, None) == 1


def test_norm_no_rows_enqueues_nothing(L):
    assert L.dvl_add_rmsnorm(ctypes.byref(norm(rows=0)), None) == 0


def cache(**kw):
    from draft_vocab_lm_gb300._native import DvlKVCache
    a = dict(dtype=0, pages=8, page_size=16, heads=2, D=64, reserved=0, k=0x1000, v=0x2000,
             k_page_stride=2048, k_token_stride=128, k_head_stride=64, v_page_stride=2048, v_token_stride=128,
             v_head_stride=64, k_scale=1.0, v_scale=1.0)
    a.update(kw)
    return DvlKVCache(**a)


BAD_CACHES = [
    dict(dtype=1), dict(dtype=3), dict(pages=0), dict(page_size=0), dict(heads=0), dict(D=0), dict(D=24), dict(D=272),
    dict(reserved=1), dict(k=None), dict(v=None), dict(k=0x1008), dict(v=0x2008), dict(k_page_stride=2052),
    dict(k_token_stride=-128), dict(v_head_stride=4), dict(dtype=2, k_head_stride=72), dict(k_scale=float("nan")),
    dict(v_scale=float("inf")),
]


def attend(L, c, **kw):
    a = dict(q=0x3000, qb=256, qt=256, qh=64, B=1, T=1, Hq=4, table=0x4000, ts=4, width=4, lengths=0x5000, scale=0.125,
             out=0x6000, lse=None, ws=0x7000, bytes=1 << 40)
    a.update(kw)
    return L.dvl_paged_attention(c, *a.values(), None)


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_cache_checks(L, bad):
    c = cache(**bad)
    assert attend(L, c) == 1
    assert L.dvl_attention_workspace_bytes(c, 1, 4) == 0
    assert reorder(L, cache=c) == 1


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(q=0x3008), dict(qb=252), dict(qt=4), dict(qh=65), dict(B=-1), dict(T=0), dict(T=9), dict(Hq=0),
    dict(Hq=3), dict(Hq=130), dict(T=8, Hq=18), dict(table=None), dict(table=0x4002), dict(ts=-1), dict(width=0),
    dict(width=1 << 27), dict(width=(1 << 27) - 7), dict(lengths=None), dict(lengths=0x5001), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(out=None), dict(out=0x6004), dict(lse=0x6002),
])
def test_attention_checks(L, bad):
    assert attend(L, cache(), **bad) == 1


@pytest.mark.parametrize("T,Hq", [(0, 4), (9, 4), (1, 0), (1, 3), (1, 130), (8, 18)])
def test_attention_workspace_limits(L, T, Hq):
    assert L.dvl_attention_workspace_bytes(cache(), T, Hq) == 0
    assert L.dvl_attention_workspace_bytes(None, 1, 4) == 0


def select(L, **kw):
    a = dict(logits=0x1000, dtype=3, bs=300, js=100, scores=0x2000, batch=2, beams=3, N=100, k=4, d2t=None,
             out=0x3000, parents=0x4000, tokens=0x5000, ws=0x6000, bytes=1 << 40)
    a.update(kw)
    return L.dvl_beam_select(*a.values(), None)


@pytest.mark.parametrize("bad", [
    dict(dtype=1), dict(dtype=2), dict(logits=None), dict(logits=0x1002), dict(dtype=0, logits=0x1001), dict(bs=-1),
    dict(js=-1), dict(scores=None), dict(scores=0x2002), dict(batch=-1), dict(beams=0), dict(beams=33), dict(N=0),
    dict(N=0x7fffffff), dict(k=0), dict(k=33), dict(d2t=0x2), dict(out=None), dict(parents=None), dict(tokens=0x5001),
    dict(batch=1 << 27, beams=32),
])
def test_beam_checks(L, bad):
    assert select(L, **bad) == 1


def test_beam_workspace(L):
    assert select(L, ws=None) == 4 and select(L, ws=0x6008) == 4 and select(L, bytes=100) == 4
    assert select(L, batch=0) == 0
    assert L.dvl_beam_workspace_bytes(1, 33, 10) == 0 and L.dvl_beam_workspace_bytes(1, 1, 0) == 0
    # header, tickets, and one list of 32 keys and one sum per segment: at least 608
    need = [L.dvl_beam_workspace_bytes(b, 4, 16000) for b in (1, 100, 200, 5000)]
    assert need[0] == need[1] == 512 + 16384 + 608 * (32 * 8 + 8)
    assert need[2] == 512 + 16384 + 800 * (32 * 8 + 8) and need[3] == 512 + 16384 + 16384 * (32 * 8 + 8)


def reorder(L, cache=None, n=1, parents=0x9000, batch=2, beams=3, k=3, state=None, pages=None):
    from draft_vocab_lm_gb300._native import DvlBeamPages, DvlState
    s = dict(src=0x10000, dst=0x20000, row_bytes=64, src_stride=64, dst_stride=64)
    s.update(state or {})
    states = (DvlState * max(n, 1))(*[DvlState(**s) for _ in range(max(n, 1))])
    p = None
    if cache is not None or pages is not None:
        a = dict(table=0x1000, table_out=0x2000, lengths=0x3000, lengths_out=0x4000, spare=0x5000, width=4, reserved=0)
        a.update(pages or {})
        p = DvlBeamPages(**a)
    return L.dvl_beam_reorder(states, n, p, cache, parents, batch, beams, k, None)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(n=9), dict(parents=None), dict(parents=0x9002), dict(batch=-1), dict(beams=0), dict(beams=33),
    dict(k=0), dict(k=33), dict(state=dict(src=None)), dict(state=dict(dst=None)), dict(state=dict(row_bytes=0)),
    dict(state=dict(src_stride=32)), dict(state=dict(dst_stride=32)), dict(state=dict(dst=0x10100)), dict(pages={}),
])
def test_reorder_checks(L, bad):
    assert reorder(L, **bad) == 1


@pytest.mark.parametrize("bad", [
    dict(table=None), dict(table_out=None), dict(lengths=None), dict(lengths_out=None), dict(spare=None),
    dict(table=0x1002), dict(spare=0x5001), dict(width=0), dict(reserved=1),
])
def test_reorder_page_checks(L, bad):
    assert reorder(L, cache=cache(), pages=bad) == 1


def test_reorder_nothing_to_do(L):
    assert reorder(L, batch=0) == 0
    assert reorder(L, n=0) == 0


def test_e4m3_table_and_planted_mistakes():
    # the tests' own tables and bounds: known values, and an oracle with a
    # mistake planted is told apart
    v = R.e4m3_values()
    assert v[0x38] == 1.0 and v[0x7e] == 448.0 and v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6
    assert v[0xb8] == -1.0 and np.isnan(v[0x7f]) and np.isnan(v[0xff])
    rng = np.random.default_rng(0)
    q, k, vv = rng.normal(size=(1, 2, 2, 16)), rng.normal(size=(3, 4, 1, 16)), rng.normal(size=(3, 4, 1, 16))
    table, n = np.array([[2, 0, 1]]), np.array([9])
    good = R.attention(q, k, vv, table, n, 0.25)
    tol, tol_lse = R.attention_bounds(*good, n_max=9, fp8=False)
    for wrong in (R.attention(q, k, vv, table, n - 1, 0.25), R.attention(q, k, vv, table[:, ::-1], n, 0.25),
                  R.attention(q, k, vv, table, n, 0.26)):
        assert np.any(np.abs(wrong[0] - good[0]) > tol) and np.any(np.abs(wrong[1] - good[1]) > tol_lse)
    x, s = rng.normal(size=(1, 2, 50)), np.zeros((1, 2))
    a = R.beam_scores(x, s)
    assert np.allclose(np.exp(a).sum(axis=2), 1)
    b = R.beam_scores(x + np.array([0.0, 1.0])[None, :, None], s)  # lse takes a shift out
    assert np.abs(a - b).max() < 1e-12
