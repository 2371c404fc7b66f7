"""dvl_add_rmsnorm against the 64-bit form.

Bounds: a thread adds at most 24 squares, two five-step butterflies follow, so
the mean square is off by at most 36 u and its root by half that; the
reciprocal root is within 4 u, 1 / K, its product, two products and the
addition of the residual round once each: y is within 28 u.  bf16 then adds 2^-8.  A code is the nearest
E4M3 value of y / scale: half a step is at most 2^-4 of the quotient or, below
the normal range, 2^-10."""
import numpy as np
import pytest

import step_reference as R
import synthetic as S

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

Y = 28 * R.U
E4M3 = R.e4m3_values()


@pytest.fixture(scope="module")
def dvl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from draft_vocab_lm_gb300 import build
    build.build()
    import draft_vocab_lm_gb300 as d
    return d


def inputs(seed, rows, K, kind, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, K, generator=g) * std).bfloat16()
    w = (1 + 0.1 * torch.randn(K, generator=g)).bfloat16()
    r = None
    if kind:
        r = (torch.randn(rows, K, generator=g) * 3 * std).to(torch.float32 if kind == "fp32" else torch.bfloat16)
    return x, w, r


def f64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def verify(x, w, r, eps, group, got):
    out, res, codes, scales = got
    u, y = R.norm(f64(x), f64(w), f64(r), eps)
    if r is not None:
        want = (x.float() + r.float()).to(r.dtype)  # one fp32 addition, one rounding
        assert torch.equal(res.cpu(), want)
    if out is not None:
        err = np.abs(f64(out) - y)
        assert np.all(err <= (R.BF16 + 2 * Y) * np.abs(y) + 1e-38), err.max()
    if codes is not None:
        amax = R.group_amax(y, group)
        s = scales.cpu().numpy().astype(np.float64)
        assert s.shape == amax.shape
        assert np.all(np.abs(s - amax / 448) <= (Y + 2 * R.U) * amax / 448 + 1e-45)
        size = group or y.shape[1]
        per = np.repeat(s, size, axis=1)[:, :y.shape[1]]
        c = E4M3[codes.view(torch.uint8).cpu().numpy()]
        quo = np.divide(y, per, out=np.zeros_like(y), where=per > 0)
        step = np.maximum(2.0 ** -4 * np.abs(quo), 2.0 ** -10)
        assert np.all(np.abs(c - quo) <= step * (1 + 1e-4) + 448 * 4 * Y)


@pytest.mark.parametrize("kind", [None, "bf16", "fp32"])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 64), (3, 65), (2, 2560), (33, 5120), (5, 1001), (1, 8191),
                                    (2, 8192), (3, 8200), (2, 16392), (1, 24576), (300, 80), (257, 328)])
def test_norm_shapes(dvl, rows, K, kind):
    x, w, r = inputs(rows + K, rows, K, kind)
    for group, bf16 in [(None, True), (0, False), (128, True)]:
        got = dvl.add_rmsnorm(x.cuda(), w.cuda(), None if r is None else r.cuda(), bf16=bf16, fp8_group=group)
        assert (got[0] is not None) == bf16 and (got[2] is not None) == (group is not None)
        verify(x, w, r, 1e-6, group, got)


@pytest.mark.parametrize("group", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("K", [16, 72, 200, 640, 2567, 5120])
def test_norm_groups(dvl, K, group):
    x, w, r = inputs(K + group, 7, K, "bf16")
    # groups of very different size, one all zero
    x[:, :min(K, 40)] *= 1e-3
    x[2] = 0
    r[2] = 0
    verify(x, w, r, 1e-5, group, dvl.add_rmsnorm(x.cuda(), w.cuda(), r.cuda(), eps=1e-5, fp8_group=group))


@pytest.mark.parametrize("K,offset,extra", [(2560, 0, 8), (2560, 1, 3), (64, 0, 1), (1000, 4, 24)])
def test_norm_strides_and_in_place(dvl, K, offset, extra):
    rows = 9
    x, w, r = inputs(K, rows, K, "bf16")
    wide = torch.zeros(rows, K + offset + extra, dtype=torch.bfloat16, device="cuda")
    xs = wide[:, offset:offset + K]
    xs.copy_(x)
    buf = torch.full((rows, K + offset + extra), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:, offset:offset + K]
    res = r.cuda()
    got = dvl.add_rmsnorm(xs, w.cuda(), res, out=out, residual_out=res)  # the residual stream in place
    assert got[0] is out and got[1] is res
    verify(x, w, r, 1e-6, None, got)
    assert torch.all(buf[:, :offset] == 7) and torch.all(buf[:, offset + K:] == 7)
    # u over x itself
    x2, r2 = x.cuda(), r.cuda()
    verify(x, w, r, 1e-6, None, dvl.add_rmsnorm(x2, w.cuda(), r2, residual_out=x2))
    # one row for all (stride 0)
    one = x[:1].cuda().expand(rows, K)
    verify(x[:1].expand(rows, K), w, r, 1e-6, 64, dvl.add_rmsnorm(one, w.cuda(), r.cuda(), fp8_group=64))


def test_norm_scale_extremes_and_non_finite(dvl):
    K = 256
    x, w, _ = inputs(5, 6, K, None)
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 9] = float("inf")
    x[3] *= 1e30   # squares past fp32: y is 0
    x[4] = 2.0 ** -80  # squares below fp32: the mean square is eps
    out, _, codes, scales = dvl.add_rmsnorm(x.cuda(), w.cuda(), eps=1e-6, fp8_group=128)
    out, c, s = f64(out), E4M3[codes.view(torch.uint8).cpu().numpy()], scales.cpu().numpy()
    assert np.all(out[0] == 0) and np.all(c[0] == 0) and np.all(s[0] == 0)
    assert np.isnan(out[1]).all() and np.isnan(s[1]).all() and np.isnan(c[1]).all()
    assert np.isnan(out[2, 9]) and np.all(out[2, :9] == 0) and np.isnan(s[2, 0]) and s[2, 1] == 0
    assert np.all(out[3] == 0) and np.all(s[3] == 0)
    want = f64(x)[4] * f64(w) / np.sqrt(1e-6)
    assert np.all(np.abs(out[4] - want) <= (R.BF16 + 2 * Y) * np.abs(want))
    verify(x[5:], w, None, 1e-6, 128, [t[5:] if t is not None else None
                                       for t in dvl.add_rmsnorm(x.cuda(), w.cuda(), fp8_group=128)])


def test_norm_tiny_groups_have_codes_zero(dvl):
    # |y| below 2^-119: the multiplier 448 / a is no fp32 number
    x = torch.ones(1, 64, dtype=torch.bfloat16)
    w = torch.full((64,), 2.0 ** -121, dtype=torch.bfloat16)
    w[32:] = 2.0 ** -117
    _, _, codes, scales = dvl.add_rmsnorm(x.cuda(), w.cuda(), bf16=False, fp8_group=32)
    c = E4M3[codes.view(torch.uint8).cpu().numpy()]
    assert np.all(c[0, :32] == 0) and np.all(c[0, 32:] == 448)
    assert np.allclose(scales.cpu().numpy().astype(np.float64)[0, 1] * 448, 2.0 ** -117, rtol=1e-5)


def test_norm_on_another_stream_and_repeatable(dvl):
    x, w, r = inputs(11, 4000, 2560, "bf16")
    a, b, c = x.cuda(), w.cuda(), r.cuda()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    one = dvl.add_rmsnorm(a, b, c, fp8_group=0, stream=st)
    st.synchronize()
    two = dvl.add_rmsnorm(a, b, c, fp8_group=0)
    torch.cuda.synchronize()
    for p, q in zip(one, two):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))
    verify(x[:50], w, r[:50], 1e-6, 0, [t[:50] for t in one])


def test_norm_no_rows(dvl):
    e = torch.empty(0, 2560, dtype=torch.bfloat16, device="cuda")
    out, res, codes, scales = dvl.add_rmsnorm(e, torch.ones(2560, dtype=torch.bfloat16, device="cuda"), e.clone(),
                                              fp8_group=0)
    assert out.shape == (0, 2560) and res.shape == (0, 2560) and codes.shape == (0, 2560) and scales.shape == (0, 1)


def test_norm_refusals(dvl):
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for bad in [dict(x=x.cpu()), dict(x=x.float()), dict(x=x[0]), dict(weight=w[:32]), dict(weight=w.float()),
                dict(residual=x[:1]), dict(residual=x.double()), dict(fp8_group=100), dict(fp8_group=8),
                dict(bf16=False), dict(out=x[:, :32]), dict(codes=x), dict(residual_out=x),
                dict(residual=x, residual_out=x.float()), dict(x=x.t()), dict(residual=x.cpu())]:
        with pytest.raises(ValueError):
            args = dict(x=x, weight=w)
            args.update(bad)
            dvl.add_rmsnorm(**args)
    for bad in [dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))]:
        with pytest.raises(dvl.DvlError):
            dvl.add_rmsnorm(x, w, **bad)
    big = torch.zeros(1, 24577, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(dvl.DvlError):
        dvl.add_rmsnorm(big, big[0])
