"""Softmax weights of dvl_paged_attention far below the largest one: a position
that takes nearly all the weight (an attention sink) and a long tail that
shares the rest.

Bound: that of step_reference.attention_bounds, with less room for small
weights.  An f16 weight (FP8 cache) keeps 2^-11 relative down to 2^-29 of the
row's largest and lies on a grid of 2^-39 of it below, so each position adds at
most 2^-40 |v|, the sum of weights being at least the largest."""
import numpy as np
import pytest

import step_reference as R

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


def tight_bounds(out, lse, A, S, V1, n_max, fp8):
    w = 2.0 ** -11 if fp8 else R.BF16
    rel = w + 2 * (S + 2.0 ** -21)[..., None] + (n_max / 16 + 64) * R.U
    return R.BF16 * np.abs(out) + rel * A * (1 + R.BF16) + 2.0 ** -40 * V1 + 1e-30


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,G,D", [(1, 4, 128), (1, 1, 64), (3, 5, 128), (1, 16, 64), (8, 8, 128), (1, 2, 256)])
@pytest.mark.parametrize("nats", [12, 16, 18, 22, 26])
def test_attention_sink_and_a_flat_tail(dvl, nats, T, G, D, fp8):
    # scores: q = (1, 0, ..), keys (nats, 0, ..) for the sink, else 0; every
    # value of the sink is 0, so the output is the tail's share of the weight
    lengths, page = [40_000, 17, 3], 64
    need = [-(-n // page) for n in lengths]
    table = torch.zeros(len(lengths), max(need), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    k = torch.zeros(at, page, 1, D)
    v = torch.ones(at, page, 1, D)
    v[..., 1::2] = torch.tensor([0.5, 2.0, 1.0, 0.25]).repeat(D // 8)
    for b, sink in enumerate((777, 0, 1)):
        k[table[b, sink // page].long(), sink % page, 0, 0] = nats
        v[table[b, sink // page].long(), sink % page] = 0
    q = torch.zeros(len(lengths), T, G, D)
    q[..., 0] = 1
    kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
    kd, vd = k.to(kind), v.to(kind)
    assert torch.equal(kd.float(), k) and torch.equal(vd.float(), v)
    out, lse = dvl.paged_attention(dvl.KVCache(kd.cuda(), vd.cuda()), q.bfloat16().cuda(), table.cuda(),
                                   torch.tensor(lengths, dtype=torch.int32).cuda(), scale=1.0)
    # the heads are alike: one is enough for the 64-bit form
    ref = R.attention(q[:, :, :1].double().numpy(), k.double().numpy(), v.double().numpy(), table.numpy(), lengths, 1.0)
    tol = tight_bounds(*ref, n_max=max(lengths), fp8=fp8)
    _, tol_lse = R.attention_bounds(*ref, n_max=max(lengths), fp8=fp8)
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for h in range(G):
        err = np.abs(got[:, :, h:h + 1] - ref[0])
        assert np.all(err <= tol), (h, (err / np.maximum(np.abs(ref[0]), 1e-30)).max())
        seen = np.isfinite(ref[1])  # (rows past a short sequence's start see nothing)
        assert np.array_equal(got_lse[:, :, h:h + 1][~seen], ref[1][~seen])
        assert np.all(np.abs(got_lse[:, :, h:h + 1][seen] - ref[1][seen]) <= tol_lse[seen])


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_scores_past_any_common_offset(dvl, fp8):
    # scores so large that a constant in the exponent would round: equal ones share the weight all the same
    D, n = 64, 300
    for size in (2.0 ** 20, 2.0 ** 27, 2.0 ** 60):
        k = torch.zeros(5, 64, 1, D)
        k[..., 0] = 1.0
        v = torch.full((5, 64, 1, D), 2.0)
        v[:, ::2] = 1.0
        q = torch.zeros(1, 1, 2, D)
        q[..., 0] = size
        kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
        out, _ = dvl.paged_attention(dvl.KVCache(k.to(kind).cuda(), v.to(kind).cuda()), q.bfloat16().cuda(),
                                     torch.arange(5, dtype=torch.int32, device="cuda").view(1, 5),
                                     torch.tensor([n], dtype=torch.int32, device="cuda"), scale=1.0)
        assert torch.all((out.float() - 1.5).abs() <= 1.5 * (R.BF16 + 2.0 ** -11))
