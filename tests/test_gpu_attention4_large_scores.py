"""Scores far above what fp32 holds to a unit, over an NVFP4 cache: positions
with the same score share the weight, and a smaller one has none."""
import numpy as np
import pytest

import cache_reference as C
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


def check(dvl, seed, lengths, T, G, heads, D, exponents):
    """Every key is 1 everywhere but one token's of each sequence, which is 2: of
    heads with positive scores it takes all the weight, of the others none.  The
    scores' sizes lie around 2^exponents."""
    g = torch.Generator().manual_seed(seed)
    page = 16
    need = [-(-n // page) for n in lengths]
    pages, width, B = sum(need) + 2, max(need), len(lengths)
    ids, at = torch.randperm(pages, generator=g).int(), 0
    table = torch.zeros(B, width, dtype=torch.int32)
    shape = (pages, page, heads)
    k = torch.full((*shape, D // 2), 0x22, dtype=torch.uint8)
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
        if lengths[b] > T:  # (a position that every row sees)
            p = int(torch.randint(lengths[b] - T, (1,), generator=g))
            k[table[b, p // page].long(), p % page] = 0x44
    v = torch.randint(256, (*shape, D // 2), generator=g, dtype=torch.uint8)
    kb = torch.full((*shape, D // 16), 0x38, dtype=torch.uint8)  # 1
    vb = torch.randint(0x30, 0x40, (*shape, D // 16), generator=g, dtype=torch.uint8)
    # the sum of D numbers near 1.5, times 2^x: about 2^e / sqrt(D)
    Hq = G * heads
    e = torch.tensor([exponents[i % len(exponents)] for i in range(B * T * Hq)], dtype=torch.float64).view(B, T, Hq, 1)
    sign = torch.randint(2, (B, T, Hq, 1), generator=g) * 2 - 1
    q = (1 + torch.rand(B, T, Hq, D, generator=g, dtype=torch.float64)) * sign * 2.0 ** (e - np.log2(1.5 * D ** 0.5))
    q = q.bfloat16()
    scales = (1.0, 0.02)
    cache = dvl.KVCache(k.cuda(), v.cuda(), k_scale=scales[0], v_scale=scales[1], k_blocks=kb.cuda(), v_blocks=vb.cuda())
    out, lse = dvl.paged_attention(cache, q.cuda(), table.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    kk, vv = (C.decode(c.numpy(), b.numpy(), s) for c, b, s in ((k, kb, scales[0]), (v, vb, scales[1])))
    ref, ref_lse, A, S, V1 = R.attention(q.double().numpy(), kk, vv, table.numpy(), np.array(lengths), D ** -0.5)
    # Equal scores are equal in fp32, too, and the others' difference is above
    # 2^18: a score's error moves no weight, only lse.
    assert S.max() < 2.0 ** 17
    tol, _ = R.attention_bounds(ref, ref_lse, A, 0 * S, V1, max(lengths), fp8=True)
    _, tol_lse = R.attention_bounds(ref, ref_lse, A, S, V1, max(lengths), fp8=True)
    err = np.abs(out.float().cpu().numpy() - ref)
    assert np.all(err <= tol), (np.nanmax(err - tol), np.isnan(err).sum())
    seen = np.isfinite(ref_lse)
    got = lse.cpu().numpy()
    assert np.array_equal(got[~seen], ref_lse[~seen])
    assert np.all(np.abs(got[seen] - ref_lse[seen]) <= tol_lse[seen])


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("T,G", [(1, 5), (3, 4), (1, 32), (8, 8)])
def test_attention4_large_scores(dvl, D, T, G):
    check(dvl, D + T, [1, 40, 333, 2], T, G, 2, D, [19, 20, 21, 22, 23, 24, 25, 26, 27, 28, 29, 30])


def test_attention4_large_scores_split_and_joined(dvl):
    for D in (64, 128, 256):
        check(dvl, D, [20011, 64], 1, 8, 1, D, [19, 22, 24, 25, 26, 28, 30])


def test_attention4_scores_without_a_finite_maximum(dvl):
    # a score of +infinity makes its row NaN, as over the other caches
    D = 64
    k = torch.full((4, 16, 1, D // 2), 0x22, dtype=torch.uint8, device="cuda")
    b = torch.full((4, 16, 1, D // 16), 0x38, dtype=torch.uint8, device="cuda")
    cache = dvl.KVCache(k, k, k_blocks=b, v_blocks=b)
    q = torch.ones(1, 1, 3, D, dtype=torch.bfloat16, device="cuda")
    q[0, 0, 1] = 2.0 ** 126
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    lengths = torch.tensor([50], dtype=torch.int32, device="cuda")
    out, lse = dvl.paged_attention(cache, q, table, lengths, scale=1.0)
    assert torch.all(out[0, 0, ::2] == 1.0) and torch.isnan(out[0, 0, 1]).all() and torch.isnan(lse[0, 0, 1])
    # the other caches' answer
    ones = torch.ones(4, 16, 1, D, dtype=torch.bfloat16, device="cuda")
    out, _ = dvl.paged_attention(dvl.KVCache(ones, ones), q, table, lengths, scale=1.0)
    assert torch.all(out[0, 0, ::2] == 1.0) and torch.isnan(out[0, 0, 1]).all()
