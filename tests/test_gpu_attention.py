"""dvl_paged_attention against the 64-bit form, within the bounds of
step_reference.attention_bounds."""
import numpy as np
import pytest

import step_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

E4M3 = R.e4m3_values()


@pytest.fixture(scope="module")
def dvl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from draft_vocab_lm_gb300 import build
    build.build()
    import draft_vocab_lm_gb300 as d
    return d


class Case:
    """A cache, its table and the queries of one call, on the GPU and as 64-bit values."""

    def __init__(self, seed, lengths, T, Hq, heads, D, page, fp8=False, layout="tokens", std=1.0):
        g = torch.Generator().manual_seed(seed)
        B = len(lengths)
        need = [-(-max(n, 0) // page) for n in lengths]
        self.width = max(max(need), 1) + 1
        pages = sum(need) + 2
        shape = (pages, page, heads, D) if layout == "tokens" else (pages, heads, page, D)
        self.k_scale, self.v_scale = (0.03, 0.05) if fp8 else (1.0, 1.0)
        pool = []
        for _ in range(2):
            x = torch.randn(shape, generator=g) * std
            pool.append((x * 30).clamp(-440, 440).to(torch.float8_e4m3fn) if fp8 else x.bfloat16())
        ids = torch.randperm(pages, generator=g).int()
        table = torch.full((B, self.width), -1, dtype=torch.int32)  # never read past the length
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        used = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(lengths):
            for p in range(need[b]):
                used[table[b, p].long(), :min(page, n - p * page)] = True
        self.dead = ~used  # slots no sequence reads
        self.q = (torch.randn(B, T, Hq, D, generator=g) * 2).bfloat16()
        self.k, self.v = (x.cuda() for x in pool)
        if layout == "heads":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.table, self.lengths, self.T, self.fp8 = table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(), T, fp8

    def poison(self):
        """NaN in every slot that no sequence's length reaches."""
        for x in (self.k, self.v):
            x.view(torch.uint8)[self.dead.cuda()] = 0x7f if self.fp8 else 0xff

    def values(self, x, scale):
        if self.fp8:
            return E4M3[x.contiguous().view(torch.uint8).cpu().numpy()] * scale
        return x.float().cpu().numpy().astype(np.float64)

    def call(self, dvl, **kw):
        self.cache = dvl.KVCache(self.k, self.v, k_scale=self.k_scale, v_scale=self.v_scale)
        return dvl.paged_attention(self.cache, kw.pop("q", self.q.cuda()), self.table, self.lengths, **kw)

    def verify(self, got, scale=None):
        D = self.q.shape[3]
        ref = R.attention(self.q.float().numpy().astype(np.float64), self.values(self.k, self.k_scale),
                          self.values(self.v, self.v_scale), self.table.cpu().numpy(),
                          self.lengths.cpu().numpy(), D ** -0.5 if scale is None else scale)
        tol, tol_lse = R.attention_bounds(*ref, n_max=int(self.lengths.max()), fp8=self.fp8)
        out = got[0].float().cpu().numpy().reshape(ref[0].shape)
        err = np.abs(out - ref[0])
        assert np.all(err <= tol), (err - tol).max()
        if got[1] is not None:
            lse = got[1].cpu().numpy().reshape(ref[1].shape)
            finite = np.isfinite(ref[1])
            assert np.array_equal(lse[~finite], ref[1][~finite])
            assert np.all(np.abs(lse[finite] - ref[1][finite]) <= tol_lse[finite])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,heads,D", [(20, 4, 128), (8, 8, 64), (16, 2, 256), (4, 1, 80), (5, 5, 16), (6, 2, 208),
                                        (12, 2, 48)])
@pytest.mark.parametrize("T", [1, 3])
def test_attention_heads_and_widths(dvl, Hq, heads, D, T, fp8):
    c = Case(D + Hq + T, [1, 63, 64, 65, 200, 0, 131], T, Hq, heads, D, 16, fp8)
    c.verify(c.call(dvl))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,G", [(1, 1), (2, 8), (3, 5), (8, 8), (8, 1), (1, 64), (5, 7), (4, 4), (1, 17)])
def test_attention_query_rows(dvl, T, G, fp8):
    # up to 64 query rows per cached head; lengths below T leave rows empty
    for D in (64, 128, 256):
        c = Case(T * 100 + G, [0, 1, T - 1, T, 67, 130], T, 2 * G, 2, D, 32, fp8)
        c.verify(c.call(dvl))


@pytest.mark.parametrize("page", [1, 7, 16, 48, 64, 100, 1000])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
def test_attention_pages(dvl, page, layout):
    for fp8 in (False, True):
        c = Case(page, [5, 64, 333, 128, 1], 2, 10, 2, 128, page, fp8, layout)
        c.verify(c.call(dvl))


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_long_sequences_are_split_and_joined(dvl, fp8):
    for lengths, heads, D in [([20011], 1, 128), ([9000, 3, 0, 30000], 2, 64), ([12345], 2, 256)]:
        c = Case(len(lengths), lengths, 1, 4 * heads, heads, D, 64, fp8)
        c.verify(c.call(dvl))
    c = Case(5, [7001, 64], 3, 8, 1, 128, 64, fp8)
    c.verify(c.call(dvl))


def test_attention_many_sequences(dvl):
    rng = np.random.default_rng(1)
    lengths = [int(n) if rng.random() > 0.1 else 0 for n in rng.integers(1, 150, size=700)]
    c = Case(2, lengths, 1, 4, 2, 64, 16)
    c.verify(c.call(dvl))
    c = Case(3, [0] * 300, 2, 4, 2, 64, 16)
    out, lse = c.call(dvl)
    assert torch.all(out == 0) and torch.all(lse == -float("inf"))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D", [16, 80, 208])
def test_attention_padded_widths_on_blocks_with_many_sequences(dvl, D, fp8):
    # blocks that finish many (sequence, head) pairs reuse their shared memory
    rng = np.random.default_rng(D)
    c = Case(D, [int(n) for n in rng.integers(1, 300, size=150)], 1, 16, 8, D, 16, fp8)
    c.verify(c.call(dvl))
    c = Case(D + 1, [int(n) for n in rng.integers(1, 200, size=90)], 3, 24, 4, D, 48, fp8)
    c.verify(c.call(dvl))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 4])
def test_attention_masked_slots_may_hold_anything(dvl, T, fp8):
    lengths = [1, 3, 70, 129, 200, 2]
    c = Case(T, lengths, T, 8, 2, 128, 16, fp8)
    clean = c.call(dvl)
    c.verify(clean)
    c.poison()
    dirty = c.call(dvl)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_later_tokens_do_not_reach_earlier_rows(dvl, fp8):
    # the newest token's key and value are NaN: only the rows that see it change
    T, lengths = 3, [3, 64, 65, 66, 130]
    c = Case(8, lengths, T, 4, 2, 64, 16, fp8)
    clean = c.call(dvl)
    for b, n in enumerate(lengths):
        at = (int(c.table[b, (n - 1) // 16]), (n - 1) % 16)
        for x in (c.k, c.v):
            x.view(torch.uint8)[at] = 0x7f if fp8 else 0xff
    dirty = c.call(dvl)
    assert torch.equal(clean[0][:, :T - 1], dirty[0][:, :T - 1])
    assert torch.equal(clean[1][:, :T - 1], dirty[1][:, :T - 1])
    assert torch.isnan(dirty[0][:, T - 1]).all()


def test_attention_extreme_scores(dvl):
    # one position far above the rest, scores past 2^10, and a scale of 0
    c = Case(4, [300, 70], 1, 4, 2, 128, 16, std=6.0)
    c.verify(c.call(dvl, scale=2.0), 2.0)
    c.verify(c.call(dvl, scale=0.0), 0.0)
    c.verify(c.call(dvl, scale=-0.1), -0.1)


def test_attention_fp8_query_range(dvl):
    # rows of very large, very small and mixed values: the power of two keeps them exact
    c = Case(6, [100, 40], 1, 4, 2, 128, 16, True)
    c.q[0, 0, 0] *= 2.0 ** 60
    c.q[0, 0, 1] *= 2.0 ** -60
    c.q[0, 0, 2, ::2] *= 2.0 ** -12
    c.q[1, 0, 0] = 0
    # the large row's scores are huge: one position takes all
    c.verify(c.call(dvl, scale=2.0 ** -55), 2.0 ** -55)
    c.verify(c.call(dvl, scale=1.0), 1.0)


def test_attention_strided_queries_and_shapes(dvl):
    c = Case(7, [40, 100, 7], 2, 6, 2, 128, 16)
    fused = torch.zeros(3, 2, 6 * 128 + 512, dtype=torch.bfloat16, device="cuda")
    q = fused[:, :, 256:256 + 768].view(3, 2, 6, 128)
    q.copy_(c.q)
    assert not q.is_contiguous()
    c.verify(c.call(dvl, q=q))
    out, lse = c.call(dvl, want_lse=False)
    assert lse is None
    c.verify((out, None))
    one = Case(9, [40, 100, 7], 1, 6, 2, 128, 16)
    out, lse = one.call(dvl, q=one.q.cuda()[:, 0])
    assert out.shape == (3, 6, 128) and lse.shape == (3, 6)
    one.verify((out, lse))


def test_attention_large_offsets(dvl):
    # pages past 2^32 bytes of the pool
    pages, page, heads, D = 70_000, 64, 8, 128
    pool = torch.empty(pages, page, heads, D, dtype=torch.uint8, device="cuda")
    assert pool.numel() > 1 << 32
    c = Case(3, [150, 64], 1, 8, heads, D, page, True)
    far = pages - 1 - torch.arange(c.k.shape[0], device="cuda")
    pool[far] = c.k.view(torch.uint8)
    c.v = c.k
    c.v_scale = c.k_scale
    want = c.call(dvl)
    c.verify(want)
    table = c.table.clone()
    c.table = torch.where(table >= 0, (pages - 1 - table).int(), table)
    small, c.k, c.v = c.k, pool, pool
    got = c.call(dvl)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attention_status_and_workspace_reuse(dvl):
    c = Case(11, [100, 130, 20], 1, 4, 2, 64, 16)
    cache = dvl.KVCache(c.k, c.v)
    ws = dvl.attention_workspace(cache, 3, 1, 4)
    ws[512 + 16 * 1024:] = 0x7f  # what earlier calls leave in the parts must not matter
    good = c.call(dvl, ws=ws)
    c.verify(good)
    assert dvl.workspace_status(ws) == 0
    table, lengths = c.table.clone(), c.lengths.clone()
    c.table[1, 2] = c.k.shape[0]          # outside the pool
    bad = c.call(dvl, ws=ws)
    assert torch.equal(bad[0][0], good[0][0]) and torch.equal(bad[0][2], good[0][2])  # the others keep theirs
    assert torch.isfinite(bad[0].float()).all()
    assert dvl.workspace_status(ws) == 1 << 2 and dvl.workspace_status(ws) == 0
    c.table = table[:, :7].contiguous()   # 112 tokens: the second sequence is cut
    c.lengths = lengths.clone()
    c.lengths[2] = -5
    cut = c.call(dvl, ws=ws)
    assert dvl.workspace_status(ws) == 1 << 2
    assert torch.all(cut[0][2] == 0)
    c.lengths = torch.tensor([100, 112, -5], dtype=torch.int32, device="cuda")
    c.verify(c.call(dvl, ws=ws))
    assert dvl.workspace_status(ws) == 0
    # the same workspace serves other batches, and other shapes that fit
    ws = dvl.attention_workspace(dvl.KVCache(torch.zeros(1, 1, 2, 256, dtype=torch.bfloat16, device="cuda"),
                                             torch.zeros(1, 1, 2, 256, dtype=torch.bfloat16, device="cuda")), 1, 8, 16)
    for T, Hq, D in [(1, 4, 64), (8, 8, 256), (2, 16, 128), (1, 4, 64), (3, 10, 256), (1, 2, 128)]:
        for fp8 in (False, True):
            x = Case(T * D + Hq, [900, 5, 3000, 129], T, Hq, 2, D, 64, fp8)
            x.verify(x.call(dvl, ws=ws))
    other = Case(12, [5000, 1], 1, 4, 2, 64, 16)
    other.verify(other.call(dvl, ws=ws))


def test_attention_on_another_stream_and_repeatable(dvl):
    c = Case(13, [5000, 300, 9000], 3, 10, 2, 128, 64)
    q = c.q.cuda()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    one = c.call(dvl, q=q, stream=st, ws=dvl.attention_workspace(dvl.KVCache(c.k, c.v), 3, 3, 10, stream=st))
    st.synchronize()
    for _ in range(4):
        two = c.call(dvl, q=q)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


def test_attention_in_a_cuda_graph(dvl):
    c = Case(14, [700, 20], 1, 8, 2, 128, 16)
    q, cache = c.q.cuda(), dvl.KVCache(c.k, c.v)
    ws = dvl.attention_workspace(cache, 2, 1, 8)
    out, lse = dvl.paged_attention(cache, q, c.table, c.lengths, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dvl.paged_attention(cache, q, c.table, c.lengths, out=out, lse=lse, ws=ws)
    c.lengths.copy_(torch.tensor([333, 21], dtype=torch.int32))  # lengths are read at replay
    g.replay()
    torch.cuda.synchronize()
    c.verify((out, lse))


def test_attention_refusals(dvl):
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    n = torch.ones(2, dtype=torch.int32, device="cuda")
    for bad in [(k.float(), k.float()), (k, k[:2]), (k.cpu(), k.cpu()), (k[0], k[0]), (k.transpose(2, 3), k.transpose(2, 3))]:
        with pytest.raises(ValueError):
            dvl.KVCache(*bad)
    with pytest.raises(ValueError):
        dvl.KVCache(k, k, k_scale=0.5)
    cache = dvl.KVCache(k, k)
    ws = dvl.attention_workspace(cache, 2, 1, 4)
    for bad in [dict(q=q.float()), dict(q=q.cpu()), dict(q=q[..., :32]), dict(q=q[0, 0]), dict(table=table.long()),
                dict(table=table[:1]), dict(table=table.cpu()), dict(table=table.t()), dict(lengths=n.long()),
                dict(lengths=n[:1]), dict(out=q.float()), dict(lse=torch.zeros(2, 1, 4, device="cuda").half()),
                dict(ws=ws.cpu())]:
        args = dict(q=q, table=table, lengths=n, ws=ws)
        args.update(bad)
        with pytest.raises(ValueError):
            dvl.paged_attention(cache, **args)
    wide = torch.zeros(2, 9, 4, 64, dtype=torch.bfloat16, device="cuda")   # T above the limit
    odd = torch.zeros(2, 1, 5, 64, dtype=torch.bfloat16, device="cuda")    # heads do not divide
    many = torch.zeros(2, 8, 20, 64, dtype=torch.bfloat16, device="cuda")  # 80 rows per cached head
    for x in (wide, odd, many):
        with pytest.raises(dvl.DvlError):
            dvl.paged_attention(cache, x, table, n, ws=ws)
    for scale in (float("nan"), float("inf")):
        with pytest.raises(dvl.DvlError):
            dvl.paged_attention(cache, q, table, n, ws=ws, scale=scale)
    with pytest.raises(dvl.DvlError) as e:
        dvl.paged_attention(cache, q, table, n, ws=ws[:256])
    assert e.value.status == 4
    with pytest.raises(dvl.DvlError):  # rows off 16-byte boundaries
        dvl.paged_attention(cache, torch.zeros(2, 1, 4, 66, dtype=torch.bfloat16, device="cuda")[..., :64], table, n, ws=ws)
    narrow = torch.zeros(4, 16, 2, 24, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        dvl.attention_workspace(dvl.KVCache(narrow, narrow), 2, 1, 4)
