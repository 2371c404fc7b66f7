"""dvl_paged_attention over NVFP4 caches against the 64-bit form, within the
bounds of step_reference.attention_bounds (weights are f16, as with E4M3)."""
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


class Case:
    """A 4-bit cache, its table and the queries of one call."""

    def __init__(self, seed, lengths, T, Hq, heads, D, page, layout="tokens", spread=6):
        g = torch.Generator().manual_seed(seed)
        need = [-(-max(n, 0) // page) for n in lengths]
        width, pages = max(max(need), 1) + 1, sum(need) + 2
        shape = (pages, page, heads) if layout == "tokens" else (pages, heads, page)
        self.scales = (0.01, 0.02)
        self.codes = [torch.randint(256, (*shape, D // 2), generator=g, dtype=torch.uint8) for _ in range(2)]
        # scales of 2^-spread .. 2^0.9 and some of 0
        self.blocks = [torch.randint(0x38 + 8 - 8 * spread, 0x38 + 16, (*shape, D // 16), generator=g).clamp(min=0).to(torch.uint8)
                       for _ in range(2)]
        self.codes, self.blocks = ([x.cuda() for x in y] for y in (self.codes, self.blocks))
        if layout == "heads":
            self.codes, self.blocks = ([x.transpose(1, 2) for x in y] for y in (self.codes, self.blocks))
        ids = torch.randperm(pages, generator=g).int()
        table, at = torch.full((len(lengths), width), -1, dtype=torch.int32), 0
        used = torch.zeros(pages, page, dtype=torch.bool)
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
            for p in range(n):
                used[table[b, p].long(), :min(page, lengths[b] - p * page)] = True
        self.dead = ~used
        self.q = (torch.randn(len(lengths), T, Hq, D, generator=g) * 20).bfloat16()
        self.table, self.lengths, self.page = table.cuda(), torch.tensor(lengths, dtype=torch.int32).cuda(), page

    def poison(self):
        """NaN in every slot that no sequence's length reaches."""
        for x in self.blocks:
            x[self.dead.cuda()] = 0x7f
        for x in self.codes:
            x[self.dead.cuda()] = 0xff

    def call(self, dvl, **kw):
        self.cache = dvl.KVCache(*self.codes, k_scale=self.scales[0], v_scale=self.scales[1], k_blocks=self.blocks[0],
                                 v_blocks=self.blocks[1])
        return dvl.paged_attention(self.cache, kw.pop("q", self.q.cuda()), self.table, self.lengths, **kw)

    def verify(self, got, scale=None):
        k, v = (C.decode(c.contiguous().cpu().numpy(), b.contiguous().cpu().numpy(), s)
                for c, b, s in zip(self.codes, self.blocks, self.scales))
        ref = R.attention(self.q.float().numpy().astype(np.float64), k, v, self.table.cpu().numpy(),
                          self.lengths.cpu().numpy(), self.q.shape[3] ** -0.5 if scale is None else scale)
        tol, tol_lse = R.attention_bounds(*ref, n_max=int(self.lengths.max()), fp8=True)
        out = got[0].float().cpu().numpy().reshape(ref[0].shape)
        err = np.abs(out - ref[0])
        assert np.all(err <= tol), (err - tol).max()
        if got[1] is not None:
            lse = got[1].cpu().numpy().reshape(ref[1].shape)
            finite = np.isfinite(ref[1])
            assert np.array_equal(lse[~finite], ref[1][~finite])
            assert np.all(np.abs(lse[finite] - ref[1][finite]) <= tol_lse[finite])


@pytest.mark.parametrize("Hq,heads,D", [(20, 4, 128), (8, 8, 64), (16, 2, 256), (6, 2, 192), (40, 8, 128), (1, 1, 64),
                                        (3, 3, 256)])
@pytest.mark.parametrize("T", [1, 3])
def test_attention4_heads_and_widths(dvl, Hq, heads, D, T):
    c = Case(D + Hq + T, [1, 63, 64, 65, 200, 0, 131], T, Hq, heads, D, 16)
    c.verify(c.call(dvl))


@pytest.mark.parametrize("T,G", [(1, 1), (2, 8), (3, 5), (8, 8), (8, 1), (1, 64), (5, 7), (4, 4), (1, 17)])
@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_attention4_query_rows(dvl, T, G, D):
    # up to 64 query rows per cached head; lengths below T leave rows empty
    c = Case(T * 100 + G, [0, 1, T - 1, T, 67, 130], T, 2 * G, 2, D, 32)
    c.verify(c.call(dvl))


@pytest.mark.parametrize("page", [1, 7, 16, 48, 64, 100, 1000])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
def test_attention4_pages(dvl, page, layout):
    for D in (64, 128):
        c = Case(page, [5, 64, 333, 128, 1], 2, 10, 2, D, page, layout)
        c.verify(c.call(dvl))


def test_attention4_long_sequences_are_split_and_joined(dvl):
    for lengths, heads, D in [([20011], 1, 128), ([9000, 3, 0, 30000], 2, 64), ([12345], 2, 256), ([7777], 1, 192)]:
        c = Case(len(lengths), lengths, 1, 4 * heads, heads, D, 64)
        c.verify(c.call(dvl))
    c = Case(5, [7001, 64], 3, 8, 1, 128, 64)
    c.verify(c.call(dvl))


def test_attention4_many_sequences(dvl):
    rng = np.random.default_rng(1)
    lengths = [int(n) if rng.random() > 0.1 else 0 for n in rng.integers(1, 150, size=700)]
    c = Case(2, lengths, 1, 4, 2, 64, 16)
    c.verify(c.call(dvl))
    # blocks that finish many (sequence, head) pairs reuse their shared memory
    for D, T in ((192, 1), (128, 3), (256, 2)):
        c = Case(D, [int(n) for n in rng.integers(1, 300, size=90)], T, 16, 8, D, 48)
        c.verify(c.call(dvl))


@pytest.mark.parametrize("T", [1, 4])
@pytest.mark.parametrize("D", [64, 128, 192])
def test_attention4_masked_slots_may_hold_anything(dvl, T, D):
    c = Case(T, [1, 3, 70, 129, 200, 2], T, 8, 2, D, 16)
    clean = c.call(dvl)
    c.verify(clean)
    c.poison()
    dirty = c.call(dvl)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("G", [2, 5, 8, 16])
def test_attention4_later_tokens_do_not_reach_earlier_rows(dvl, G, D):
    # the newest token's scales are NaN: only the rows that see it change
    T, lengths = 3, [3, 64, 65, 66, 130]
    c = Case(8, lengths, T, 2 * G, 2, D, 16)
    clean = c.call(dvl)
    for b, n in enumerate(lengths):
        for x in c.blocks:
            x[int(c.table[b, (n - 1) // 16]), (n - 1) % 16] = 0x7f
    dirty = c.call(dvl)
    assert torch.equal(clean[0][:, :T - 1], dirty[0][:, :T - 1])
    assert torch.equal(clean[1][:, :T - 1], dirty[1][:, :T - 1])
    assert torch.isnan(dirty[0][:, T - 1]).all()


def test_attention4_extreme_values(dvl):
    # every finite scale there is, scores far apart, and scales of the call
    for seed, spread in ((1, 15), (2, 1)):
        c = Case(seed, [300, 70], 1, 4, 2, 128, 16, spread=spread)
        for scale in (2.0, 0.0, -0.1):
            c.verify(c.call(dvl, scale=scale), scale)
    c = Case(3, [300], 1, 4, 2, 64, 16)
    for x in c.blocks:
        x.fill_(0x7e)  # the largest block scale
    c.verify(c.call(dvl))


def test_attention4_one_row_alone_keeps_a_long_tail(dvl):
    # 40,000 positions 18 nats below one: their share stays
    n = 40001
    c = Case(4, [n], 1, 4, 1, 64, 64)
    c.codes[0].zero_()
    c.blocks[0].fill_(0x38)
    page, slot = int(c.table[0, 100]), 5
    c.codes[0][page, slot, 0, 0] = 0x02  # +1 at d = 0
    c.q = torch.zeros_like(c.q)
    c.q[..., 0] = 18.0 * 64 ** 0.5 / c.scales[0]
    c.codes[1].fill_(0x22)  # +1 everywhere
    c.blocks[1].fill_(0x38)
    c.codes[1][page, slot] = 0
    out = c.call(dvl)[0].double().cpu()
    want = (n - 1) * np.exp(-18.0) * c.scales[1] / (1 + (n - 1) * np.exp(-18.0))
    # weights of 2^-26 are normal f16 numbers; a score of 18 is off by (D + 4) u of it
    assert torch.all((out - want).abs() <= want * (2.0 ** -8 + 2.0 ** -11 + 2 * 18 * 68 * 2.0 ** -24 + 2.0 ** -11))


def test_attention4_bad_pages_and_lengths(dvl):
    c = Case(5, [100, 100, 100], 1, 4, 2, 64, 16)
    clean = c.call(dvl)[0]
    ws = dvl.attention_workspace(c.cache, 3, 1, 4)
    c.table[1, 2] = 10_000
    c.lengths[2] = 1 << 20
    c.table[2, 7:] = 0
    got = c.call(dvl, ws=ws)[0]
    assert torch.equal(got[0], clean[0]) and torch.isfinite(got.float()).all()
    assert dvl.workspace_status(ws) & (1 << 2)


def test_attention4_shares_a_workspace_and_a_graph(dvl):
    # calls of different cache types share one workspace, eagerly and replayed
    four = Case(6, [3000, 17, 0], 2, 8, 2, 128, 16)
    want = four.call(dvl)
    kv = [torch.randn(40, 16, 2, 128, device="cuda").bfloat16() for _ in range(2)]
    sixteen = dvl.KVCache(*kv)
    table, lengths = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20), torch.tensor([320, 99], dtype=torch.int32, device="cuda")
    q16 = torch.randn(2, 1, 8, 128, device="cuda").bfloat16()
    want16 = dvl.paged_attention(sixteen, q16, table, lengths)
    ws = max((dvl.attention_workspace(four.cache, 3, 2, 8), dvl.attention_workspace(sixteen, 2, 1, 8)),
             key=lambda t: t.numel())
    q = four.q.cuda()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")

    def both():
        a = dvl.paged_attention(four.cache, q, four.table, four.lengths, out=out, lse=lse, ws=ws)
        return a, dvl.paged_attention(sixteen, q16, table, lengths, ws=ws)
    for got, ref in zip(both(), (want, want16)):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_nvfp4_cache_refusals(dvl):
    k = torch.zeros(4, 16, 2, 64, dtype=torch.uint8, device="cuda")
    s = torch.zeros(4, 16, 2, 8, dtype=torch.uint8, device="cuda")
    dvl.KVCache(k, k, k_blocks=s, v_blocks=s.view(torch.float8_e4m3fn))
    dvl.KVCache(k[:1, :1, :1], k[:1, :1, :1], k_blocks=s[:1, :1, :1], v_blocks=s[:1, :1, :1])
    for kw in (dict(k_blocks=s), dict(k_blocks=s, v_blocks=s[..., :4]), dict(k_blocks=s, v_blocks=s.cpu()),
               dict(k_blocks=s, v_blocks=s.float()), dict(k_blocks=s, v_blocks=s.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            dvl.KVCache(k, k, **kw)
    with pytest.raises(ValueError):
        dvl.KVCache(k.view(torch.int8), k.view(torch.int8), k_blocks=s, v_blocks=s)
    with pytest.raises(ValueError):  # D of 96
        dvl.KVCache(k[..., :48], k[..., :48], k_blocks=s[..., :6], v_blocks=s[..., :6])
    cache = dvl.KVCache(k, k, k_blocks=s, v_blocks=s)
    with pytest.raises(ValueError):
        dvl.paged_attention(cache, torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda"),
                            torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
