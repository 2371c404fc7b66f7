"""dvl_qk_norm_rope against the 64-bit form, within the bounds of cache_reference."""
import numpy as np
import pytest

import cache_reference as C

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


def f64(x):
    return x.float().cpu().numpy().astype(np.float64)


def u8(x):
    return x.contiguous().view(torch.uint8).cpu().numpy()


class Case:
    """New tokens of some sequences and the cache they go to."""

    def __init__(self, seed, news, Hq, H, D, page, kind="bf16", padding=0, ragged=True, layout="tokens", norm=True,
                 rot=None, interleaved=False, theta=1e6):
        # news: (tokens before, new tokens) of each sequence
        g = torch.Generator().manual_seed(seed)
        self.news, self.kind, self.D, self.H, self.page = news, kind, D, H, page
        lens = [p + n for p, n in news]
        need = [-(-max(n, 0) // page) for n in lens]
        pages, width = sum(need) + 2, max(max(need), 1) + 1
        ids = torch.randperm(pages, generator=g).int()
        table, at = torch.full((len(news), width), -1, dtype=torch.int32), 0
        for b, n in enumerate(need):
            table[b, :n] = ids[at:at + n]
            at += n
        self.table, self.lengths = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        self.rows = sum(n for _, n in news) + padding
        starts = np.concatenate([[0], np.cumsum([n for _, n in news])])
        self.starts = torch.tensor(starts, dtype=torch.int32).cuda() if ragged else None
        self.where = C.places(self.rows, lens, starts)
        qkv = (torch.randn(self.rows, Hq + 2 * H, D, generator=g) * 2).bfloat16().cuda()
        self.q, self.k, self.v = qkv[:, :Hq], qkv[:, Hq:Hq + H], qkv[:, Hq + H:]
        self.wq, self.wk = ((1 + 0.2 * torch.randn(D, generator=g)).bfloat16().cuda() if norm else None for _ in range(2))
        self.rot = D if rot is None else rot
        self.interleaved, self.theta, self.eps = interleaved, theta, 1e-5
        shape = (pages, page, H) if layout == "tokens" else (pages, H, page)

        def pool(last, fill):
            x = torch.full((*shape, last), fill, dtype=torch.uint8).cuda()
            return x if layout == "tokens" else x.transpose(1, 2)
        self.scales, blocks = {"bf16": (1.0, 1.0), "fp8": (0.03, 0.02), "nvfp4": (0.002, 0.004)}[kind], {}
        last = {"bf16": 2 * D, "fp8": D, "nvfp4": D // 2}[kind]
        self.raw = [pool(last, 0xee), pool(last, 0xdd)]
        self.blocks = [pool(D // 16, 0xcc), pool(D // 16, 0xbb)] if kind == "nvfp4" else None
        self.was = [x.clone() for x in self.raw + (self.blocks or [])]
        if kind == "nvfp4":
            blocks = dict(k_blocks=self.blocks[0], v_blocks=self.blocks[1])
        pools = [x.view(torch.bfloat16) if kind == "bf16" else x.view(torch.float8_e4m3fn) if kind == "fp8" else x
                 for x in self.raw]
        self.pools = (pools, dict(k_scale=self.scales[0], v_scale=self.scales[1], **blocks))

    def freqs(self):
        return [self.theta ** (-2 * i / self.rot) for i in range(self.rot // 2)]

    def call(self, dvl, **kw):
        pools, named = self.pools
        self.cache = dvl.KVCache(*pools, **named)
        rope = dvl.Rope(self.rot, theta=self.theta, interleaved=self.interleaved) if self.rot else None
        args = dict(q=self.q, k=self.k, v=self.v, rope=rope, q_weight=self.wq, k_weight=self.wk, eps=self.eps,
                    cache=self.cache, table=self.table, lengths=self.lengths, starts=self.starts)
        args.update(kw)
        return dvl.qk_norm_rope(args.pop("q"), args.pop("k"), args.pop("v"), **args)

    def verify(self, q_out, k_out=None, positions=None, fill=None):
        """Every output and every byte of the cache; fill: what q_out's padded rows held."""
        used = np.array([b >= 0 for b, _ in self.where])
        places = np.array([p for _, p in self.where])
        pos = places if positions is None else np.asarray(positions)
        freqs = self.freqs() if self.rot else None
        w = [None if x is None else f64(x) for x in (self.wq, self.wk)]
        z, err = C.turned(f64(self.q), w[0], self.eps, pos, freqs, self.interleaved)
        got = f64(q_out).reshape(z.shape)
        off = np.abs(got - z)[used]
        assert np.all(off <= C.bf16_bound(z, err)[used]), off.max()
        if fill is not None:
            assert np.all(got[~used] == fill)
        zk, ek = C.turned(f64(self.k), w[1], self.eps, pos, freqs, self.interleaved)
        zv = f64(self.v)
        if k_out is not None:
            assert np.all((np.abs(f64(k_out).reshape(zk.shape) - zk) <= C.bf16_bound(zk, ek))[used])
        table, pages = self.table.cpu().numpy(), self.raw[0].shape[0]
        written = np.zeros((pages, self.page), dtype=bool)
        at = []
        for r, (b, p) in enumerate(self.where):
            if b >= 0 and 0 <= p < table.shape[1] * self.page and 0 <= table[b, p // self.page] < pages:
                at.append((r, table[b, p // self.page], p % self.page))
                written[at[-1][1:]] = True
        rows, pg, slot = (np.array([x[i] for x in at], dtype=int) for i in range(3))
        for i, (x, e) in enumerate(((zk, ek), (zv, np.zeros_like(zv)))):
            x, e, raw = x[rows], e[rows], u8(self.raw[i])[pg, slot]
            if self.kind == "bf16":
                val = f64(self.raw[i].contiguous().view(torch.bfloat16))[pg, slot]
                assert np.all(np.abs(val - x) <= C.bf16_bound(x, e))
            elif self.kind == "fp8":
                C.check_e4m3(raw, x, e, self.scales[i])
            else:
                C.check_nvfp4(raw, u8(self.blocks[i])[pg, slot], x, e, self.scales[i])
        for now, was in zip(self.raw + (self.blocks or []), self.was):
            assert np.array_equal(u8(now)[~written], u8(was)[~written])


KINDS = ["bf16", "fp8", "nvfp4"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,H,D", [(20, 4, 128), (8, 8, 64), (16, 2, 256), (5, 5, 192), (1, 1, 128), (7, 1, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_heads_and_widths(dvl, Hq, H, D, kind, interleaved):
    c = Case(D + Hq, [(0, 1), (731, 3), (15, 2), (40000, 1)], Hq, H, D, 16, kind, interleaved=interleaved)
    c.verify(*c.call(dvl))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("D,rot", [(16, 16), (48, 16), (80, 80), (80, 48), (208, 112), (112, 0), (128, 64), (256, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_partial_widths(dvl, D, rot, kind, interleaved):
    for norm in (False, True):
        c = Case(D + rot, [(100, 5), (3, 4)], 6, 2, D, 16, kind, rot=rot, interleaved=interleaved, norm=norm)
        c.verify(*c.call(dvl))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [1, 7, 16, 48, 1000])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
def test_rope_pages(dvl, page, layout, kind):
    c = Case(page, [(5, 60), (64, 1), (0, 33)], 10, 2, 128, page, kind, layout=layout)
    c.verify(*c.call(dvl))


@pytest.mark.parametrize("kind", KINDS)
def test_rope_rows_of_every_count(dvl, kind):
    # from one row, whose heads are shared by many warps, to more rows than warps
    for rows in (1, 2, 3, 17, 100, 700, 2500):
        c = Case(rows, [(rows % 7, rows)], 9, 3, 64, 32, kind)
        c.verify(*c.call(dvl))


def test_rope_ragged_rows_and_padding(dvl):
    rng = np.random.default_rng(0)
    for B in (1, 2, 31, 33, 200, 1100):
        news = [(int(rng.integers(0, 50)), int(rng.integers(0, 4)) if rng.random() < 0.7 else 0) for _ in range(B)]
        news[B // 2] = (9, 3)
        c = Case(B, news, 4, 2, 64, 16, padding=13)
        out = torch.full(c.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        k_out = torch.full(c.k.shape, 5.0, dtype=torch.bfloat16, device="cuda")
        got = c.call(dvl, q_out=out, k_out=k_out)
        assert got[0] is out and got[1] is k_out
        c.verify(out, k_out, fill=7.0)
        assert torch.all(k_out[c.rows - 13:] == 5.0)


@pytest.mark.parametrize("T", [1, 3, 8])
def test_rope_sequences_and_tokens(dvl, T):
    # [B][T] rows, and the same as rows; the kernel's positions are the tokens' places
    c = Case(T, [(n, T) for n in (0, 15, 16, 99)], 8, 2, 128, 16, ragged=False)
    out, k_out = c.call(dvl)
    assert k_out is None
    c.verify(out)
    q, k, v = (x.contiguous().view(4, T, -1, 128) for x in (c.q, c.k, c.v))
    again = c.call(dvl, q=q, k=k, v=v)[0]
    assert torch.equal(again.view_as(out), out)
    if T > 1:  # a part of longer rows: not evenly spaced
        longer = torch.zeros(4, T + 1, 8, 128, dtype=torch.bfloat16, device="cuda")[:, :T]
        with pytest.raises(ValueError):
            c.call(dvl, q=longer, k=k, v=v)


@pytest.mark.parametrize("kind", KINDS)
def test_rope_places_outside_the_table_or_the_pool_are_not_written(dvl, kind):
    c = Case(3, [(-2, 4), (30, 6), (10, 3), (0, 2)], 4, 2, 64, 16, kind)
    # sequence 1's last places lie past its table's end; a page id of sequence 2 is wrong
    c.table = c.table[:, :2].contiguous()
    c.lengths[1] = 36
    c.table[2, 0], c.table[3, 0] = 10_000, -5
    c.verify(*c.call(dvl))


def test_rope_positions_of_a_tree(dvl):
    # rotated by depth, written by place
    c = Case(4, [(20, 7), (3, 7)], 6, 3, 128, 16)
    depth = [20, 21, 21, 22, 22, 22, 23, 3, 4, 4, 5, 5, 5, 6]
    pos = torch.tensor(depth, dtype=torch.int32, device="cuda")
    c.verify(c.call(dvl, positions=pos)[0], positions=depth)


def test_rope_without_a_cache(dvl):
    c = Case(5, [(0, 50)], 6, 2, 128, 16)
    depth = [int(x) for x in np.random.default_rng(1).integers(-1000, 2 ** 31, size=50)]
    depth[:2] = [2 ** 31 - 1, -2 ** 31]
    rope = dvl.Rope(128, theta=c.theta)
    out, k_out = dvl.qk_norm_rope(c.q, c.k, rope=rope, q_weight=c.wq, k_weight=c.wk, eps=c.eps,
                                  positions=torch.tensor(depth, dtype=torch.int32, device="cuda"))
    z, err = C.turned(f64(c.q), f64(c.wq), c.eps, depth, c.freqs(), False)
    # (64-bit angles of 2^31 positions are themselves good to 2^-21 only)
    assert np.all(np.abs(f64(out) - z) <= C.bf16_bound(z, 2 * err))
    z, err = C.turned(f64(c.k), f64(c.wk), c.eps, depth, c.freqs(), False)
    assert np.all(np.abs(f64(k_out) - z) <= C.bf16_bound(z, 2 * err))
    # the norm alone
    out, k_out = dvl.qk_norm_rope(c.q, c.k, q_weight=c.wq, k_weight=c.wk, eps=c.eps)
    z, err = C.turned(f64(c.q), f64(c.wq), c.eps, None, None, False)
    assert np.all(np.abs(f64(out) - z) <= C.bf16_bound(z, err))
    # only the keys normed; nothing to do at all
    out, k_out = dvl.qk_norm_rope(c.q, c.k, k_weight=c.wk, eps=c.eps)
    assert torch.equal(out, c.q)
    assert torch.equal(k_out, dvl.qk_norm_rope(c.q, c.k, q_weight=c.wq, k_weight=c.wk, eps=c.eps)[1])


def test_rope_far_positions_and_given_frequencies(dvl):
    c = Case(6, [(262139, 4), (99991, 2)], 2, 1, 64, 64)
    c.verify(*c.call(dvl))
    freqs = [(-1) ** i * 3.0 / (1 + i) for i in range(32)]
    rope = dvl.Rope(64, freqs=freqs)
    c.freqs = lambda: freqs
    c.verify(c.call(dvl, rope=rope)[0])


def test_rope_in_place(dvl):
    for H, D, interleaved in ((3, 128, False), (3, 80, True)):
        c = Case(7, [(5, 40)], 6, H, D, 16, interleaved=interleaved)
        want = c.call(dvl, k_out=torch.empty_like(c.k.contiguous()))
        q, k = c.q.clone(), c.k.clone()
        qkv = torch.cat([c.q, c.k, c.v], 1)  # in the projection's own rows
        got = c.call(dvl, q=qkv[:, :6], k=qkv[:, 6:6 + H], v=qkv[:, 6 + H:], q_out=qkv[:, :6], k_out=qkv[:, 6:6 + H])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(qkv[:, 6 + H:], c.v) and torch.equal(c.q, q) and torch.equal(c.k, k)
        c.verify(*want)


def test_rope_strided_outputs(dvl):
    c = Case(8, [(5, 20)], 6, 2, 64, 16)
    heads_first = torch.zeros(6, 20, 64, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    c.verify(c.call(dvl, q_out=heads_first)[0])
    wide = torch.zeros(20, 9, 64, dtype=torch.bfloat16, device="cuda")
    c.verify(c.call(dvl, q_out=wide[:, 2:8])[0])
    assert torch.all(wide[:, :2] == 0) and torch.all(wide[:, 8:] == 0)


@pytest.mark.parametrize("kind", KINDS)
def test_rope_large_small_and_zero_rows(dvl, kind):
    c = Case(9, [(0, 6)], 4, 2, 64, 16, kind)
    for x in (c.q, c.k):
        x[0] = 0
        x[1] *= 2.0 ** 40
        x[2] *= 2.0 ** -40
    c.v[0], c.v[1] = 0, c.v[1] * 2.0 ** 20  # saturates in 8 and 4 bits
    c.verify(*c.call(dvl))


@pytest.mark.parametrize("kind", KINDS)
def test_rope_nan_and_infinity_stay_in_their_heads(dvl, kind):
    c = Case(10, [(0, 4)], 4, 2, 64, 16, kind)
    clean = c.call(dvl)[0].clone()
    cache = [u8(x) for x in c.raw]
    c.q[1, 2, 5], c.k[2, 1, 7], c.v[3, 0, 9] = float("nan"), float("inf"), float("nan")
    dirty = c.call(dvl)[0]
    same = torch.ones(4, 4, dtype=torch.bool)
    same[1, 2] = False
    assert torch.equal(clean.cpu()[same], dirty.cpu()[same]) and torch.isnan(dirty[1, 2]).all()
    page = int(c.table[0, 0])
    for was, now, (t, h), blocks in ((cache[0], u8(c.raw[0]), (2, 1), 0), (cache[1], u8(c.raw[1]), (3, 0), 1)):
        keep = np.ones((4, 2), dtype=bool)
        keep[t, h] = False
        assert np.array_equal(was[page, :4][keep], now[page, :4][keep])
        # an infinity's norm is 0: it and the other half of its pair (32 further)
        # are infinity times 0, the rest 0; a value's NaN is its own
        nan = [9] if blocks else [7, 39]
        if kind == "nvfp4":
            s = u8(c.blocks[blocks])[page, t, h]
            assert (s == 0x7f).tolist() == [i in [x // 16 for x in nan] for i in range(4)]
        else:
            x = c.raw[blocks].contiguous().view(torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn)[page, t, h].float()
            assert torch.isnan(x).nonzero().flatten().tolist() == nan


def test_rope_empty_calls(dvl):
    c = Case(11, [(3, 2)], 4, 2, 64, 16)
    out, _ = c.call(dvl, q=c.q[:0], k=c.k[:0], v=c.v[:0], starts=torch.zeros(2, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 64)
    # no sequence at all: every row is padding
    filled = torch.full_like(c.q.contiguous(), 3.0)
    c.call(dvl, table=c.table[:0], lengths=c.lengths[:0], starts=torch.zeros(1, dtype=torch.int32, device="cuda"),
           q_out=filled)
    assert torch.all(filled == 3.0)


def test_rope_refusals(dvl):
    with pytest.raises(ValueError):
        dvl.Rope(24)
    with pytest.raises(ValueError):
        dvl.Rope(32, freqs=[1.0] * 15)
    with pytest.raises(ValueError):
        dvl.Rope(32, theta=float("inf"))
    c = Case(12, [(3, 2)], 4, 2, 64, 16)
    with pytest.raises(dvl.DvlError):
        c.call(dvl, q_out=c.k.expand(2, 2, 64).repeat(1, 2, 1)[:, :1].expand(2, 4, 64))
    grad = c.q.clone().requires_grad_()
    assert not c.call(dvl, q=grad)[0].requires_grad
