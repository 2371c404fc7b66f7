"""dvl_cache_keep and the 4-bit pages of dvl_beam_reorder, byte for byte."""
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


KINDS = ["bf16", "fp8", "nvfp4"]


class Pools:
    """Random pools of a cache, viewed as bytes [pages][page][heads * bytes]."""

    def __init__(self, dvl, seed, pages, page, heads, D, kind, layout="tokens"):
        g = torch.Generator().manual_seed(seed)
        shape = (pages, page, heads) if layout == "tokens" else (pages, heads, page)
        sizes = {"bf16": [2 * D] * 2, "fp8": [D] * 2, "nvfp4": [D // 2] * 2 + [D // 16] * 2}[kind]
        self.raw = [torch.randint(256, (*shape, n), generator=g, dtype=torch.uint8).cuda() for n in sizes]
        if layout == "heads":
            self.raw = [x.transpose(1, 2) for x in self.raw]
        k, v = (x.view(torch.bfloat16) if kind == "bf16" else x for x in self.raw[:2])
        more = dict(k_blocks=self.raw[2], v_blocks=self.raw[3]) if kind == "nvfp4" else {}
        self.cache = dvl.KVCache(k, v, **more)

    def bytes(self):
        return [x.contiguous().cpu().numpy() for x in self.raw]


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def tables(rng, lens, page):
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    ids = rng.permutation(pages)
    table, at = np.full((len(lens), max(need) + 1), -1), 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, pages


def run(dvl, seed, seqs, heads, D, page, kind, layout="tokens", M=None, change=None, out=None):
    """seqs: (first, nodes, kept nodes) of each sequence."""
    rng = np.random.default_rng(seed)
    lens = [f + n for f, n, _ in seqs]
    table, pages = tables(rng, lens, page)
    M = max(len(k) for _, _, k in seqs) if M is None else M
    keep = np.full((len(seqs), M), -1)
    for b, (_, _, k) in enumerate(seqs):
        keep[b, :len(k)] = k
    a = dict(table=table, lengths=np.array(lens), first=np.array([f for f, _, _ in seqs]), keep=keep,
             counts=np.array([len(k) for _, _, k in seqs]))
    if change:
        change(a)
    p = Pools(dvl, seed, pages, page, heads, D, kind, layout)
    want = [C.kept(x, a["table"], a["lengths"], a["first"], a["keep"], a["counts"]) for x in p.bytes()]
    got = dvl.cache_keep(p.cache, *(ints(a[n]) for n in ("table", "lengths", "first", "keep", "counts")), lengths_out=out)
    for x, y in zip(p.bytes(), want):
        assert np.array_equal(x, y)
    count = np.clip(a["counts"], 0, M)
    assert got.tolist() == (np.maximum(a["first"], 0) + count).tolist()


def path(rng, nodes, n):
    return [0] + sorted(rng.choice(np.arange(1, nodes), size=n - 1, replace=False).tolist()) if n else []


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,D", [(4, 128), (1, 64), (8, 256), (3, 192), (5, 64)])
def test_keep_paths_of_trees(dvl, kind, heads, D):
    rng = np.random.default_rng(D + heads)
    seqs = [(int(rng.integers(0, 300)), 63, path(rng, 63, int(n))) for n in (1, 7, 0, 20, 63, 2)]
    run(dvl, 1, seqs, heads, D, 16, kind)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("D", [16, 80, 208])
def test_keep_odd_widths(dvl, kind, D):
    rng = np.random.default_rng(D)
    run(dvl, 2, [(17, 40, path(rng, 40, 9)), (0, 31, path(rng, 31, 30))], 3, D, 16, kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [1, 7, 48, 1000])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
def test_keep_pages(dvl, kind, page, layout):
    rng = np.random.default_rng(page)
    run(dvl, 3, [(5, 130, path(rng, 130, 64)), (70, 65, path(rng, 65, 33))], 2, 128, page, kind, layout)


@pytest.mark.parametrize("kind", KINDS)
def test_keep_long_lists(dvl, kind):
    # rows are targets and sources at once, over many steps of a block
    rng = np.random.default_rng(4)
    seqs = [(3, 5000, path(rng, 5000, 2500)), (0, 4097, path(rng, 4097, 4000)), (9, 300, path(rng, 300, 299)),
            (1, 2000, list(range(1000, 2000))), (0, 1500, list(range(1, 1500)))]
    run(dvl, 4, seqs, 4, 64, 32, kind)


def test_keep_nothing_and_everything(dvl):
    run(dvl, 5, [(10, 5, []), (0, 7, list(range(7))), (64, 64, list(range(64)))], 2, 64, 16, "bf16")
    run(dvl, 6, [(10, 5, [])], 2, 64, 16, "bf16")  # M = 0
    run(dvl, 7, [(10, 5, [0, 3])], 2, 64, 16, "nvfp4", M=40)


@pytest.mark.parametrize("kind", KINDS)
def test_keep_places_that_are_not_there_move_nothing(dvl, kind):
    def change(a):
        a["keep"][0, 2] = 100_000           # past the length
        a["keep"][1, 1] = -7
        a["table"][2, 1] = 10_000           # a page id outside the pool
        a["counts"][3] = 1_000_000          # more than there are
        a["first"][4] = -3
        a["counts"][5] = -1
        a["lengths"][6] = 1 << 30           # past the table
        a["lengths"][7] = -5
    rng = np.random.default_rng(8)
    run(dvl, 8, [(5, 40, path(rng, 40, 8)) for _ in range(8)], 2, 64, 16, kind, change=change)


def test_keep_many_sequences_and_a_given_output(dvl):
    rng = np.random.default_rng(9)
    seqs = [(int(rng.integers(0, 40)), 15, path(rng, 15, int(rng.integers(0, 15)))) for _ in range(500)]
    run(dvl, 9, seqs, 1, 64, 16, "fp8", out=torch.empty(500, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("kind", KINDS)
def test_keep_values_that_are_the_keys(dvl, kind):
    # one pool for both: its rows move once (M past a block's step, so that rows
    # that have moved would be moved again)
    rng = np.random.default_rng(13)
    seqs = [(0, 4000, path(rng, 4000, 2500)), (2, 900, path(rng, 900, 700))]
    lens = [f + n for f, n, _ in seqs]
    table, pages = tables(rng, lens, 16)
    p = Pools(dvl, 13, pages, 16, 8, 64, kind)
    k = p.raw[0].view(torch.bfloat16) if kind == "bf16" else p.raw[0]
    more = dict(k_blocks=p.raw[2], v_blocks=p.raw[2]) if kind == "nvfp4" else {}
    keep = np.full((2, 2500), -1)
    for b, (_, _, x) in enumerate(seqs):
        keep[b, :len(x)] = x
    first, counts = [f for f, _, _ in seqs], [len(x) for _, _, x in seqs]
    want = [C.kept(x, table, lens, first, keep, counts) for x in p.bytes()[::2]]
    for _ in range(3):
        q = Pools(dvl, 13, pages, 16, 8, 64, kind)
        for x, y in zip(p.raw, q.raw):
            x.copy_(y)
        dvl.cache_keep(dvl.KVCache(k, k, **more), ints(table), ints(lens), ints(first), ints(keep), ints(counts))
        for x, y in zip(p.bytes()[::2], want):
            assert np.array_equal(x, y)


def test_keep_strided_lists(dvl):
    rng = np.random.default_rng(10)
    lens = [50, 60]
    table, pages = tables(rng, lens, 16)
    p = Pools(dvl, 10, pages, 16, 2, 64, "bf16")
    wide_table, wide_keep = ints(np.pad(table, ((0, 0), (0, 5)), constant_values=-9)), ints([[0, 4, 9, -1, 77], [0, 1, 5, 8, 77]])
    want = [C.kept(x, table, lens, [30, 40], np.array([[0, 4, 9, -1], [0, 1, 5, 8]]), [3, 4]) for x in p.bytes()]
    got = dvl.cache_keep(p.cache, wide_table[:, :table.shape[1]], ints(lens), ints([30, 40]), wide_keep[:, :4], ints([3, 4]))
    assert got.tolist() == [33, 44] and all(np.array_equal(x, y) for x, y in zip(p.bytes(), want))
    empty = dvl.cache_keep(p.cache, wide_table[:0], ints([]), ints([]), wide_keep[:0], ints([]))
    assert empty.shape == (0,)
    with pytest.raises(dvl.DvlError):
        lengths = ints(lens)
        dvl.cache_keep(p.cache, wide_table, lengths, ints([30, 40]), wide_keep[:, :4], ints([3, 4]), lengths_out=lengths)


@pytest.mark.parametrize("heads,D,page,length", [(2, 64, 16, 37), (4, 128, 48, 47), (8, 256, 64, 191), (1, 192, 7, 6),
                                                 (2, 64, 16, 32), (3, 64, 1000, 999)])
def test_reorder_copies_the_4_bit_page(dvl, heads, D, page, length):
    batch, beams = 3, 4
    width = length // page + 2
    pages = batch * beams * (width + 1)
    p = Pools(dvl, 11, pages, page, heads, D, "nvfp4", "heads" if D == 128 else "tokens")
    rng = np.random.default_rng(12)
    ids = rng.permutation(pages)
    table = ids[:batch * beams * width].reshape(batch, beams, width)
    spare = ids[batch * beams * width:].reshape(batch, beams)
    parents = rng.integers(-1, beams, size=(batch, beams))
    lengths = np.full((batch, beams), length)
    want = p.bytes()
    slot, r = length // page, length % page
    for b in range(batch):
        for i in range(beams):
            if parents[b, i] >= 0:
                for x in want:
                    x[spare[b, i], :r] = x[table[b, parents[b, i], slot], :r]
    _, t, n = dvl.beam_reorder(ints(parents), cache=p.cache, table=ints(table), lengths=ints(lengths), spare=ints(spare))
    for x, y in zip(p.bytes(), want):
        assert np.array_equal(x, y)
    for b in range(batch):
        for i in range(beams):
            if parents[b, i] >= 0:
                row = table[b, parents[b, i]].copy()
                row[slot] = spare[b, i]
                assert t[b, i].tolist() == row.tolist() and int(n[b, i]) == length
