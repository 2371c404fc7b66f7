"""dvl_beam_reorder: rows move bit for bit, the page tables follow, and each
new beam's partly filled page is its own."""
import numpy as np
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


def moved(x, parents):
    """x [batch][beams][...], parents [batch][k] (NumPy): the definition."""
    batch, beams = x.shape[:2]
    out = np.zeros((batch, parents.shape[1]) + x.shape[2:], dtype=x.dtype)
    for b in range(batch):
        for i, p in enumerate(parents[b]):
            if 0 <= p < beams:
                out[b, i] = x[b, p]
    return out


def choose(seed, batch, beams, k):
    rng = np.random.default_rng(seed)
    p = rng.integers(0, beams, size=(batch, k)).astype(np.int32)
    p[rng.random((batch, k)) < 0.1] = -1
    return p


@pytest.mark.parametrize("batch,beams,k", [(1, 1, 1), (1, 4, 4), (3, 8, 5), (2, 3, 32), (5, 32, 7)])
def test_reorder_states(dvl, batch, beams, k):
    rng = np.random.default_rng(batch + beams)
    p = choose(k, batch, beams, k)
    tails = [(2560,), (1,), (3, 7), (4097,), (8, 64, 64), (8192,), (5, 1)]
    kinds = [np.int16, np.int32, np.uint8, np.uint8, np.float32, np.uint8, np.int64]
    states = [rng.integers(0, 100, size=(batch, beams) + t).astype(d) for t, d in zip(tails, kinds)]
    out, table, lengths = dvl.beam_reorder(torch.from_numpy(p).cuda(), [torch.from_numpy(s).cuda() for s in states])
    assert table is None and lengths is None
    for s, o in zip(states, out):
        assert np.array_equal(o.cpu().numpy(), moved(s, p))


def test_reorder_parents_outside_the_beams_give_zeros(dvl):
    x = torch.ones(1, 2, 100, device="cuda")
    p = torch.tensor([[0, 2, -1, 1, 2147483647, -2147483648]], dtype=torch.int32, device="cuda")
    out = dvl.beam_reorder(p, [x])[0][0]
    assert out.sum(dim=2).tolist() == [[100.0, 0.0, 0.0, 100.0, 0.0, 0.0]]


def test_reorder_large_rows(dvl):
    # more than 2^32 bytes moved, the last row past 2^32
    x = torch.empty(1, 3, 1_500_000_016, dtype=torch.uint8, device="cuda")
    x[0, :, :64] = 1
    x[0, 2, -70:] = torch.arange(70, dtype=torch.uint8, device="cuda")
    p = torch.tensor([[2, 0, 2]], dtype=torch.int32, device="cuda")
    out = dvl.beam_reorder(p, [x])[0][0]
    for i, j in enumerate([2, 0, 2]):
        assert torch.equal(out[0, i], x[0, j])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout", ["tokens", "heads"])
@pytest.mark.parametrize("page,heads,D,length", [(16, 4, 128, 37), (16, 1, 64, 32), (1, 2, 16, 5), (7, 3, 80, 20),
                                                 (64, 8, 128, 63), (64, 2, 256, 0), (32, 8, 256, 31)])
def test_reorder_pages(dvl, page, heads, D, length, layout, fp8):
    batch, beams, k = 3, 4, 5
    rng = np.random.default_rng(page + length)
    width = length // page + 2
    pages = batch * (beams * width + k) + 1
    shape = (pages, page, heads, D) if layout == "tokens" else (pages, heads, page, D)
    if fp8:
        pool = [torch.from_numpy(rng.integers(0, 120, size=shape).astype(np.uint8)).cuda() for _ in range(2)]
    else:
        pool = [torch.randn(shape, device="cuda").bfloat16() for _ in range(2)]
    kv = pool if layout == "tokens" else [x.transpose(1, 2) for x in pool]
    cache = dvl.KVCache(*kv)
    ids = rng.permutation(pages)[:batch * (beams * width + k)].astype(np.int32)
    table = ids[:batch * beams * width].reshape(batch, beams, width)
    spare = ids[batch * beams * width:].reshape(batch, k)
    lengths = np.full((batch, beams), length, np.int32)
    if length:
        lengths[1] = rng.integers(0, length + 1, size=beams)
    p = choose(page, batch, beams, k)
    before = [x.contiguous().view(torch.uint8).cpu().numpy().copy().reshape(pages, page, heads, -1) for x in kv]
    _, t_out, l_out = dvl.beam_reorder(torch.from_numpy(p).cuda(), cache=cache, table=torch.from_numpy(table).cuda(),
                                       lengths=torch.from_numpy(lengths).cuda(), spare=torch.from_numpy(spare).cuda())
    want_t, want_l = moved(table, p), moved(lengths, p)
    want = [x.copy() for x in before]
    for b in range(batch):
        for i in range(k):
            if p[b, i] < 0:
                continue
            n = want_l[b, i]
            slot, rest = n // page, n % page
            if slot < width:
                src = want_t[b, i, slot]
                for x, y in zip(want, before):
                    x[spare[b, i], :rest] = y[src, :rest]
                want_t[b, i, slot] = spare[b, i]
    assert np.array_equal(t_out.cpu().numpy(), want_t)
    assert np.array_equal(l_out.cpu().numpy(), want_l)
    for x, w in zip(kv, want):
        assert np.array_equal(x.contiguous().view(torch.uint8).cpu().numpy().reshape(w.shape), w)


def test_reorder_full_table_and_foreign_pages_copy_nothing(dvl):
    pool = torch.randn(4, 4, 1, 16, device="cuda").bfloat16()
    cache = dvl.KVCache(pool, pool.clone())
    before = pool.clone()
    p = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
    table = torch.tensor([[[0], [1], [99]]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([[4, 2, 3]], dtype=torch.int32, device="cuda")   # full; page 1; a page outside the pool
    spare = torch.tensor([[2, 77, 3]], dtype=torch.int32, device="cuda")    # 77 is outside the pool
    _, t, n = dvl.beam_reorder(p, cache=cache, table=table, lengths=lengths, spare=spare)
    assert t.tolist() == [[[0], [77], [3]]] and n.tolist() == [[4, 2, 3]]
    assert torch.equal(pool, before)


def test_reorder_on_another_stream(dvl):
    x = torch.randn(16, 8, 50000, device="cuda")
    p = choose(1, 16, 8, 8)
    pd = torch.from_numpy(p).cuda()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = dvl.beam_reorder(pd, [x], stream=st)[0][0]
    st.synchronize()
    assert np.array_equal(out.cpu().numpy(), moved(x.cpu().numpy(), p))


def test_reorder_refusals(dvl):
    x = torch.zeros(2, 3, 8, device="cuda")
    p = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    cache = dvl.KVCache(torch.zeros(4, 4, 1, 16, dtype=torch.bfloat16, device="cuda"),
                        torch.zeros(4, 4, 1, 16, dtype=torch.bfloat16, device="cuda"))
    t = torch.zeros(2, 3, 2, dtype=torch.int32, device="cuda")
    n = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    ok = dict(cache=cache, table=t, lengths=n, spare=n)
    for bad in [dict(parents=p.long()), dict(parents=p.cpu()), dict(parents=p[0]), dict(states=[x.cpu()]),
                dict(states=[x.transpose(1, 2)]), dict(states=[x] * 9), dict(states=[]), dict(states=[x[:1]]),
                dict(states_out=[]), dict(states_out=[x.int()]), dict(table=t), dict(ok, spare=None),
                dict(ok, lengths=n.long()), dict(ok, table=t.cpu()), dict(ok, spare=n[:1]), dict(ok, table_out=t[:1])]:
        args = dict(parents=p, states=[x])
        args.update(bad)
        with pytest.raises(ValueError):
            dvl.beam_reorder(**args)
    with pytest.raises(dvl.DvlError):
        dvl.beam_reorder(p, [x], states_out=[x])  # over itself
    wide = torch.zeros(1, 33, 8, device="cuda")
    with pytest.raises(dvl.DvlError):
        dvl.beam_reorder(p[:1], [wide])
