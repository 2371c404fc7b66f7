"""dvl_beam_select against the 64-bit form: scores within the summation bound,
the chosen candidates exactly where the scores are further apart than it, and
exact order on inputs made of ties."""
import numpy as np
import pytest

import step_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INF = float("inf")


@pytest.fixture(scope="module")
def dvl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from draft_vocab_lm_gb300 import build
    build.build()
    import draft_vocab_lm_gb300 as d
    return d


def verify(logits, scores, k, got, d2t=None):
    """logits, scores: host values as the call saw them."""
    out, parents, tokens = (t.cpu().numpy() for t in got)
    exact = R.beam_scores(logits, scores)
    tol = R.beam_tolerance(logits, scores)
    batch, beams, N = exact.shape
    back = None if d2t is None else {int(t): n for n, t in enumerate(d2t)}
    for b in range(batch):
        flat = exact[b].reshape(-1)
        order = np.argsort(-flat, kind="stable")
        live = int((flat > -np.inf).sum())
        seen = set()
        for i in range(k):
            if i >= live:
                assert (out[b, i], parents[b, i], tokens[b, i]) == (-np.inf, -1, -1)
                continue
            n = int(tokens[b, i]) if back is None else back[int(tokens[b, i])]
            at = int(parents[b, i]) * N + n
            assert 0 <= parents[b, i] < beams and 0 <= n < N and at not in seen
            seen.add(at)
            assert abs(out[b, i] - flat[at]) <= tol
            want = flat[order[i]]
            assert abs(flat[at] - want) <= 2 * tol, (b, i, flat[at], want)
            near = np.abs(flat[order[max(0, i - 1):i + 2]] - want)
            if np.count_nonzero(near <= 2 * tol) == 1:
                assert at == order[i]
            assert i == 0 or out[b, i] <= out[b, i - 1]


def make(seed, batch, beams, N, std=2.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(batch, beams, N, generator=g) * std
    scores = -5 * torch.rand(batch, beams, generator=g)
    return logits, scores


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("batch,beams,N,k", [
    (1, 1, 1, 1), (1, 1, 3, 8), (2, 3, 100, 6), (1, 4, 16000, 4), (3, 2, 2047, 5), (2, 2, 2048, 32),
    (1, 5, 2049, 10), (2, 8, 8193, 16), (1, 32, 4001, 32), (4, 4, 70001, 8), (1, 2, 248320, 4), (1, 31, 257, 32),
])
def test_beam_shapes(dvl, batch, beams, N, k, bf16):
    logits, scores = make(N + k, batch, beams, N)
    x = logits.bfloat16() if bf16 else logits
    got = dvl.beam_select(x.cuda(), scores.cuda(), k)
    verify(x.float().numpy(), scores.numpy(), k, got)


def test_beam_long_rows_and_a_reused_workspace(dvl):
    ws = dvl.beam_workspace(8, 8, 248320)
    d2t = torch.randperm(300000, generator=torch.Generator().manual_seed(0))[:248320].int()
    for seed, (batch, beams, k) in enumerate([(8, 8, 16), (2, 8, 8), (8, 8, 32)]):
        logits, scores = make(seed, batch, beams, 248320)
        verify(logits.numpy(), scores.numpy(), k,
               dvl.beam_select(logits.cuda(), scores.cuda(), k, d2t=d2t.cuda(), ws=ws), d2t.numpy())


@pytest.mark.parametrize("bf16", [False, True])
def test_beam_ties_go_to_the_lower_beam_then_row(dvl, bf16):
    # equal rows have equal lse, so every candidate of a logit value ties
    N, beams, k = 20011, 5, 32
    base = torch.zeros(N)
    base[torch.tensor([7, 8192, 8191, 15000, 20010, 40])] = 1.0
    logits = base.expand(2, beams, N).contiguous()
    scores = torch.zeros(2, beams)
    scores[1, 0] = -1.0  # the first beam of the second request is a step behind
    x = (logits.bfloat16() if bf16 else logits).cuda()
    _, parents, tokens = dvl.beam_select(x, scores.cuda(), k)
    top = sorted([7, 40, 8191, 8192, 15000, 20010])
    low = [n for n in range(100) if n not in top]
    want = [(j, n) for j in range(beams) for n in top] + [(0, n) for n in low[:2]]
    assert list(zip(parents[0].tolist(), tokens[0].tolist())) == want
    # exactly one natural unit behind: its best tie with nothing above the rest
    want = [(j, n) for j in range(1, beams) for n in top]
    assert list(zip(parents[1].tolist(), tokens[1].tolist()))[:24] == want


def test_beam_all_equal_logits(dvl):
    # the most keys that can reach the threshold
    for N, k in [(8192, 32), (30000, 32), (5, 8)]:
        x = torch.full((1, 3, N), 2.5, device="cuda")
        out, parents, tokens = dvl.beam_select(x, torch.zeros(1, 3, device="cuda"), k)
        flat = [(j, n) for j in range(3) for n in range(N)][:k]
        assert list(zip(parents[0].tolist(), tokens[0].tolist())) == flat
        assert np.allclose(out.cpu().numpy(), -np.log(N), atol=1e-5)


@pytest.mark.parametrize("bf16", [False, True])
def test_beam_rows_that_overflow_the_buffer(dvl, bf16):
    # rising logits pass every bound set so far; falling ones none
    N = 70000
    up = torch.linspace(-20, 20, N)
    saw = torch.arange(N).remainder(9000).float() / 300
    logits = torch.stack([up, up.flip(0), saw, torch.full((N,), torch.finfo(torch.float32).min)])[None]
    logits[0, 3, 69990:] = torch.arange(10).float()  # ten rows that a mask of the lowest value leaves
    scores = torch.tensor([[0.0, -0.5, 3.0, 1.0]])
    x = logits.bfloat16() if bf16 else logits
    for k in (4, 32):
        verify(x.float().numpy(), scores.numpy(), k, dvl.beam_select(x.cuda(), scores.cuda(), k))
    # each row by itself: every place of the selection is its own
    for j in range(4):
        verify(x[:, j:j + 1].float().numpy(), scores[:, j:j + 1].numpy(), 32,
               dvl.beam_select(x[:, j:j + 1].cuda(), scores[:, j:j + 1].contiguous().cuda(), 32))


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("k", [4, 32])
def test_beam_long_segments(dvl, k, bf16):
    # so many rows that each is one segment of several chunks: every way a
    # segment's room can fill, and ties at every bound
    N, beams, batch = 40001, 4, 152
    g = torch.Generator().manual_seed(k)
    pool = torch.randn(beams, N, generator=g)
    logits = pool[None].repeat(batch, 1, 1)
    logits[0] = torch.linspace(-20, 20, N)                                    # rising: everything passes
    logits[1] = torch.arange(N).remainder(9000).float() / 300                 # a saw
    logits[2] = 2.5                                                           # all equal
    logits[3] = -INF
    logits[3, :, 20000:25000] = torch.randn(beams, 5000, generator=g)         # an island of candidates
    logits[4] = torch.finfo(torch.float32).min
    logits[4, 1, 39990:] = torch.arange(11).float()                           # eleven rows left by a mask
    logits[5] = (torch.arange(N) % 97 == 5).float()                           # two values only
    logits[6, :, :16384] = pool[:, :16384] - 30                               # the first chunks say nothing
    logits[7, :, 4096:4160] = 9.0                                             # a plateau past the first bound
    scores = -5 * torch.rand(batch, beams, generator=g)
    scores[2], scores[5] = 0.0, 0.0
    x = logits.bfloat16() if bf16 else logits
    got = dvl.beam_select(x.cuda(), scores.cuda(), k)
    for b in list(range(9)) + [batch - 1]:
        verify(x[b:b + 1].float().numpy(), scores[b:b + 1].numpy(), k, tuple(t[b:b + 1] for t in got))
    assert list(zip(got[1][2].tolist(), got[2][2].tolist())) == [(0, n) for n in range(k)]
    assert list(zip(got[1][5].tolist(), got[2][5].tolist())) == [(0, 97 * i + 5) for i in range(k)]


def test_beam_masked_dead_and_non_finite(dvl):
    logits, scores = make(3, 6, 4, 5000)
    scores[0, 1:] = -INF            # the first step: one live beam
    scores[1] = -INF                # a finished request
    logits[2, 1] = -INF             # a beam with everything banned
    logits[2, 0, 3:] = -INF         # three tokens left
    logits[2, 2:] = -INF
    logits[3, 2, 77] = float("nan")
    logits[4, 0, 9] = INF
    scores[5, 3] = float("nan")
    logits[5, :, ::2] = -INF        # half the vocabulary banned
    got = dvl.beam_select(logits.cuda(), scores.cuda(), 8)
    x = logits.numpy().copy()
    verify(x, scores.numpy(), 8, got)
    parents = got[1].cpu().numpy()
    assert (parents[1] == -1).all() and (parents[2, :3] == 0).all() and (parents[2, 3:] == -1).all()
    assert 2 not in parents[3] and 0 not in parents[4] and 3 not in parents[5]


@pytest.mark.parametrize("shift", [0, 1, 3, 7])
@pytest.mark.parametrize("bf16", [False, True])
def test_beam_strides_and_alignment(dvl, bf16, shift):
    batch, beams, N = 3, 4, 9001
    logits, scores = make(shift, batch, beams, N)
    dt = torch.bfloat16 if bf16 else torch.float32
    # neighbours of a row hold values that would win
    buf = torch.full((batch, beams + 1, N + 11), 50.0, dtype=dt, device="cuda")
    view = buf[:, :beams, shift:shift + N]
    view.copy_(logits)
    got = dvl.beam_select(view, scores.cuda(), 8)
    verify(view.float().cpu().numpy(), scores.numpy(), 8, got)
    # all beams of a request share one row of logits
    shared = view[:, :1].expand(batch, beams, N)
    verify(shared.float().cpu().numpy(), scores.numpy(), 8, dvl.beam_select(shared, scores.cuda(), 8))


def test_beam_large_offsets(dvl):
    # the last request starts past 2^32 bytes
    N = 120_000
    buf = torch.empty(9300 * N, dtype=torch.float32, device="cuda")
    x = buf.as_strided((2, 2, N), (9297 * N, N, 1))
    logits, scores = make(1, 2, 2, N)
    x.copy_(logits)
    verify(logits.numpy(), scores.numpy(), 4, dvl.beam_select(x, scores.cuda(), 4))


def test_beam_on_another_stream_and_repeatable(dvl):
    logits, scores = make(9, 4, 8, 60000)
    a, b = logits.cuda(), scores.cuda()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    ws = dvl.beam_workspace(4, 8, 60000, stream=st)
    one = [t.clone() for t in dvl.beam_select(a, b, 16, ws=ws, stream=st)]
    st.synchronize()
    for _ in range(5):
        for p, q in zip(one, dvl.beam_select(a, b, 16)):
            assert torch.equal(p, q)


def test_beam_refusals(dvl):
    x = torch.zeros(2, 3, 64, device="cuda")
    s = torch.zeros(2, 3, device="cuda")
    for bad in [dict(logits=x.cpu()), dict(logits=x.half()), dict(logits=x[0]), dict(logits=x.transpose(1, 2)),
                dict(scores=s[:1]), dict(scores=s.double()), dict(scores=s.cpu()),
                dict(d2t=torch.zeros(63, dtype=torch.int32, device="cuda")),
                dict(d2t=torch.zeros(64, dtype=torch.int64, device="cuda")),
                dict(parents=torch.zeros(2, 4, dtype=torch.int32, device="cuda")),
                dict(ws=torch.zeros(1 << 20, dtype=torch.uint8))]:
        with pytest.raises(ValueError):
            args = dict(logits=x, scores=s, k=3)
            args.update(bad)
            dvl.beam_select(**args)
    for k in (0, 33, -1):
        with pytest.raises(ValueError):
            dvl.beam_select(x, s, k)
    with pytest.raises(dvl.DvlError) as e:
        dvl.beam_select(x, s, 3, ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    with pytest.raises(ValueError):
        dvl.beam_workspace(1, 33, 100)
    assert dvl.beam_select(x[:0], s[:0], 3, ws=dvl.beam_workspace(1, 3, 64))[0].shape == (0, 3)
