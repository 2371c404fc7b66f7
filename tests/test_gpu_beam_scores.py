"""Scores of dvl_beam_select against log_softmax in 64 bits, where adding the
row's maximum to the logarithm of its sum in one number would lose the latter.

Bound: x - m rounds once (u |x - m|), the logarithm's argument is off by at
most ~100 u (32 logits per thread, butterflies, the chunks) and 2^-21 for the
exponentials, the logarithm and the two last additions round once each."""
import math

import pytest

import step_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

INF = float("inf")
LOWEST = torch.finfo(torch.float32).min


@pytest.fixture(scope="module")
def dvl():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from draft_vocab_lm_gb300 import build
    build.build()
    import draft_vocab_lm_gb300 as d
    return d


def verify(x, scores, k, got):
    """x: the logits as the call saw them, on the CPU; the result's own candidates and the best ones."""
    exact = torch.log_softmax(x.double(), dim=2)
    off = x.double() - x.double().amax(2, keepdim=True)
    out, parents, tokens = (t.cpu() for t in got)
    total = scores.double().unsqueeze(2) + exact
    batch, beams, N = x.shape
    for b in range(batch):
        best = total[b].flatten().sort(descending=True).values
        for i in range(k):
            j, n = int(parents[b, i]), int(tokens[b, i])
            assert 0 <= j < beams and 0 <= n < N
            tol = R.U * (3 * abs(float(total[b, j, n])) + 2 * abs(float(scores[b, j])) + abs(float(off[b, j, n])) + 40)
            tol += 100 * R.U + 2.0 ** -20
            assert abs(float(out[b, i]) - float(total[b, j, n])) <= tol, (b, i, float(out[b, i]), float(total[b, j, n]))
            assert abs(float(total[b, j, n] - best[i])) <= 2 * tol


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("N", [100, 16000, 70001])
def test_beam_rows_of_lowest_values_are_uniform(dvl, N, bf16):
    # a mask that writes the type's lowest value over a whole row leaves a uniform distribution
    low = torch.finfo(torch.bfloat16).min if bf16 else LOWEST
    x = torch.full((2, 3, N), low)
    g = torch.Generator().manual_seed(N)
    x[1, 0] = torch.randn(N, generator=g)
    x[1, 1] = torch.randn(N, generator=g)
    x[1, 1, N // 2:] = low
    scores = torch.tensor([[0.0, -0.5, -1.0], [-1.0, -0.25, 0.0]])
    xd = x.bfloat16() if bf16 else x
    got = dvl.beam_select(xd.cuda(), scores.cuda(), 4)
    verify(xd.float(), scores, 4, got)
    assert abs(float(got[0][0, 0]) + math.log(N)) <= 1e-5
    # an all-masked beam has no advantage over the live ones: its k-th best is a uniform candidate
    assert float(got[0][1, 0]) < 0 and torch.all(got[1][1].cpu() != 2) or N == 100


@pytest.mark.parametrize("offset", [0.0, 1000.0, -1000.0, 1e5, -1e5, 1e30])
def test_beam_scores_do_not_depend_on_a_common_offset(dvl, offset):
    # logits on a grid that the offset leaves exact (below 2^17 + 2^3: multiples of 2^-6); 1e30 takes all in
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(2, 4, 9001, generator=g) * 2 * 64).round() / 64 + offset
    scores = -4 * torch.rand(2, 4, generator=g)
    verify(x, scores, 6, dvl.beam_select(x.cuda(), scores.cuda(), 6))


def test_beam_one_candidate_left_by_a_lowest_value_mask(dvl):
    # a forced token: its log-probability is 0, and the others' are far below anything
    x = torch.full((1, 2, 5000), LOWEST)
    x[0, 0, 4321] = -3.0
    x[0, 1, 17] = 7.5
    scores = torch.tensor([[-1.0, -2.0]])
    out, parents, tokens = dvl.beam_select(x.cuda(), scores.cuda(), 2)
    assert out.tolist() == [[-1.0, -2.0]] and parents.tolist() == [[0, 1]] and tokens.tolist() == [[4321, 17]]
