"""Rope's frequencies, 64-bit fractions of a turn, against arithmetic in 400
decimal digits (host only)."""
import decimal
import math

import pytest

torch = pytest.importorskip("torch")

DIGITS = 400


def pi():
    """By the Gauss-Legendre iteration."""
    D = decimal.Decimal
    a, b, t, p = D(1), 1 / D(2).sqrt(), D("0.25"), D(1)
    for _ in range(10):
        c = (a + b) / 2
        b, t, p, a = (a * b).sqrt(), t - p * (a - c) ** 2, 2 * p, c
    return (a + b) ** 2 / (4 * t)


@pytest.fixture(scope="module")
def turns_of():
    """freq in radians -> its exact fraction of a turn in units of 2^-64 (a Decimal in [0, 2^64))."""
    with decimal.localcontext() as c:
        c.prec = DIGITS + 40
        two_pi = 2 * pi()
        assert str(two_pi / 2).startswith("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706")

    def exact(f):
        with decimal.localcontext() as c:
            c.prec = DIGITS
            t = decimal.Decimal(f) / two_pi
            return (t - t.to_integral_value(decimal.ROUND_FLOOR)) * 2 ** 64
    return exact


def off(got, want):
    """Distance of two fractions, around the turn."""
    d = abs(decimal.Decimal(got % 2 ** 64) - want)
    return min(d, 2 ** 64 - d)


@pytest.mark.parametrize("theta", [1e2, 1e4, 5e5, 1e6, 1e8])
@pytest.mark.parametrize("dim", [16, 64, 128, 256])
def test_turns_of_a_models_frequencies(turns_of, dim, theta):
    from draft_vocab_lm_gb300 import Rope
    freq = Rope(dim, theta=theta, device="cpu").freq
    assert freq.dtype == torch.int64 and freq.shape == (dim // 2,)
    for i, t in enumerate(freq.tolist()):
        assert off(t, turns_of(theta ** (-2 * i / dim))) <= 1


def test_turns_of_any_frequencies(turns_of):
    from draft_vocab_lm_gb300 import Rope
    freqs = [0.0, 1.0, -1.0, math.pi, -2 * math.pi, 3.0, 1e5, -7.25e10, 2.0 ** 70, -1e30, 1e100, 1.7e308, 5e-324, -1e-18,
             0.5, -0.125, 2.0 ** 63, 123456789.0, 1 / 3, 1e-6, 2.0 ** -64, 6.0, 6.5, -6.283185307179586, 1e16, 3e-5]
    freqs += [0.1 * i for i in range(32 - len(freqs))]
    for f, t in zip(freqs, Rope(64, freqs=freqs, device="cpu").freq.tolist()):
        assert off(t, turns_of(f)) <= 1, f


def test_a_far_positions_angle(turns_of):
    # what the kernel makes of it: 2^31 positions on, within 2^-32 of a turn
    from draft_vocab_lm_gb300 import Rope
    for i, t in enumerate(Rope(128, theta=1e6, device="cpu").freq.tolist()):
        f = 1e6 ** (-2 * i / 128)
        for position in (2 ** 31 - 1, -2 ** 31, 14_000_001):
            with decimal.localcontext() as c:
                c.prec = DIGITS
                want = turns_of(f) * position % 2 ** 64
            assert off(position * t, want % 2 ** 64) <= 2 ** 32


def test_turns_are_those_of_the_double(turns_of):
    # the mistake these tests have to tell: the quotient rounded to 53 bits
    far = 0
    for i in range(64):
        f = 1e6 ** (-2 * i / 128)
        far = max(far, off(round(math.ldexp(math.fmod(f / (2 * math.pi), 1.0), 64)), turns_of(f)))
    assert far > 100
