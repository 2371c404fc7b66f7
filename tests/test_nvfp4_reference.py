"""The NVFP4 reference against known codes and the requantizer's oracle, and the
mistakes it has to tell."""
import numpy as np

import nvfp4_reference as N
import synthetic as S
from cache_reference import E4M3

F = np.float32


def test_middles_go_to_the_even_code():
    y = np.zeros((1, 16), dtype=F)
    y[0, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]
    codes, s = N.encode(y, 1.0)
    assert s[0, 0] == 0x38
    assert codes[0, :4].tolist() == [0x07, 0x22, 0x44, 0x66]
    codes, s = N.encode(-y, 0.5)
    assert s[0, 0] == 0x40 and codes[0, :4].tolist() == [0x8f, 0xaa, 0xcc, 0xee]
    # block scales round to even, too, saturate, and one of 0 makes the codes 0
    y = np.zeros((4, 16), dtype=F)
    y[:, 3] = [6 * 1.0625, 6 * 1.1875, 6 * 500, 6 * 2.0 ** -11]
    codes, s = N.encode(y, 1.0)
    assert s[:, 0].tolist() == [0x38, 0x3a, 0x7e, 0] and not codes[3].any()


def test_a_reciprocal_in_place_of_the_division_is_told():
    rng = np.random.default_rng(0)
    y = N.ties(rng, 50, 2, 64, 1.0).astype(F)
    codes, s = N.encode(y, 1.0)
    unit = E4M3[s].astype(F)[..., None]
    z = y.reshape(*s.shape, 16) * (F(1) / unit)
    c = (N.nearest_even(np.abs(z), N._E2M1) + 8 * np.signbit(z)).reshape(*s.shape[:-1], -1, 2).astype(np.uint8)
    assert np.mean((c[..., 0] | c[..., 1] << 4) != codes) > 0.01


def test_the_same_codes_as_a_requantized_head(oracle_mod):
    # with the tensor's own scale the recipe is the load-time requantizer's
    rng = np.random.default_rng(1)
    bits = S.f32_to_bf16_bits(rng.normal(size=(7, 64)).astype(F))
    codes, scales, g = oracle_mod.quantize_nvfp4(bits)
    mine, s = N.encode((bits.astype(np.uint32) << 16).view(F), g)
    assert np.array_equal(mine, codes) and np.array_equal(s, scales)
