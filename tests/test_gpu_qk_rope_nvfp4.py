"""The codes and scales that dvl_qk_norm_rope writes to an NVFP4 cache, bit for
bit: of values, and of keys that are neither normed nor rotated, the fp32 numbers
that are rounded are the inputs."""
import numpy as np
import pytest

import nvfp4_reference as N

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


def written(dvl, x, scale, rot=0, positions=None):
    """(codes, block scales) of keys and values x [rows][heads][D]."""
    rows, heads, D = x.shape
    pages = -(-rows // 16)
    pools = [torch.full((pages, 16, heads, n), 0xaa, dtype=torch.uint8, device="cuda") for n in (D // 2, D // 2, D // 16, D // 16)]
    cache = dvl.KVCache(*pools[:2], k_scale=scale, v_scale=scale, k_blocks=pools[2], v_blocks=pools[3])
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
    dvl.qk_norm_rope(torch.zeros_like(x[:, :1]), x, x, cache=cache, table=table,
                     lengths=torch.tensor([rows], dtype=torch.int32, device="cuda"),
                     rope=dvl.Rope(rot) if rot else None, positions=positions)
    return [p.reshape(pages * 16, heads, -1)[:rows].cpu().numpy() for p in pools]


def compare(dvl, x, scale, **kw):
    x = torch.from_numpy(np.ascontiguousarray(x)).bfloat16()
    codes, blocks = N.encode(x.float().numpy(), scale)
    k, v, kb, vb = written(dvl, x.cuda(), scale, **kw)
    for got, want in ((kb, blocks), (vb, blocks), (k, codes), (v, codes)):
        assert np.array_equal(got, want), np.mean(got != want)


@pytest.mark.parametrize("heads,D", [(2, 64), (3, 128), (1, 192), (2, 256)])
@pytest.mark.parametrize("scale", [1.0, 0.5, 0.002, 3.7, 2.0 ** -100, 2.0 ** 100])
def test_nvfp4_codes_are_the_definitions(dvl, heads, D, scale):
    rng = np.random.default_rng(D)
    compare(dvl, N.ties(rng, 200, heads, D, scale), scale)
    # blocks of every size, some with a scale of 0, some saturated
    size = 2.0 ** rng.integers(-14, 14, size=(200, heads, D // 16, 1))
    x = (rng.normal(size=(200, heads, D // 16, 16)) * size).reshape(200, heads, D)
    x[0] = 0
    x[1, :, 5] = -0.0
    compare(dvl, np.clip(x * scale, -3e38, 3e38), scale)


def test_nvfp4_codes_of_keys_turned_by_nothing(dvl):
    # at position 0 a rotation leaves the fp32 values as they are
    rng = np.random.default_rng(3)
    compare(dvl, N.ties(rng, 40, 2, 128, 1.0), 1.0, rot=64, positions=torch.zeros(40, dtype=torch.int32, device="cuda"))


def test_nvfp4_infinities_and_nan(dvl):
    x = np.ones((4, 1, 64), dtype=np.float32)
    x[0, 0, 3], x[1, 0, 20], x[2, 0, 40] = np.inf, -np.inf, np.nan
    k, v, kb, vb = written(dvl, torch.from_numpy(x).bfloat16().cuda(), 1.0)
    for codes, blocks in ((k, kb), (v, vb)):
        one = N.encode(x[3], 1.0)
        assert np.array_equal(codes[3], one[0]) and np.array_equal(blocks[3], one[1])
        # an infinity is the largest number, and its neighbours' quotients are 1 / 448
        assert blocks[0, 0].tolist() == [0x7e, *one[1][0, 1:]] and codes[0, 0, :8].tolist() == [0, 0x70, 0, 0, 0, 0, 0, 0]
        assert blocks[1, 0].tolist() == [one[1][0, 0], 0x7e, *one[1][0, 2:]] and codes[1, 0, 10] == 0x0f
        assert blocks[2, 0].tolist() == [*one[1][0, :2], 0x7f, one[1][0, 3]]
