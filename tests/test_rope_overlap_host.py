"""What dvl_qk_norm_rope takes for an overlap of its outputs, against the bytes
themselves (no GPU here: the pointers are never dereferenced)."""
import concurrent.futures as cf
import ctypes

import numpy as np
import pytest

from test_cache_host import NO_DEVICE, cache, qk


@pytest.fixture(scope="module")
def L():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("no pointers to give a device")
    from draft_vocab_lm_gb300 import build
    build.build()
    from draft_vocab_lm_gb300 import _native
    return _native.lib()


@pytest.fixture(scope="module")
def status(L):
    """A call's status, on a thread of its own (the failure's description is the thread's)."""
    with cf.ThreadPoolExecutor(1) as one:
        yield lambda **kw: one.submit(lambda: L.dvl_qk_norm_rope(ctypes.byref(qk(**kw)), None)).result()


def interleaved(**kw):
    """[rows][heads][3][64]: every head's query, key and value side by side."""
    a = dict(cache=cache(), Hq=2, H=2, q=0x100000, k=0x100080, v=0x100100)
    for n in ("q", "k", "v", "q_out", "k_out"):
        a[n + "_stride"], a[n + "_head_stride"] = 384, 192
    a.update(kw)
    return a


def test_heads_of_one_projection_side_by_side(status):
    assert status(**interleaved(q_out=0x100000)) == NO_DEVICE
    assert status(**interleaved(q_out=0x100000, k_out=0x100080)) == NO_DEVICE
    assert status(**interleaved(q_out=0x140000, k_out=0x140080)) == NO_DEVICE
    assert status(**interleaved(q_out=0x140000, k_out=0x140100)) == NO_DEVICE
    assert status(**interleaved(q_out=0x100010)) == 1
    assert status(**interleaved(q_out=0x100080)) == 1  # over the keys
    assert status(**interleaved(q_out=0x100100, k_out=0x100080)) == 1  # over the values
    assert status(**interleaved(q_out=0x140000, k_out=0x140040)) == 1
    assert status(**interleaved(q_out=0x140000, k_out=0x140180)) == 1  # over the next head
    # a row on: only the rows that both have meet
    assert status(**interleaved(q_out=0x140000, k_out=0x140000 + 6 * 768)) == NO_DEVICE
    assert status(**interleaved(q_out=0x140000, k_out=0x140000 + 5 * 768)) == 1


def bytes_of(at, rows, stride, heads, head_stride, D):
    """The bytes of a tensor, as a set."""
    return {at + 2 * (r * stride + h * head_stride) + i for r in range(rows) for h in range(heads) for i in range(2 * D)}


def test_every_overlap_is_refused_and_with_one_stride_nothing_else(status):
    rng = np.random.default_rng(0)
    seen = [0, 0]
    for _ in range(1500):
        rows, Hq, H, D = (int(rng.integers(1, n)) for n in (4, 4, 4, 2)) if rng.random() < 0.5 else (3, 2, 2, 1)
        D = 16
        base = 0x200000
        hs = int(rng.choice([16, 24, 32, 48, 64]))
        rs = int(rng.choice([hs * max(Hq, H), hs * max(Hq, H) + 8, 16, 192]))
        if rng.random() < 0.3:
            rs, hs = hs, int(rng.choice([hs * rows, hs * rows + 16]))
        one = rng.random() < 0.7
        rs2, hs2 = (rs, hs) if one else (int(rng.choice([64, 96, 200])), int(rng.choice([16, 32, 48])))
        q_out, k_out = base + 4096, base + 4096 + 16 * int(rng.integers(-60, 60))
        kw = dict(rows=rows, Hq=Hq, H=H, D=D, rot=16, q=0x100000, k=0x110000, v=0x120000, q_out=q_out, q_out_stride=rs,
                  q_out_head_stride=hs, k_out=k_out, k_out_stride=rs2, k_out_head_stride=hs2, B=1,
                  cache=cache(heads=H, D=D))
        a, b = bytes_of(q_out, rows, rs, Hq, hs, D), bytes_of(k_out, rows, rs2, H, hs2, D)
        itself = len(a) < rows * Hq * 2 * D or len(b) < rows * H * 2 * D
        got = status(**kw)
        if itself or a & b:
            assert got == 1, kw
        elif one and got == 1:
            # refused only where heads and rows of one output lie between each other
            nested = [(n == 1 or rows == 1 or rs >= (n - 1) * hs + D or hs >= (rows - 1) * rs + D) for n in (Hq, H)]
            assert not all(nested), kw
        seen[got == 1] += 1
    assert min(seen) > 200


def test_rows_side_by_side_with_heads_of_different_strides(status):
    # rows of four query heads, then keys and values of two heads side by side
    # (k, v, k, v); a million of them are no more work to compare than a few
    kw = dict(cache=cache(), q=0x100000000, k=0x100000200, v=0x100000280, k_head_stride=128, v_head_stride=128)
    for n in ("q", "k", "v", "q_out", "k_out"):
        kw[n + "_stride"] = 512
    for rows in (6, 3 << 18):
        many = dict(kw, rows=rows)
        assert status(**many, q_out=0x100000000) == NO_DEVICE
        assert status(**many, q_out=0x900000000) == NO_DEVICE
        assert status(**many, q_out=0x100000000, k_out=0x100000200, k_out_head_stride=128) == NO_DEVICE
        assert status(**many, q_out=0x900000000, k_out=0x900000200, k_out_head_stride=128) == NO_DEVICE
        assert status(**many, q_out=0x900000000, k_out=0x9000001f0, k_out_head_stride=128) == 1
        assert status(**many, q_out=0x100000040) == 1
        assert status(**many, q_out=0x100000000, k_out=0x100000280, k_out_head_stride=128) == 1
