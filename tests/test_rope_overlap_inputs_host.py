"""dvl_qk_norm_rope refuses outputs over any of its inputs and over the cache's
pages (no GPU here: the pointers are never dereferenced)."""
import pytest

from test_cache_host import NO_DEVICE, cache, nvfp4
from test_rope_overlap_host import L, interleaved, status  # noqa: F401

# six rows of four query heads and two key heads of 64: q_out is 0x130000 ..
# 0x130c00, k_out (where it is given) 0x150000 .. 0x150600
INPUTS = [("q_weight", 128), ("k_weight", 128), ("freq", 256), ("positions", 24), ("table", 48), ("lengths", 12),
          ("starts", 16)]


@pytest.mark.parametrize("name,size", INPUTS)
def test_outputs_over_an_input(status, name, size):
    kw = dict(cache=cache(), k_out=0x150000)
    unit = 16 if name.endswith("weight") else 8
    for at in (0x130000, 0x130400, 0x130c00 - 16, 0x150000, 0x150600 - 16, 0x130000 - size + unit // 2 * 2 if unit == 8 else 0x130000 - size + 16):
        assert status(**kw, **{name: at}) == 1, hex(at)
    for at in (0x130c00, 0x150600, 0x130000 - size - size % 16, 0x150000 - size - size % 16):
        assert status(**kw, **{name: at}) == NO_DEVICE, hex(at)


def test_table_rows_and_weights_between_an_outputs_rows(status):
    # q_out's rows lie 1,024 bytes apart and take 512: the second halves are free
    apart = dict(cache=cache(), q_out_stride=512)
    for name in ("table", "lengths", "starts", "positions", "freq", "q_weight"):
        assert status(**apart, **{name: 0x130200}) == NO_DEVICE
        assert status(**apart, **{name: 0x130400}) == 1
        assert status(**apart, **{name: 0x130000 + 5 * 1024}) == 1
        assert status(**apart, **{name: 0x130000 + 5 * 1024 + 512}) == NO_DEVICE
    # three rows of a table, 1,024 bytes apart, in them, and one that reaches a row
    assert status(**apart, table=0x130200, table_stride=256) == NO_DEVICE
    assert status(**apart, table=0x130200, table_stride=192) == 1
    assert status(**apart, table=0x130200 - 4096, table_stride=1024) == NO_DEVICE
    assert status(**apart, table=0x130000 - 2048, table_stride=256) == 1
    # weights between the heads of a row
    assert status(**interleaved(q_out=0x140000, q_weight=0x140080)) == NO_DEVICE
    assert status(**interleaved(q_out=0x140000, q_weight=0x140040)) == 1


def test_outputs_in_the_caches_pages(status):
    # 8 pages of 4,096 bytes (bf16), 1,024 bytes of codes and 128 of scales (NVFP4)
    far = dict(k=0x200000, v=0x300000)
    for c in (cache(**far), nvfp4(**far, k_blocks=0x400000, v_blocks=0x500000)):
        ends = [(0x200000, 8 * (4096 if c.dtype == 0 else 1024)), (0x300000, 8 * (4096 if c.dtype == 0 else 1024))]
        ends += [] if c.dtype == 0 else [(0x400000, 1024), (0x500000, 1024)]
        for at, size in ends:
            for first in (at - 0xc00 + 16, at, at + size - 16):
                assert status(cache=c, q_out=first) == 1, hex(first)
            for first in (at - 0x600 + 16, at, at + size - 16):
                assert status(cache=c, k_out=first) == 1, hex(first)
            for first in (at - 0xc00, at + size):
                assert status(cache=c, q_out=first) == NO_DEVICE, hex(first)
    # between pages that lie apart
    gaps = dict(k_page_stride=8192, v_page_stride=8192)
    assert status(cache=cache(**far, **gaps), q_out=0x201000) == NO_DEVICE
    assert status(cache=cache(**far, **gaps), q_out=0x201000 + 7 * 0x4000) == NO_DEVICE
    assert status(cache=cache(**far, **gaps), q_out=0x201410) == NO_DEVICE
    assert status(cache=cache(**far, **gaps), q_out=0x203410) == 1  # reaches the next page


def test_no_rows_meet_nothing(status):
    assert status(cache=cache(), rows=0, q_weight=0x130000, k_out=0x1000) == 0
