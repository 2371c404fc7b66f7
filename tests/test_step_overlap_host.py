"""dvl_beam_reorder refuses outputs that share bytes with an input or with
another output (no GPU here: nothing is enqueued)."""
import random

import pytest

from test_step_host import L, cache  # noqa: F401  (L is a fixture)

# 2 requests of 3 beams, 3 new ones; widths of 4 table entries
ROWS, TABLE = 6, 6 * 4 * 4


def call(L, states, pages=None):  # noqa: F811
    from draft_vocab_lm_gb300._native import DvlBeamPages, DvlState
    a = dict(table=0x1000, table_out=0x2000, lengths=0x3000, lengths_out=0x4000, spare=0x5000, width=4, reserved=0)
    a.update(pages or {})
    array = (DvlState * len(states))(*[DvlState(*s) for s in states])
    p = DvlBeamPages(**a) if pages is not None else None
    return L.dvl_beam_reorder(array, len(states), p, cache() if p else None, 0x9000, 2, 3, 3, None)


def state(src, dst, row=64, src_stride=None, dst_stride=None):
    return src, dst, row, src_stride or row, dst_stride or row


@pytest.mark.parametrize("pages", [
    dict(table_out=0x1000),                                    # the table in place
    dict(lengths_out=0x3000),                                  # the lengths in place
    dict(table_out=0x1000, lengths_out=0x3000),
    dict(table_out=0x1000 + TABLE - 4), dict(table_out=0x1000 - TABLE + 4), dict(lengths_out=0x3000 + 20),
    dict(table_out=0x3000), dict(table_out=0x3000 - TABLE + 4),  # over the lengths
    dict(table_out=0x5000), dict(lengths_out=0x5000 + 20),     # over the spare pages
    dict(lengths_out=0x9000), dict(table_out=0x9000 - 4),      # over the parents
    dict(lengths_out=0x1000 + 40),                             # over the table
    dict(lengths_out=0x2000 + TABLE - 4),                      # two outputs
])
def test_tables_and_lengths(L, pages):  # noqa: F811
    assert call(L, [], pages) == 1


@pytest.mark.parametrize("states", [
    [state(0x10000, 0x10000)], [state(0x10000, 0x10000 + 64 * 5)], [state(0x10000 + 64 * 5, 0x10000)],
    [state(0x10000, 0x20000), state(0x20000, 0x10000)],        # swapped
    [state(0x10000, 0x20000), state(0x30000, 0x10000 + 100)],
    [state(0x10000, 0x20000), state(0x30000, 0x20000)],        # one output for two
    [state(0x10000, 0x20000), state(0x30000, 0x20000 + 64 * 6 - 1)],
    [state(0x10000, 0x9000 - 64 * 6 + 1)],                     # over the parents
    [state(0x10000, 0x10000 + 63, 64, 128, 128)],              # strided rows that share one byte
    [state(0x10000, 0x10000 + 100, 64, 256, 40 + 64)],         # strides that meet further on
    [state(0x10000, 0x10000 + 64 * 5 + 63, 1)] * 2,            # (the same output twice)
])
def test_states(L, states):  # noqa: F811
    assert call(L, states) == 1


def test_states_and_tables(L):  # noqa: F811
    assert call(L, [state(0x10000, 0x1000 + 32)], {}) == 1     # a state over the table
    assert call(L, [state(0x2000, 0x10000)], {}) == 1          # the new table over a state
    assert call(L, [state(0x10000, 0x2000)], {}) == 1          # a state and the new table


def test_strided_rows_that_share_a_byte(L):  # noqa: F811
    rng, seen = random.Random(1), 0
    while seen < 500:
        row = rng.randrange(1, 9)
        src, dst = ((0x10000 + rng.randrange(60), row + rng.randrange(12)) for _ in range(2))
        a, b = ({at + i * stride + j for i in range(ROWS) for j in range(row)} for at, stride in (src, dst))
        if a & b:
            seen += 1
            assert call(L, [state(src[0], dst[0], row, src[1], dst[1])]) == 1
