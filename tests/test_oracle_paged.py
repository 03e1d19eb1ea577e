"""Pins of the paged-cache oracle: a hand-worked step, the invariants of a
block table, and the identity with the unpaged attention."""

import numpy as np
import pytest

from oracle import attention, paged


def test_hand_worked_step():
    # blocks of 4; request 0 holds 3 entries in block 9 and gets 3: one fits, then block 20
    # request 1 is empty and gets none; request 2 holds 4 (block 7 full) and gets 5: blocks 21, 22
    table = [[9, -1, -1], [-1, -1, -1], [7, -1, -1]]
    t, slots, start, ln, info = paged.block_tables([3, 0, 4], [3, 0, 5], [5, 20, 21, 22, 30], table, 4, 10, free_pos=1)
    np.testing.assert_array_equal(t, [[9, 20, -1], [-1, -1, -1], [7, 21, 22]])
    np.testing.assert_array_equal(slots, [39, 80, 81, 84, 85, 86, 87, 88, -1, -1])
    np.testing.assert_array_equal(start, [0, 3, 3, 8])
    np.testing.assert_array_equal(ln, [6, 0, 9])
    np.testing.assert_array_equal(info, [4, 0])


def test_refusals():
    table = np.full((5, 2), -1)
    # 0: too long for its table row; 1: negative; 2: takes the last block; 3: none left; 4: fits in its own block
    table[4, 0] = 8
    t, slots, start, ln, info = paged.block_tables([7, -1, 0, 0, 2], [2, 1, 4, 1, 1], [3], table, 4, 9)
    np.testing.assert_array_equal(start, [0, 2, 3, 7, 8, 9])
    np.testing.assert_array_equal(slots, [-1, -1, -1, 12, 13, 14, 15, -1, 34])
    np.testing.assert_array_equal(ln, [7, -1, 4, 0, 3])
    np.testing.assert_array_equal(info, [1, 4 - 1])
    # rows beyond the list are refused whole
    t, slots, start, ln, info = paged.block_tables([0, 0], [2, 2], [0, 1], np.full((2, 1), -1), 4, 3)
    np.testing.assert_array_equal(slots, [0, 1, -1])
    np.testing.assert_array_equal(start, [0, 2, 3])
    np.testing.assert_array_equal(ln, [2, 0])
    np.testing.assert_array_equal(info, [1, 1])


@pytest.mark.parametrize("block", [1, 3, 16])
def test_steps_keep_a_table_consistent(block):
    """Random steps: no block belongs to two requests, every entry's row is
    the one its writer got, and paged_rows finds it."""
    rng = np.random.default_rng(block)
    B, width = 5, 40
    table, ln, pos = np.full((B, width), -1), np.zeros(B, int), 0
    free = rng.permutation(200)
    where = {}
    for _ in range(8):
        new = rng.integers(0, 5, B)
        table, slots, start, out, info = paged.block_tables(ln, new, free, table, block, 32, pos)
        for b in range(B):
            for i in range(out[b] - ln[b]):
                where[b, ln[b] + i] = slots[start[b] + i]
        ln, pos = out, info[0]
    used = table[table >= 0]
    assert len(set(used.tolist())) == len(used) and len(set(where.values())) == len(where)
    positions = np.array([[[j for j in range(ln.max() + 2)]] for _ in range(B)])
    rows = paged.paged_rows(positions, table, block, 200, ln[:, None])
    for b in range(B):
        assert rows[b, 0].tolist() == [where.get((b, j), -1) for j in range(ln.max() + 2)]


def test_attention_is_the_unpaged_one():
    rng = np.random.default_rng(0)
    q, keys, win = rng.normal(size=(64, 512)), rng.normal(size=(10, 512)), rng.normal(size=(3, 512))
    o, lse = paged.paged_mqa(q, lambda j: keys[j], 7, win)
    o2, lse2 = attention.sparse_mqa(q, keys, np.arange(7), win)
    np.testing.assert_array_equal(o, o2)
    np.testing.assert_array_equal(lse, lse2)
    o, lse = paged.paged_mqa(q, lambda j: None if j == 2 else keys[j], 4, win[:0])
    o2, lse2 = attention.sparse_mqa(q, keys, np.array([0, 1, -1, 3]), win[:0])
    np.testing.assert_array_equal(o, o2)
    o, lse = paged.paged_mqa(q, lambda j: keys[j], -3, win[:0])
    assert np.all(o == 0) and np.all(np.isneginf(lse))
