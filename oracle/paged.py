"""Oracle: the paged cache (block tables, pool rows, attention over all visible entries).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

The pages do not describe paging; the definitions are those of the C ABI's
header.  Plain loops over requests and entries; the attention gathers the
entries one request at a time and hands them to ``attention.sparse_mqa``.

Parity: pinned (tests/test_oracle_paged.py) by a hand-worked step, by the
invariants of a block table (no block in two requests, every entry's row
where the writer put it) and by the identity with the unpaged attention.
"""

import numpy as np

from . import attention


def block_tables(lens, n_new, free_blocks, table, block_size, max_new, free_pos=0):
    """One step's bookkeeping.  Returns (table, slots, start, len_out, info)
    as new arrays: see csa2_block_tables."""
    table = np.array(table, dtype=np.int64)
    B, max_blocks = table.shape
    slots = np.full(max_new, -1, dtype=np.int64)
    start = np.zeros(B + 1, dtype=np.int64)
    len_out = np.array(lens, dtype=np.int64)
    first, refused, exhausted = free_pos, 0, False
    at = 0
    for b in range(B):
        n, add = int(lens[b]), int(n_new[b])
        start[b] = min(at, max_new)
        fits = n >= 0 and add >= 0 and n + add <= max_blocks * block_size and at + add <= max_new
        need = -(-(n + add) // block_size) - -(-n // block_size) if fits else 0
        if need > 0 and (exhausted or free_pos < 0 or first + need > len(free_blocks)):
            fits, exhausted = False, True
        if fits:
            have = -(-n // block_size)
            for j in range(need):
                table[b, have + j] = free_blocks[first + j]
            first += need
            for i in range(add):
                blk = table[b, (n + i) // block_size]
                slots[at + i] = blk * block_size + (n + i) % block_size if blk >= 0 else -1
            len_out[b] = n + add
        else:
            refused += 1
        at += max(add, 0)
    start[B] = min(at, max_new)
    return table, slots, start, len_out, np.array([first, refused])


def paged_rows(positions, table, block_size, n_blocks, n_vis=None):
    """positions [B, Q, K] -> pool rows, -1 where there is none."""
    table = np.asarray(table)
    out = np.full(np.shape(positions), -1, dtype=np.int64)
    for b, q, k in np.ndindex(*np.shape(positions)):
        pos = int(positions[b, q, k])
        if pos < 0 or pos // block_size >= table.shape[1] or (n_vis is not None and pos >= n_vis[b, q]):
            continue
        blk = int(table[b, pos // block_size])
        if 0 <= blk < n_blocks:
            out[b, q, k] = blk * block_size + pos % block_size
    return out


def paged_mqa(q, rows_of, n_vis, window, scale=None):
    """One query: ``rows_of(j)`` the dequantised entry j (or None where the
    table names no block), window [W, 512].  Returns (o, lse)."""
    keys = [k for k in (rows_of(j) for j in range(max(0, int(n_vis)))) if k is not None]
    keys = np.array(keys, dtype=np.float64).reshape(-1, np.asarray(q).shape[1])
    return attention.sparse_mqa(q, keys, np.arange(len(keys)), window, scale)
