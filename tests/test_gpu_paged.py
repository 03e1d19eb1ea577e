"""GPU tests of the paged cache: block tables and pool rows (exact), the
attention over all visible entries (float64 oracle), and a run of them
together with the cache writer and the sparse attention.

Attention tolerance, element by element, from the roundings that the kernel
makes (A = sum_j w_j |k_jd|, the weighted mean of magnitudes):
* the output's bf16 rounding: 2^-8 |o|;
* each softmax weight is rounded to bf16 (2^-8 relative) before it multiplies
  its key, in the numerator and (at most) in the sum: 2 * 2^-8 A;
* logits: bf16 products are exact in float32, sums of 512 of them carry at
  most 512 * 2^-24 * scale * sum_d |q_d k_d|; a logit off by e changes a
  weight by a factor e, in numerator and sum: 2 e A, e the largest over the
  query's keys (plus 2^-20 for exp2's own error and the float32 sums).
The log-sum-exp: e, and 2^-8 where rounded weights enter the sum, plus
float32 rounding of its own value.
"""

import numpy as np
import pytest
import torch

from fp4_kv_cache_mxfp4_b200 import csa2
from oracle import attention, fp4, fp8, paged
from parity import check_attention, f32

pytestmark = pytest.mark.gpu
DEV = "cuda"


# ---------------------------------------------------------------------------
# block tables
# ---------------------------------------------------------------------------

def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class Step:
    """Device arrays of one csa2_block_tables call."""

    def __init__(self, lens, new, free, table, block, max_new, free_pos=None, in_place=False):
        B = len(lens)
        self.len, self.new, self.free = _i32(lens), _i32(new), _i32(free)
        self.table = _i32(table)
        self.slots = torch.full((max_new,), 77, dtype=torch.int64, device=DEV)
        self.start = torch.full((B + 1,), 77, dtype=torch.int32, device=DEV)
        self.len_out = self.len if in_place else torch.full((B,), 77, dtype=torch.int32, device=DEV)
        self.info = torch.full((2,), 77, dtype=torch.int32, device=DEV)
        self.pos = None
        if free_pos is not None:
            if in_place:
                self.info[0] = free_pos
                self.pos = self.info[:1]
            else:
                self.pos = _i32([free_pos])
        self.args = csa2.block_table_args(self.len, self.new, self.free, self.table, self.slots, self.start, self.len_out,
                                          self.info, block_size=block, free_pos=self.pos)
        self.ws = csa2.workspace(self.args, csa2.WS_BLOCK_TABLES)

    def run(self, stream=None):
        csa2.csa2_block_tables(self.args, self.ws, stream)

    def results(self):
        torch.cuda.synchronize()
        return [t.cpu().numpy() for t in (self.table, self.slots, self.start, self.len_out, self.info)]


def _compare(step, expected):
    for name, got, want in zip(("table", "slots", "start", "len_out", "info"), step.results(), expected):
        np.testing.assert_array_equal(got, want, err_msg=name)


def _case(rng, B, block, max_len, max_new_each, spare, width_extra=1):
    lens = rng.integers(0, max_len + 1, B)
    new = rng.integers(0, max_new_each + 1, B)
    have = -(-lens // block)
    width = int((-(-(lens + new) // block)).max(initial=0)) + width_extra
    table = np.full((B, width), -1)
    ids = rng.permutation(int(have.sum()) + 20)
    at = 0
    for b in range(B):
        table[b, : have[b]] = ids[at: at + have[b]]
        at += have[b]
    need = int((-(-(lens + new) // block) - have).sum())
    free = rng.permutation(need + 3) + len(ids)
    return lens, new, free, table, int(new.sum()) + spare


@pytest.mark.parametrize("B,block,max_len,max_new,spare", [
    (1, 64, 0, 1, 0), (1, 1, 5, 7, 2), (3, 16, 40, 1, 0), (33, 7, 100, 9, 5), (257, 64, 1000, 1, 0),
    (1025, 16, 300, 3, 11),               # more requests than scanning threads
    (20, 64, 3000, 1000, 100),            # more rows than one launch writes
    (2500, 3, 10, 8, 0),
    (5, 128, 700, 0, 17),                 # nothing new, padding only
])
@pytest.mark.parametrize("in_place", [False, True])
def test_block_tables(B, block, max_len, max_new, spare, in_place):
    rng = np.random.default_rng(B * 1000 + block)
    lens, new, free, table, n = _case(rng, B, block, max_len, max_new, spare)
    n = max(n, 1)
    s = Step(lens, new, free, table, block, n, free_pos=2, in_place=in_place)
    s.run()
    _compare(s, paged.block_tables(lens, new, free, table, block, n, 2))


@pytest.mark.parametrize("short", [1, 40, 10 ** 6])
@pytest.mark.parametrize("max_new", [3, 900, 30])
def test_block_tables_refuse_what_does_not_fit(short, max_new):
    """Too few blocks, too few rows, negative and overlong requests: those
    requests are refused, the others served, nothing else is touched."""
    rng = np.random.default_rng(short)
    lens, new, free, table, n = _case(rng, 300, 8, 50, max_new, 0, width_extra=0)
    lens[7], new[9], lens[11] = -5, -1, table.shape[1] * 8 - 1
    new[11] = 2
    free = free[: max(0, len(free) - short)]
    n = n * 3 // 4
    s = Step(lens, new, free, table, 8, n)
    s.run()
    want = paged.block_tables(lens, new, free, table, 8, n)
    assert want[4][1] > 3
    _compare(s, want)
    # a free position outside the list serves only requests that need no block
    for pos in (-1, len(free) + 5):
        s = Step(lens, new, free, table, 8, n, free_pos=pos)
        s.run()
        _compare(s, paged.block_tables(lens, new, free, table, 8, n, pos))


def test_block_tables_rows_apart_and_empty_lists():
    rng = np.random.default_rng(5)
    lens, new, free, table, n = _case(rng, 6, 4, 30, 5, 2)
    s = Step(lens, new, free, table, 4, n)
    wide = torch.full((6, table.shape[1] + 9), 55, dtype=torch.int32, device=DEV)
    s.table = wide[:, : table.shape[1]]
    s.table.copy_(_i32(table))
    s.args = csa2.block_table_args(s.len, s.new, s.free, s.table, s.slots, s.start, s.len_out, s.info, block_size=4)
    s.run()
    _compare(s, paged.block_tables(lens, new, free, table, 4, n))
    assert torch.all(wide[:, table.shape[1]:] == 55)
    # no free blocks and no rows at all
    s = Step([3, 4], [1, 1], np.zeros(0, int), [[0], [1]], 4, 1)
    s.run()
    _compare(s, paged.block_tables([3, 4], [1, 1], [], [[0], [1]], 4, 1))


def test_block_tables_captured_steps():
    """A captured step with lengths, position and table updated in place, replayed: the cache grows step by step."""
    rng = np.random.default_rng(8)
    B, block, steps = 9, 4, 7
    lens, new = rng.integers(0, 9, B), rng.integers(0, 3, B)
    table = np.full((B, 12), -1)
    ids = rng.permutation(200)
    at = 0
    for b in range(B):
        k = -(-lens[b] // block)
        table[b, :k] = ids[at: at + k]
        at += k
    free = ids[at:]
    s = Step(lens, new, free, table, block, 32, free_pos=0, in_place=True)
    keep = [t.clone() for t in (s.len, s.info, s.table)]
    s.run()                                              # not captured: sets the kernels up
    for t, k in zip((s.len, s.info, s.table), keep):
        t.copy_(k)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    pos, ln = 0, lens
    for _ in range(steps):
        g.replay()
        want = paged.block_tables(ln, new, free, table, block, 32, pos)
        _compare(s, want)
        table, ln, pos = want[0], want[3], want[4][0]


# ---------------------------------------------------------------------------
# rows of positions
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("B,Q,K,block,vis", [(1, 1, 1, 64, True), (3, 2, 5, 1, True), (4, 1, 512, 64, True),
                                             (2, 7, 513, 33, False), (1, 300, 37, 16, True)])
def test_paged_rows(B, Q, K, block, vis):
    rng = np.random.default_rng(K)
    width, n_blocks = 9, 70
    table = rng.integers(-2, n_blocks + 2, (B, width))            # some entries name no block
    pos = rng.integers(-3, width * block + block, (B, Q, K))
    n_vis = rng.integers(0, width * block + 5, (B, Q)) if vis else None
    wide = torch.zeros(B, width + 4, dtype=torch.int32, device=DEV)
    wide[:, :width] = _i32(table)
    pos_d, rows = _i32(pos), torch.full((B, Q, K), 99, dtype=torch.int32, device=DEV)
    vis_d = _i32(n_vis) if vis else None
    want = paged.paged_rows(pos, table, block, n_blocks, n_vis)
    csa2.csa2_paged_rows(pos_d, wide[:, :width], rows, block_size=block, n_blocks=n_blocks, n_vis=vis_d)
    np.testing.assert_array_equal(rows.cpu().numpy(), want)
    csa2.csa2_paged_rows(pos_d, wide[:, :width], pos_d, block_size=block, n_blocks=n_blocks, n_vis=vis_d)   # in place
    np.testing.assert_array_equal(pos_d.cpu().numpy(), want)


def test_paged_rows_past_32_bit_positions():
    """Positions near the table's last one, where position + block overflows 31 bits nowhere."""
    block, width = 1 << 14, 1 << 16                               # 2^30 positions
    table = torch.arange(width, dtype=torch.int32, device=DEV).flip(0)[None].contiguous()
    pos = _i32([[[0, (1 << 30) - 1, 1 << 30, 2 ** 31 - 1, 5 * block + 7]]])
    rows = torch.empty_like(pos)
    csa2.csa2_paged_rows(pos, table, rows, block_size=block, n_blocks=width)
    assert rows.flatten().tolist() == [(width - 1) * block, block - 1, -1, -1, (width - 6) * block + 7]


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

class Case:
    """A paged cache with shuffled blocks; rows that no visible entry lies in hold NaN scales or NaNs."""

    def __init__(self, lens, Q=1, block=64, W=128, kv="fp4", window="bf16", step=1, seed=0, q_std=1.0, scale=0.0, vis=None,
                 gap=0, missing=()):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.lens, self.Q, self.block, self.W, self.step, self.scale = list(lens), Q, block, W, step, scale
        B = len(self.lens)
        counts = [-(-n // block) for n in self.lens]
        width = max(1, max(counts))
        self.n_blocks = sum(counts) + 2
        ids = rng.permutation(self.n_blocks)
        self.table = np.full((B, width), -7)
        fp4_rows = kv == "fp4"
        row = 288 if fp4_rows else 512
        if fp4_rows:
            pool = np.full((self.n_blocks, block, 288), 0xFF, dtype=np.uint8)     # E4M3 0xFF: NaN scales
        else:
            pool = torch.full((self.n_blocks, block, 512), float("nan"), dtype=torch.bfloat16)
        self.keys, at = [], 0
        for b, n in enumerate(self.lens):
            self.table[b, : counts[b]] = ids[at: at + counts[b]]
            at += counts[b]
            x = torch.randn(n, 512, generator=g).to(torch.bfloat16)
            raw = fp4.quantize_kv_fp4(f32(x)) if fp4_rows else x
            self.keys.append(fp4.dequantize_kv_fp4(raw) if fp4_rows and n else f32(x).astype(np.float64))
            for j in range(counts[b]):
                part = raw[j * block: (j + 1) * block]
                pool[self.table[b, j], : len(part)] = part
        if gap:                                                                   # blocks that lie apart
            wide = torch.zeros(self.n_blocks, block + gap, row, dtype=torch.uint8 if fp4_rows else torch.bfloat16, device=DEV)
            wide[:, :block] = torch.as_tensor(pool).to(DEV)
            self.pool = wide[:, :block]
        else:
            self.pool = torch.as_tensor(pool).to(DEV)
        for b, j, what in missing:                                                # blocks that the table does not name
            self.table[b, j] = what
        self.q = (torch.randn(B, Q, 64, 512, generator=g) * q_std).to(torch.bfloat16)
        if vis is None:
            vis = [[max(0, n - Q + 1 + i) for i in range(Q)] for n in self.lens]
        self.vis = np.asarray(vis).reshape(B, Q)
        self.swa = self.swa_scale = None
        self.win = np.zeros((B, 0, 512))
        if W:
            rows = W + (Q - 1) * step
            x = torch.randn(B, rows, 512, generator=g).to(torch.bfloat16)
            if window == "bf16":
                self.swa, self.win = x.to(DEV), f32(x)
            else:
                codes, scales = zip(*(fp8.quantize_window_fp8(f32(x[b])) for b in range(B)))
                self.win = np.stack([fp8.dequantize_window_fp8(c, s) for c, s in zip(codes, scales)])
                self.swa = torch.from_numpy(np.stack(codes)).to(DEV)
                self.swa_scale = torch.from_numpy(np.stack(scales)).float().to(DEV)
        self.q_d, self.table_d, self.vis_d = self.q.to(DEV), _i32(self.table), _i32(self.vis)
        self.out = torch.full((B, Q, 64, 512), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((B, Q, 64), float("nan"), device=DEV)
        self.args = csa2.paged_attn_args(self.q_d, self.pool, self.table_d, self.vis_d, self.out, self.lse, swa=self.swa, W=W,
                                         swa_step=step, swa_scale=self.swa_scale, scale=scale)
        self.ws = csa2.workspace(self.args, csa2.WS_PAGED_ATTN)

    def run(self):
        csa2.csa2_paged_attn(self.args, self.ws)
        return self

    def _visible(self, b, i):
        n = min(max(0, int(self.vis[b, i])), self.table.shape[1] * self.block)
        k = np.array([self.keys[b][j] for j in range(n)
                      if 0 <= self.table[b, j // self.block] < self.n_blocks]).reshape(-1, 512)
        return np.concatenate([k, self.win[b][i * self.step: i * self.step + self.W]])

    def check(self, rows=None):
        torch.cuda.synchronize()
        assert csa2.csa2_device_status() == (0, 0)
        out, lse = self.out.float().cpu().numpy(), self.lse.cpu().numpy()
        scale = self.scale if self.scale > 0 else 512 ** -0.5
        B = len(self.lens)
        for b, i in (rows if rows is not None else np.ndindex(B, self.Q)):
            keys, q = self._visible(b, i), f32(self.q[b, i]).astype(np.float64)
            o, l = attention.sparse_mqa(q, keys, np.arange(len(keys)), np.zeros((0, 512)), scale)
            if not len(keys):
                assert np.all(out[b, i] == 0) and np.all(np.isneginf(lse[b, i]))
                continue
            w = np.exp(q @ keys.T * scale - l[:, None])
            A = w @ np.abs(keys)
            e = (512 * 2.0 ** -24 * scale * (np.abs(q) @ np.abs(keys).T)).max(1, keepdims=True) + 2.0 ** -20
            tol = 2.0 ** -8 * np.abs(o) + (2 * 2.0 ** -8 + 2 * e) * A
            err = np.abs(out[b, i] - o)
            assert np.all(err <= tol), f"query {b},{i}: {np.max(err / tol):.2f} of the tolerance"
            assert np.all(np.abs(lse[b, i] - l) <= e[:, 0] + 2.0 ** -8 + 2.0 ** -22 * np.abs(l)), f"lse of {b},{i}"
        return self


@pytest.mark.parametrize("kv", ["fp4", "bf16"])
@pytest.mark.parametrize("lens,Q,block,W,window,seed", [
    ([1], 1, 64, 0, "bf16", 1),                       # one key
    ([0], 1, 64, 0, "bf16", 2),                       # no key at all
    ([0, 5, 0], 1, 16, 3, "bf16", 3),                 # window only beside short rows
    ([128], 1, 128, 128, "bf16", 4),                  # exact tiles
    ([127, 129, 300], 1, 64, 128, "fp8", 5),          # pages that end inside a tile
    ([1, 2, 3, 4, 5, 6, 7, 1000], 1, 1, 1, "bf16", 6),    # one entry per block
    ([700, 33], 1, 7, 130, "fp8", 7),                 # odd blocks, the window over two tiles
    ([900], 5, 32, 128, "bf16", 8),                   # a verify block, causal
    ([2, 300], 5, 48, 100, "fp8", 9),                 # ... with rows that see nothing yet
    ([2500, 1, 1300], 1, 300, 128, "bf16", 10),       # blocks longer than a tile
    ([40] * 60, 1, 16, 20, "bf16", 11),               # many short rows
    ([500], 1, 64, 1024, "bf16", 12),                 # the widest window
])
def test_attention(lens, Q, block, W, window, seed, kv):
    Case(lens, Q, block, W, kv, window, seed=seed).run().check()


@pytest.mark.parametrize("kv", ["fp4", "bf16"])
def test_more_queries_than_ctas(kv):
    """Ranges that hold several whole queries, and cuts inside them."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 700, 170).tolist()
    c = Case(lens, 1, 64, 0, kv, seed=20).run()
    c.check([(b, 0) for b in range(0, 170, 3)] + [(169, 0)])


def test_one_long_query_over_every_cta():
    Case([20000], 1, 64, 128, seed=21).run().check()
    Case([18900, 1, 130], 1, 64, 0, "bf16", seed=22).run().check()


def test_peaked_softmax_moves_the_reference():
    """Logits spread over hundreds of log2 units: the running reference moves often, and partials differ widely."""
    Case([3000, 700], 1, 64, 128, seed=23, q_std=4.0, scale=0.2).run().check()
    Case([900], 1, 64, 128, "bf16", "fp8", seed=24, q_std=4.0, scale=0.2).run().check()
    # one CTA per query: growing maxima inside one accumulator
    Case([900] * 150, 1, 64, 0, seed=25, q_std=4.0, scale=0.2).run().check([(b, 0) for b in range(0, 150, 11)])


def test_visible_lengths_are_clipped_and_missing_blocks_hold_no_keys():
    c = Case([300, 200, 100], 1, 32, 16, seed=26, vis=[[-4], [10 ** 6], [64]], missing=[(1, 2, -1), (2, 0, 10 ** 6)])
    c.keys[1] = np.concatenate([c.keys[1], np.full((c.table.shape[1] * 32 - 200, 512), np.nan)])
    c.table[1, 7:] = -9                                 # the clipped length reaches entries without a block
    c.table_d.copy_(_i32(c.table))
    c.keys[1][200:] = np.nan                            # (entries 200..223 of the last block are stale: name no block either)
    c.table[1, 6] = -1
    c.table_d.copy_(_i32(c.table))
    c.run().check()
    # every block missing and no window: no key
    c = Case([64], 1, 32, 0, seed=27, missing=[(0, 0, -1), (0, 1, 9999)])
    c.run().check()


def test_blocks_and_table_rows_apart():
    c = Case([400, 77], 2, 16, 8, seed=28, gap=5)
    wide = torch.full((2, c.table.shape[1] + 3), 1 << 20, dtype=torch.int32, device=DEV)
    wide[:, : c.table.shape[1]] = c.table_d
    c.args = csa2.paged_attn_args(c.q_d, c.pool, wide[:, : c.table.shape[1]], c.vis_d, c.out, c.lse, swa=c.swa, W=8, swa_step=1)
    c.run().check()
    Case([400, 77], 1, 16, 8, "bf16", seed=29, gap=3).run().check()


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes, the request's blocks at its far end."""
    block, n_blocks = 1024, 16384                       # 4.8 GB of FP4 entries
    pool = torch.zeros(n_blocks, block, 288, dtype=torch.uint8, device=DEV)
    c = Case([3000], 1, block, 64, seed=30)
    far = [n_blocks - 1, n_blocks - 9, n_blocks - 4]
    pool[far] = c.pool[c.table_d[0].long()]
    table = _i32([far])
    c.args = csa2.paged_attn_args(c.q_d, pool, table, c.vis_d, c.out, c.lse, swa=c.swa, W=64, swa_step=1)
    c.run().check()


def test_without_lse_and_results_repeat():
    """lse is optional, and the same call gives the same bits again (partials join in a fixed order)."""
    c = Case([5000, 300, 1, 2222], 1, 64, 128, seed=31).run().check()
    first = c.out.clone()
    for _ in range(3):
        c.out.fill_(float("nan"))
        c.run()
        assert torch.equal(c.out, first)
    c.args = csa2.paged_attn_args(c.q_d, c.pool, c.table_d, c.vis_d, c.out, None, swa=c.swa, W=128, swa_step=1)
    c.out.zero_()
    c.run()
    assert torch.equal(c.out, first)


def test_other_stream_and_capture_with_growing_lengths():
    """Calls on a side stream, and a captured call replayed while n_vis grows."""
    c = Case([1500, 900], 1, 64, 32, seed=32)
    full = c.vis.copy()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run()
    torch.cuda.synchronize()
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for part in (0.0, 0.1, 0.7, 1.0):
        c.vis = (full * part).astype(int)
        c.vis_d.copy_(_i32(c.vis))
        c.out.fill_(float("nan"))
        g.replay()
        c.check()


def test_two_calls_at_once_on_two_streams():
    """Two workspaces, two streams: neither call disturbs the other."""
    a, b = Case([3000, 10], 1, 64, 128, seed=33), Case([2000] * 3, 1, 16, 0, "bf16", seed=34)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                c.run()
    torch.cuda.synchronize()
    a.check()
    b.check()


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def test_rows_without_a_place_are_not_written():
    """Negative destination rows skip an entry in all four cache writers."""
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, 512, generator=g).to(torch.bfloat16).to(DEV)
    rows = torch.tensor([4, -1, 0, -5, 7, -1], device=DEV)
    keep, dst = [0, 2, 4], [4, 0, 7]
    kv, kv2 = (torch.full((9, 288), 200, dtype=torch.uint8, device=DEV) for _ in range(2))
    csa2.csa2_quantize_kv_fp4(x, kv, dst_rows=rows)
    csa2.csa2_quantize_kv_fp4(x[keep], kv2, dst_rows=torch.tensor(dst, device=DEV))
    assert torch.equal(kv, kv2)
    c, c2 = (torch.full((9, 512), 200, dtype=torch.uint8, device=DEV) for _ in range(2))
    s, s2 = (torch.full((9,), 3.0, device=DEV) for _ in range(2))
    csa2.csa2_quantize_window_fp8(x, c, s, dst_rows=rows)
    csa2.csa2_quantize_window_fp8(x[keep], c2, s2, dst_rows=torch.tensor(dst, device=DEV))
    assert torch.equal(c, c2) and torch.equal(s, s2)
    k, k2 = (torch.full((9, 68), 200, dtype=torch.uint8, device=DEV) for _ in range(2))
    csa2.csa2_quantize_index_k_mxfp4(x[:, :128], k, dst_rows=rows)
    csa2.csa2_quantize_index_k_mxfp4(x[keep][:, :128], k2, dst_rows=torch.tensor(dst, device=DEV))
    assert torch.equal(k, k2)
    cos, sin, w = torch.ones(6, 32, device=DEV), torch.zeros(6, 32, device=DEV), torch.ones(1, 1, 512, device=DEV)
    kv.fill_(200)
    csa2.csa2_compress_rope_quantize_kv_fp4(x, 1, w, cos, sin, kv, dst_rows=rows)
    assert torch.equal(kv, kv2)


def test_a_served_batch_step_by_step():
    """Requests grow from nothing: block tables make rows, the writer fills
    the pool through them, the indexer selects on its own dense keys,
    paged_rows turns its positions into pool rows for csa2_sparse_attn, and
    while a context is no longer than K the sparse and the paged attention
    agree (both see every entry), up to the roundings of both."""
    g = torch.Generator().manual_seed(2)
    B, block, K, W, N = 5, 16, 512, 32, 1024
    n_blocks = 220
    rng = np.random.default_rng(2)
    pool = torch.full((n_blocks, block, 288), 0xFF, dtype=torch.uint8, device=DEV)
    lens = np.zeros(B, int)
    step = Step(lens, [1] * B, rng.permutation(n_blocks), np.full((B, N // block), -1), block, 1500, free_pos=0, in_place=True)
    mirror = [np.zeros((0, 288), np.uint8) for _ in range(B)]
    kI = torch.randn(B, N, 128, generator=g).to(torch.bfloat16).to(DEV)
    for new in ([300, 1, 512, 0, 40], [1, 1, 0, 1, 1], [5, 600, 0, 16, 200]):
        x = torch.randn(1500, 512, generator=g).to(torch.bfloat16)
        step.new.copy_(_i32(new))
        step.run()
        csa2.csa2_quantize_kv_fp4(x.to(DEV), pool.view(-1, 288), dst_rows=step.slots)      # the padded batch, whole
        start = np.concatenate([[0], np.cumsum(new)])
        for b in range(B):
            mirror[b] = np.concatenate([mirror[b], fp4.quantize_kv_fp4(f32(x[start[b]: start[b + 1]])).reshape(-1, 288)])
        lens = lens + np.array(new)
        torch.cuda.synchronize()
        assert step.info.tolist()[1] == 0 and step.len.tolist() == lens.tolist()
        table = step.table.cpu().numpy()
        flat = pool.view(-1, 288).cpu().numpy()
        for b in range(B):
            rows = [table[b, j // block] * block + j % block for j in range(lens[b])]
            np.testing.assert_array_equal(flat[rows], mirror[b])
        # selection on the requests' positions
        vis = step.len.view(B, 1)
        qI = torch.randn(B, 1, 32, 128, generator=g).to(torch.bfloat16).to(DEV)
        w = torch.rand(B, 1, 32, generator=g).to(DEV)
        idx = torch.empty(B, 1, K, dtype=torch.int32, device=DEV)
        ia = csa2.index_args(csa2.FULL, qI, w, kI, vis.contiguous(), idx)
        csa2.csa2_index_score_topk(ia, csa2.workspace(ia, csa2.WS_INDEX))
        rows = torch.empty_like(idx)
        csa2.csa2_paged_rows(idx, step.table, rows, block_size=block, n_blocks=n_blocks, n_vis=vis.contiguous())
        np.testing.assert_array_equal(rows.cpu().numpy(),
                                      paged.paged_rows(idx.cpu().numpy(), table, block, n_blocks, lens[:, None]))
        # sparse attention over the pool: one row of B queries, their windows W rows apart
        q = torch.randn(B, 1, 64, 512, generator=g).to(torch.bfloat16).to(DEV)
        swa = torch.randn(B, W, 512, generator=g).to(torch.bfloat16).to(DEV)
        so = torch.empty(1, B, 64, 512, dtype=torch.bfloat16, device=DEV)
        sa = csa2.attn_args(q.view(1, B, 64, 512), pool.view(1, -1, 288), rows.view(1, B, K), swa.view(1, B * W, 512), so, W=W,
                            swa_step=W)
        csa2.csa2_sparse_attn(sa, csa2.workspace(sa, csa2.WS_ATTN))
        po = torch.empty(B, 1, 64, 512, dtype=torch.bfloat16, device=DEV)
        pa = csa2.paged_attn_args(q, pool, step.table, vis.contiguous(), po, swa=swa, W=W)
        csa2.csa2_paged_attn(pa, csa2.workspace(pa, csa2.WS_PAGED_ATTN))
        torch.cuda.synchronize()
        assert csa2.csa2_device_status() == (0, 0)
        sel = idx.cpu().numpy()
        for b in range(B):
            deq = fp4.dequantize_kv_fp4(mirror[b]) if lens[b] else np.zeros((0, 512))
            qb, wb = f32(q[b, 0].cpu()), f32(swa[b].cpu())
            o, _ = attention.sparse_mqa(qb, deq, np.arange(lens[b]), wb)
            check_attention(po[b, 0], o, what=f"paged {b}")
            o, _ = attention.sparse_mqa(qb, deq, sel[b, 0], wb)
            check_attention(so[0, b], o, what=f"sparse over the pool {b}")
            if lens[b] <= K:
                # both results against one value: twice the bar's share that their roundings take
                np.testing.assert_allclose(po[b, 0].float().cpu().numpy(), so[0, b].float().cpu().numpy(), atol=2e-2, rtol=2e-2)


@pytest.mark.parametrize("B,extra", [(1024, 0), (1024, 1), (5000, 3)])
def test_block_tables_one_row_each(B, extra):
    """The longest list of one launch, the shortest of two, and more requests than starts held in shared memory."""
    rng = np.random.default_rng(B + extra)
    lens, _, free, table, _ = _case(rng, B, 16, 60, 1, 0)
    new = np.ones(B, dtype=np.int64)
    free = np.concatenate([free, np.arange(B) + 10 ** 6])
    s = Step(lens, new, free, table, 16, B + extra)
    s.run()
    _compare(s, paged.block_tables(lens, new, free, table, 16, B + extra))


@pytest.mark.parametrize("block,width", [(1 << 30, 1), (1 << 29, 2), ((1 << 29) - 3, 2), (1, 8), (1000003, 1073)])
def test_block_tables_at_the_largest_tables(block, width):
    """Divisions by the block size up to the last position that a table can name."""
    cap = block * width
    lens = np.array([cap - 4, cap - 1, 0, block - 1 if block > 1 else 3, cap - 2, cap])
    new = np.array([4, 2, 3, 3, 2, 0])
    table = np.full((6, width), -1)
    rng = np.random.default_rng(width)
    for b in range(6):
        have = -(-int(lens[b]) // block)
        table[b, :have] = rng.integers(0, 1000, have)
    s = Step(lens, new, np.arange(50) + 2000, table, block, 20)
    s.run()
    _compare(s, paged.block_tables(lens, new, np.arange(50) + 2000, table, block, 20))


@pytest.mark.parametrize("B", [2, 3, 10, 11, 40])
def test_partials_joined_for_few_and_many_queries(B):
    """Every way that the join splits its work, with queries of no key and of one tile between long ones."""
    rng = np.random.default_rng(B)
    lens = rng.integers(1500, 6000 if B < 12 else 2500, B)
    lens[1::4] = rng.integers(0, 2, lens[1::4].size) * 100
    c = Case(lens.tolist(), 1, 64, 0 if B % 2 else 40, seed=B + 50).run()
    c.check([(b, 0) for b in range(0, B, max(1, B // 8))] + [(1, 0), (B - 1, 0)])


def test_blocks_shared_by_several_requests():
    """A common prefix: the same blocks in several rows of the table."""
    c = Case([600, 600, 600, 90], 1, 64, 40, seed=61)
    for b in (1, 2):
        c.table[b, :7], c.keys[b] = c.table[0, :7], np.concatenate([c.keys[0][:7 * 64], c.keys[b][7 * 64:]])
    c.table_d.copy_(_i32(c.table))
    c.run().check()
