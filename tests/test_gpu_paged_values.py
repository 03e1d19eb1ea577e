"""GPU tests of the paged attention on the values at its borders: absent keys
beside rows that are not finite.  Cases and tolerances as in test_gpu_paged."""

import math

import numpy as np
import pytest
import torch

from fp4_kv_cache_mxfp4_b200 import csa2
from oracle import attention, fp4
from parity import check_attention, f32
from test_gpu_paged import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("kv", ["fp4", "bf16"])
def test_absent_window_keys_have_no_scale(kv, bad):
    """The last window tile of a query holds 2 keys; the 126 places behind
    them must not see the scales that an earlier tile left there, here of
    other requests whose scales are not finite."""
    c = Case([0] * 300, 1, 16, 130, kv, "fp8", seed=70)
    c.swa_scale[::2] = bad
    c.run().check([(b, 0) for b in range(1, 300, 2)])


@pytest.mark.parametrize("kv", ["fp4", "bf16"])
@pytest.mark.parametrize("W,window", [(0, "bf16"), (5, "fp8")])
def test_many_query_parts_per_cta(kv, W, window):
    """Some fourteen queries of one or two tiles per CTA: Q changes as often as the keys do."""
    lens = [(37 * b) % 190 for b in range(2100)]
    c = Case(lens, 1, 32, W, kv, window, seed=73)
    for _ in range(20):
        c.run()
    c.check([(b, 0) for b in range(0, 2100, 41)])


def test_query_parts_that_take_seconds():
    """148 requests of 2^27 entries, all in one block, each before an empty
    request: every CTA works for some 3.5 seconds on one query (2^20 tiles)
    before the next one's Q can be loaded.  Keys of ones and Q of zeros: all
    weights are 1, and the float32 sums of 2^20 of them exact."""
    B, block, per_row = 296, 1 << 17, 1 << 10
    pool = torch.full((1, block, 288), 0x22, dtype=torch.uint8, device="cuda")          # E2M1 1.0 twice
    pool[..., 256:] = 0x38                                                             # E4M3 1.0
    table = torch.zeros(B, per_row, dtype=torch.int32, device="cuda")
    vis = torch.zeros(B, 1, dtype=torch.int32, device="cuda")
    vis[::2] = block * per_row
    q = torch.zeros(B, 1, 64, 512, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, float("nan")), torch.full((B, 1, 64), float("nan"), device="cuda")
    args = csa2.paged_attn_args(q, pool, table, vis, out, lse)
    csa2.csa2_paged_attn(args, csa2.workspace(args, csa2.WS_PAGED_ATTN))
    torch.cuda.synchronize()
    assert csa2.csa2_device_status() == (0, 0)
    assert torch.all(out[::2] == 1) and torch.all(out[1::2] == 0)
    # float32: log2 and a product, half a unit in the last place each, log2 with one more
    assert torch.all((lse[::2] - 27 * math.log(2)).abs() <= 2.0 ** -22 * 27 * math.log(2)) and torch.all(lse[1::2] == -math.inf)


@pytest.mark.parametrize("B", [148, 100])                # whole queries in one CTA, and cut ones
@pytest.mark.parametrize("kv", ["fp4", "bf16"])
def test_output_sums_of_millions_of_keys(kv, B):
    """2^22 equal keys per request, all weights 1: the output is the key
    itself, to the bit.  A run's sum of 2^15 keys of 8 bits needs 23, the
    128 or more runs are added in float32, 2^-24 each: a relative 2^-16 against
    half a step of bf16, 2^-9 at least.  (One float32 accumulator
    over all of them keeps 24 bits of the 30 and loses a percent or more.)"""
    block, per_row = 4096, 1024
    if kv == "fp4":
        pool = torch.empty(1, block, 288, dtype=torch.uint8)
        codes = [1 + (c % 7) + 8 * (c % 2) for c in range(512)]
        pool[..., :256] = torch.tensor([codes[2 * i] | codes[2 * i + 1] << 4 for i in range(256)])
        pool[..., 256:] = torch.tensor([0x38 + (i % 8) for i in range(32)])            # 1 + m / 8
        key = torch.from_numpy(fp4.dequantize_kv_fp4(pool[0, :1].numpy())[0]).float()
    else:
        key = (1 + (torch.arange(512) % 128) / 128) * (1 - 2 * (torch.arange(512) % 2))
        pool = key.to(torch.bfloat16).expand(1, block, 512).contiguous()
    table = torch.zeros(B, per_row, dtype=torch.int32, device="cuda")
    vis = torch.full((B, 1), block * per_row, dtype=torch.int32, device="cuda")
    q = torch.zeros(B, 1, 64, 512, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    args = csa2.paged_attn_args(q, pool.cuda(), table, vis, out)
    csa2.csa2_paged_attn(args, csa2.workspace(args, csa2.WS_PAGED_ATTN))
    torch.cuda.synchronize()
    assert csa2.csa2_device_status() == (0, 0)
    assert torch.equal(out.float().cpu(), key.expand(B, 1, 64, 512))


@pytest.mark.parametrize("kv,q_std,scale,sizes", [
    ("fp4", 1.0, 0.0, (1, 1, 1, 1, 1, 1)), ("fp4", 1.0, 0.0, (0.2, 1, 0.5, 2, 0.1, 1.5)),
    ("bf16", 1.0, 0.0, (1, 0.3, 1.2, 0.6, 1, 1)), ("fp4", 4.0, 0.2, (0.5, 0.8, 1, 0.7, 0.9, 1)),
])
def test_runs_of_a_long_part_are_merged(kv, q_std, scale, sizes):
    """Some 475 tiles per CTA, more than one run, whole and cut queries, with
    maxima that grow and fall along the cache.  The pool has six blocks that
    stand in the table again and again: the definition over each entry once,
    with the number of its appearances as a factor of its weight."""
    P, B = 512, 20
    g, rng = torch.Generator().manual_seed(74), np.random.default_rng(74)
    x = (torch.randn(6, P, 512, generator=g) * torch.tensor(sizes)[:, None, None]).to(torch.bfloat16)
    if kv == "fp4":
        raw = fp4.quantize_kv_fp4(f32(x).reshape(-1, 512))
        pool, keys = torch.from_numpy(raw).view(6, P, 288), fp4.dequantize_kv_fp4(raw)
    else:
        pool, keys = x, f32(x).reshape(-1, 512).astype(np.float64)
    width = 1100
    table = np.repeat(rng.integers(0, 6, (B, width // 50)), 50, axis=1)                # the same block 50 times
    n = rng.integers(300_000, P * width, B)
    q = (torch.randn(B, 1, 64, 512, generator=g) * q_std).to(torch.bfloat16)
    out, lse = torch.empty_like(q, device="cuda"), torch.empty(B, 1, 64, device="cuda")
    args = csa2.paged_attn_args(q.cuda(), pool.cuda(), torch.tensor(table, dtype=torch.int32, device="cuda"),
                                torch.tensor(n, dtype=torch.int32, device="cuda")[:, None], out, lse, scale=scale)
    csa2.csa2_paged_attn(args, csa2.workspace(args, csa2.WS_PAGED_ATTN))
    torch.cuda.synchronize()
    assert csa2.csa2_device_status() == (0, 0)
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    scale = scale or 512 ** -0.5
    for b in range(B):
        times = np.repeat(np.bincount(table[b, : n[b] // P], minlength=6), P).astype(np.float64)
        if n[b] % P:
            at = table[b, n[b] // P] * P
            times[at: at + n[b] % P] += 1
        qb = f32(q[b, 0]).astype(np.float64)
        z = np.where(times > 0, qb @ keys.T * scale, -np.inf)
        m = z.max(1, keepdims=True)
        w = times * np.exp(z - m)
        l = w.sum(1, keepdims=True)
        w /= l
        o, A = w @ keys, w @ np.abs(keys)
        e = (512 * 2.0 ** -24 * scale * (np.abs(qb) @ np.abs(keys).T)).max(1, keepdims=True) + 2.0 ** -20
        # bf16 of the output and of the weights, logits (as in test_gpu_paged), and a run's sum, 2^-25 per key of 2^15
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2 * e + 2.0 ** -10) * A
        err = np.abs(out[b, 0] - o)
        assert np.all(err <= tol), f"request {b}: {np.max(err / tol):.2f} of the tolerance"
        # the sum: a thread adds up to 256 tiles' weights, 2^-24 each
        want = (m + np.log(l))[:, 0]
        assert np.all(np.abs(lse[b, 0] - want) <= e[:, 0] + 2.0 ** -16 + 2.0 ** -22 * np.abs(want)), f"lse of {b}"


@pytest.mark.parametrize("kv", ["fp4", "bf16"])
@pytest.mark.parametrize("lens", [[300, 5, 0, 1000], [300] * 160])       # cut, and whole in one CTA
def test_a_head_that_is_not_a_number(kv, lens):
    """A NaN in a query's head gives NaN there, in the log-sum-exp too (-inf
    says that there was no key), and leaves every other head as it was."""
    c = Case(lens, 1, 64, 0, kv, seed=75).run()
    out, lse = c.out.clone(), c.lse.clone()
    at = [(0, 3), (1, 63), (2 if len(lens) == 4 else 7, 16)]
    for b, h in at:
        c.q_d[b, 0, h, 9 * b] = float("nan")
    c.run()
    torch.cuda.synchronize()
    for b, h in at:
        if lens[b]:
            assert torch.all(torch.isnan(c.out[b, 0, h])) and torch.isnan(c.lse[b, 0, h]), (b, h)
        else:
            assert torch.all(c.out[b, 0, h] == 0) and torch.isneginf(c.lse[b, 0, h])
        c.out[b, 0, h], c.lse[b, 0, h] = out[b, 0, h], lse[b, 0, h]
    assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("lens,far", [([600], 256), ([600], 700), ([520] * 150, 256)])
def test_logits_below_the_range_of_float32(lens, far):
    """Finite entries whose logits are -2^195: -inf in float32, weight 0, also
    where they fill a query's first tiles and no reference exists yet.
    Expected: the definition over the other keys."""
    c = Case(lens, 1, 64, 16, "bf16", seed=76)
    c.pool[:, :, 0] = 0
    c.swa[:, :, 0] = 0
    c.win[..., 0] = 0
    c.q[..., 0] = 0
    c.q_d[..., 0] = 2.0 ** 100
    for b, n in enumerate(lens):
        rows = [(int(c.table[b, j // 64]), j % 64) for j in range(min(far, n))]
        c.pool[[r[0] for r in rows], [r[1] for r in rows], 0] = -2.0 ** 100
        c.keys[b] = c.keys[b][far:]
        c.keys[b][:, 0] = 0
    c.run()
    c.vis = np.maximum(c.vis - far, 0)
    c.check([(b, 0) for b in range(0, len(lens), 13)])


# ---------------------------------------------------------------------------
# every key, the log-sum-exp's own precision, prompts, the largest batch
# ---------------------------------------------------------------------------

def _one_dim_each(n):
    """n rows with one value each: consecutive rows share a dim, the first of them in dim 0."""
    x = torch.zeros(n, 512)
    j = torch.arange(n)
    x[j, j * 512 // n] = 1.0 + 0.5 * (j % 5)
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("kv", ["fp4", "bf16"])
@pytest.mark.parametrize("lens,block,W,window", [
    ([20000], 64, 0, "bf16"), ([4000, 1, 600, 9000], 7, 0, "bf16"), ([128 * 9] * 200, 128, 0, "bf16"),
    ([0, 700], 32, 1024, "bf16"), ([700, 0], 32, 1000, "fp8"),
])
def test_every_key_counts(lens, block, W, window, kv):
    """A dim of the output is the weight of at most 40 keys: one of them lost,
    or read as its neighbour tile's, changes it by more than the tolerance, 3 * 2^-8 of it."""
    c = Case(lens, 1, block, W, kv, window, seed=80)
    for b, n in enumerate(lens):
        if not n:
            continue
        x = _one_dim_each(n)
        raw = torch.from_numpy(fp4.quantize_kv_fp4(f32(x))) if kv == "fp4" else x
        c.keys[b] = fp4.dequantize_kv_fp4(raw.numpy()) if kv == "fp4" else f32(x).astype(np.float64)
        j = np.arange(n)
        c.pool[c.table[b, j // block], j % block] = raw.cuda()
    if W:
        x = _one_dim_each(W)
        c.win[:] = f32(x)
        if window == "fp8":
            s = x.float().abs().amax(1) / 256               # 256 times the row: exact codes and scales
            c.swa[:] = (x.float() / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
            c.swa_scale[:] = s.cuda()
        else:
            c.swa[:] = x.cuda()
    c.run().check([(b, 0) for b in range(0, len(lens), max(1, len(lens) // 8))] + [(len(lens) - 1, 0)])


@pytest.mark.parametrize("kv", ["fp4", "bf16"])
@pytest.mark.parametrize("W,window", [(0, "bf16"), (7, "bf16"), (5, "fp8")])
def test_log_sum_exp_keeps_float32(kv, W, window):
    """Queries with 8 channels, so that logits are nearly exact and the sum
    itself is tested: 8 products, each added with at most one unit of
    float32's last place lost, 2^-23; the logit's and the exponential's own
    roundings; float32 sums over a thread's tiles, the lanes and the
    parts (fewer than 64 steps beside the tiles).  Weights rounded to bf16
    would be off by up to 2^-9."""
    lens = [1, 2, 3, 5, 17, 130, 700, 3000]
    c = Case(lens, 1, 16, W, kv, window, seed=81, q_std=3.0, scale=0.5)
    c.q[..., 8:] = 0
    c.q_d.copy_(c.q)
    c.run().check()
    for b in range(len(lens)):
        keys, q = c._visible(b, 0), f32(c.q[b, 0]).astype(np.float64)
        z = q @ keys.T * 0.5
        m = z.max(1)
        want = m + np.log(np.exp(z - m[:, None]).sum(1))
        e = 8 * 2.0 ** -23 * 0.5 * (np.abs(q) @ np.abs(keys).T).max(1) + 2.0 ** -22 * np.abs(z).max(1)
        tol = e + (len(keys) / 128 + 64) * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -22 * np.abs(want)
        err = np.abs(c.lse[b, 0].cpu().numpy() - want)
        assert np.all(err <= tol), f"request {b}: {np.max(err / tol):.2f} of the tolerance"


@pytest.mark.parametrize("kv", ["fp4", "bf16"])
@pytest.mark.parametrize("n,Q,W", [(700, 300, 16), (260, 260, 0), (1500, 130, 128)])
def test_a_prompt(n, Q, W, kv):
    """Many query positions of one request, causal, the first ones with few keys."""
    c = Case([n], Q, 32, W, kv, seed=82).run()
    c.check([(0, i) for i in range(0, Q, 7)] + [(0, Q - 1)])


def test_the_largest_batch():
    """65,535 queries: 4.3 GB of Q and of results."""
    B, P = 65535, 64
    g = torch.Generator().manual_seed(83)
    x = torch.randn(P, 512, generator=g).to(torch.bfloat16)
    raw = fp4.quantize_kv_fp4(f32(x))
    keys = fp4.dequantize_kv_fp4(raw)
    base = torch.randn(3, 64, 512, generator=g).to(torch.bfloat16)
    which = torch.arange(B, device="cuda") % 3
    q = base.cuda()[which].view(B, 1, 64, 512)
    vis = (torch.arange(B, dtype=torch.int32, device="cuda") % 61)[:, None].contiguous()
    out, lse = torch.full_like(q, float("nan")), torch.full((B, 1, 64), float("nan"), device="cuda")
    args = csa2.paged_attn_args(q, torch.from_numpy(raw).cuda().view(1, P, 288),
                                torch.zeros(B, 1, dtype=torch.int32, device="cuda"), vis, out, lse)
    csa2.csa2_paged_attn(args, csa2.workspace(args, csa2.WS_PAGED_ATTN))
    torch.cuda.synchronize()
    assert csa2.csa2_device_status() == (0, 0)
    for b in list(range(0, B, 1009)) + [B - 1]:
        n = b % 61
        o, l = attention.sparse_mqa(f32(base[b % 3]), keys, np.arange(n), np.zeros((0, 512)))
        check_attention(out[b, 0], o, what=f"query {b}")
        # 512 products in float32, 512 * 2^-24 * scale * sum |q k|, below 1e-3 for these inputs
        assert np.allclose(lse[b, 0].cpu().numpy(), l, rtol=0, atol=1e-3)
    # equal inputs, equal bits: every query against the one 183 places before it, cut ones (one per CTA at most) apart
    same = (out[183:].view(B - 183, -1) == out[:-183].view(B - 183, -1)).all(1)
    assert int((~same).sum()) <= 2 * 148
