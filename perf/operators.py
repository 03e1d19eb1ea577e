"""The paged-cache operators as measured: their cases, inputs, plain forms and exact values.

A serving program keeps the FP4 main KV of all its requests in one pool of
blocks.  Three operators work on it:

block_tables  a step's request lengths -> blocks taken from the free list,
              block tables extended, a pool row for every new entry
paged_rows    positions that the top-K selected -> pool rows, which the sparse
              attention reads
paged_attn    attention of each request's new query positions over all its
              visible entries in the pool (FP4 or bf16 rows) and its layer's
              window, one softmax

`own` false: elementary torch operations in 32 bits.  `own` true: the calls of
the framework's binding.
"""

import math
import random

import torch

own = False

H, D = 64, 512             # query heads and head width: the framework's
ENTRY = 288                # bytes of an FP4 entry: 256 of nibbles, 32 E4M3 scales
DEV = "cuda"


# ----------------------------------------------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------------------------------------------

def _bt(B, block, lo, hi, new_lo, new_hi, spare, lens):
    return {"op": "block_tables", "B": B, "block": block, "lo": lo, "hi": hi, "new_lo": new_lo, "new_hi": new_hi,
            "spare": spare, "lens": lens}


def _pr(B, Q, K, block, lo, hi, lens):
    return {"op": "paged_rows", "B": B, "Q": Q, "K": K, "block": block, "lo": lo, "hi": hi, "lens": lens}


def _pa(B, Q, block, lo, hi, W, kv, window, lens):
    return {"op": "paged_attn", "B": B, "Q": Q, "block": block, "lo": lo, "hi": hi, "W": W, "kv": kv, "window": window,
            "lens": lens}


def listed():
    out = []

    def add(name, c):
        out.append({"name": name, **c})

    # a decode step of a few long requests: one new entry each, often no new block
    add("tables_decode_b4", _bt(4, 64, 100000, 131000, 1, 1, 0, 1))
    # a decode step of a busy server, one new entry per request
    add("tables_decode_b1024", _bt(1024, 64, 1, 32768, 1, 1, 0, 2))
    # a mixed step: prefill chunks of up to 4096 entries beside decode rows, in a padded batch
    add("tables_prefill_b512", _bt(512, 16, 0, 16384, 0, 4096, 1000, 3))
    # the top-512 of four decode queries at 128K entries
    add("rows_decode_b4_k512", _pr(4, 1, 512, 64, 131072, 131072, 4))
    # the top-512 of a prefill chunk's 4096 queries
    add("rows_prefill_q4096_k512", _pr(1, 4096, 512, 64, 133120, 133120, 5))
    # a fresh conversation: fewer entries than the top-K selects, so every layer attends to all of them
    add("attn_b1_short", _pa(1, 1, 64, 300, 300, 128, "fp4", "bf16", 6))
    # the decode shape of the 4-layer group workload: four requests at 128K
    add("attn_b4_128k", _pa(4, 1, 64, 131072, 131072, 128, "fp4", "bf16", 7))
    # many requests of very different lengths, small blocks, the FP8 window
    add("attn_b64_ragged", _pa(64, 1, 16, 1, 16384, 128, "fp4", "fp8", 8))
    # a full server of short requests
    add("attn_b256_short", _pa(256, 1, 64, 16, 2048, 128, "fp4", "bf16", 9))
    # one request of a million entries: the split over the cache's length
    add("attn_b1_1m", _pa(1, 1, 64, 1048576, 1048576, 128, "fp4", "bf16", 10))
    # the five query positions of a verify block
    add("attn_verify_b4_q5", _pa(4, 5, 64, 4000, 8192, 128, "fp4", "bf16", 11))
    # a pool of unquantised entries, no window
    add("attn_bf16_b8_32k", _pa(8, 1, 64, 20000, 32768, 0, "bf16", "bf16", 12))
    return out


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["block_tables", "paged_rows", "paged_attn", "paged_attn", "paged_attn"])
    lens = rng.randrange(1 << 30)
    block = rng.choice([16, 32, 64, 128, 256, rng.randrange(1, 300)])
    if op == "block_tables":
        hi = _log(rng, 2, 131072)
        new_hi = rng.choice([1, _log(rng, 1, 4096)])
        B = max(1, min(_log(rng, 1, 4096), (2 << 20) // new_hi, (128 << 20) // (hi + new_hi)))
        if block < 16:
            B = max(1, B // 16)
        return _bt(B, block, rng.choice([0, hi // 2]), hi, rng.choice([0, 1]), new_hi, rng.choice([0, 0, rng.randrange(5000)]),
                   lens)
    if op == "paged_rows":
        n = _log(rng, 1, 4096)
        Q = rng.choice([1, 5, n])
        hi = _log(rng, 600, 262144)
        return _pr(max(1, n // Q), Q, rng.choice([512, 512, 2048, rng.randrange(1, 2049)]), block, hi // 3, hi, lens)
    total = _log(rng, 1, 524288)                     # entries that all the step's queries see
    B = min(_log(rng, 1, 256), max(1, total // 4))
    Q = rng.choice([1, 1, 1, 2, 5])
    hi = max(1, total // (B * Q))
    W = rng.choice([128, 128, 0, rng.randrange(1, 257)])
    return _pa(B, Q, block, rng.choice([max(1, hi // 8), hi]), hi, W, rng.choice(["fp4", "fp4", "bf16"]),
               rng.choice(["bf16", "fp8"]), lens)


def _lens(case):
    """Request lengths of a case, fixed by the case: spread over the logarithm when they span more than a factor of ten."""
    rng = random.Random(case["lens"])
    lo, hi = case["lo"], case["hi"]
    if hi > 10 * max(lo, 1):
        return [min(hi, max(lo, _log(rng, max(lo, 1), hi))) for _ in range(case["B"])]
    return [rng.randint(lo, hi) for _ in range(case["B"])]


def _new(case):
    rng = random.Random(case["lens"] + 1)
    lo, hi = case["new_lo"], case["new_hi"]
    # of a mixed step, most requests decode and some prefill
    return [rng.randint(lo, hi) if rng.random() < 0.3 else min(1, hi) for _ in range(case["B"])]


def _blocks(n, block):
    return -(-n // block)


def work(case):
    B, block = case["B"], case["block"]
    lens = _lens(case)
    if case["op"] == "block_tables":
        new = _new(case)
        taken = sum(_blocks(a + n, block) - _blocks(a, block) for a, n in zip(lens, new))
        slots = sum(new) + case["spare"]
        return {"bytes": 16 * B + 8 * taken + 8 * slots + 4 * B, "flops": 0}
    if case["op"] == "paged_rows":
        n = B * case["Q"] * case["K"]
        table = sum(min(_blocks(a, block), case["Q"] * case["K"]) for a in lens)
        return {"bytes": 8 * n + 4 * table + 4 * B * case["Q"], "flops": 0}
    Q, W = case["Q"], case["W"]
    row = ENTRY if case["kv"] == "fp4" else 2 * D
    wrow = 2 * D if case["window"] == "bf16" else D + 4
    keys = sum(max(0, a - Q + 1 + i) + W for a in lens for i in range(Q))
    by = sum(lens) * row + sum(4 * _blocks(a, block) for a in lens)
    by += B * (W + Q - 1 if W else 0) * wrow
    by += B * Q * (2 * H * D * 2 + 4 * H + 4)
    return {"bytes": by, "flops": keys * H * D * 4}


# ----------------------------------------------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------------------------------------------

_MID = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _quantise(x):
    """[n, 512] floats -> [n, 288] FP4 entries (nibbles, then one E4M3 scale per 16 channels)."""
    n = x.shape[0]
    g = x.view(n, 32, 16)
    s8 = (g.abs().amax(2) / 6).to(torch.float8_e4m3fn)
    s = s8.float().clamp_min(2.0 ** -9)[..., None]
    a = g.abs() / s
    code = torch.zeros_like(g, dtype=torch.uint8)
    for m in _MID:
        code += a > m
    code |= (g < 0).to(torch.uint8) << 3
    c = code.view(n, 256, 2)
    return torch.cat([c[..., 0] | (c[..., 1] << 4), s8.view(torch.uint8)], 1)


def _tables(case, lens, gen, spare_blocks=3):
    """Block tables over a shuffled pool for given final lengths: (table, blocks in the pool)."""
    block = case["block"]
    counts = [_blocks(a, block) for a in lens]
    n_blocks = sum(counts) + spare_blocks
    order = torch.randperm(n_blocks, generator=gen, device=DEV).int()
    width = max(1, max(counts))
    col = torch.arange(width, device=DEV)
    cnt = torch.tensor(counts, device=DEV)
    first = torch.cumsum(cnt, 0) - cnt
    at = (first[:, None] + col).clamp_max(n_blocks - 1)
    return torch.where(col < cnt[:, None], order[at], -1).contiguous(), n_blocks


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return {"block_tables": _prepare_tables, "paged_rows": _prepare_rows, "paged_attn": _prepare_attn}[case["op"]](case, gen)


def _prepare_tables(case, gen):
    B, block = case["B"], case["block"]
    lens, new = _lens(case), _new(case)
    table, n_used = _tables(case, lens, gen, 0)
    width = max(_blocks(a + n, block) for a, n in zip(lens, new))
    width = max(1, width) + 1
    wide = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    wide[:, : table.shape[1]] = table[:, :width]
    taken = sum(_blocks(a + n, block) - _blocks(a, block) for a, n in zip(lens, new))
    n_free = taken + 7
    free = (torch.randperm(n_free, generator=gen, device=DEV) + n_used).int()
    i32 = dict(dtype=torch.int32, device=DEV)
    s = {"op": case["op"], "block": block, "len": torch.tensor(lens, **i32), "new": torch.tensor(new, **i32), "free": free,
         "free_pos": torch.full((1,), 2, **i32), "table": wide, "max_new": max(1, sum(new) + case["spare"])}
    if own:
        from fp4_kv_cache_mxfp4_b200 import csa2
        s["slots"] = torch.empty(s["max_new"], dtype=torch.int64, device=DEV)
        s["start"], s["len_out"], s["info"] = torch.empty(B + 1, **i32), torch.empty(B, **i32), torch.empty(2, **i32)
        s["args"] = csa2.block_table_args(s["len"], s["new"], free, wide, s["slots"], s["start"], s["len_out"], s["info"],
                                          block_size=block, free_pos=s["free_pos"])
        s["ws"] = csa2.workspace(s["args"], csa2.WS_BLOCK_TABLES)
    return s


def _prepare_rows(case, gen):
    B, Q, K, block = case["B"], case["Q"], case["K"], case["block"]
    lens = _lens(case)
    table, n_blocks = _tables(case, lens, gen)
    n = torch.tensor(lens, device=DEV)
    vis = (n[:, None] - Q + 1 + torch.arange(Q, device=DEV)).clamp_min(0)          # causal: the last query sees all
    u = torch.rand(B, Q, K, generator=gen, device=DEV, dtype=torch.float64)
    pos = torch.sort((u * vis[..., None]).int(), dim=2).values
    pos = torch.where(torch.arange(K, device=DEV) < vis[..., None], pos, -1).int()  # padding of short rows
    s = {"op": case["op"], "block": block, "n_blocks": n_blocks, "pos": pos, "vis": vis.int().contiguous(), "table": table}
    if own:
        s["rows"] = torch.empty_like(pos)
    return s


def _prepare_attn(case, gen):
    B, Q, block, W = case["B"], case["Q"], case["block"], case["W"]
    lens = _lens(case)
    table, n_blocks = _tables(case, lens, gen)
    rows = n_blocks * block
    fp4 = case["kv"] == "fp4"
    pool = torch.empty((rows, ENTRY), dtype=torch.uint8, device=DEV) if fp4 else \
        torch.empty((rows, D), dtype=torch.bfloat16, device=DEV)
    for a in range(0, rows, 1 << 17):
        b = min(rows, a + (1 << 17))
        x = torch.randn(b - a, D, generator=gen, device=DEV)
        pool[a:b] = _quantise(x) if fp4 else x.to(torch.bfloat16)
    pool = pool.view(n_blocks, block, -1)
    q = torch.randn(B, Q, H, D, generator=gen, device=DEV).to(torch.bfloat16)       # logits of unit spread
    n = torch.tensor(lens, device=DEV)
    vis = (n[:, None] - Q + 1 + torch.arange(Q, device=DEV)).clamp_min(0).int().contiguous()
    s = {"op": case["op"], "block": block, "W": W, "lens": lens, "Q": Q, "q": q, "pool": pool, "table": table, "vis": vis,
         "swa": None, "swa_scale": None}
    if W:
        x = torch.randn(B, W + Q - 1, D, generator=gen, device=DEV)
        if case["window"] == "bf16":
            s["swa"] = x.to(torch.bfloat16)
        else:
            s["swa_scale"] = (x.abs().amax(2) / 448).contiguous()
            s["swa"] = (x / s["swa_scale"][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    if own:
        from fp4_kv_cache_mxfp4_b200 import csa2
        s["out"] = torch.empty_like(q)
        s["lse"] = torch.empty(B, Q, H, device=DEV)
        s["args"] = csa2.paged_attn_args(q, pool, table, vis, s["out"], s["lse"], swa=s["swa"], W=W, swa_step=1,
                                         swa_scale=s["swa_scale"])
        s["ws"] = csa2.workspace(s["args"], csa2.WS_PAGED_ATTN)
    return s


# ----------------------------------------------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------------------------------------------

def run(state):
    return {"block_tables": _run_tables, "paged_rows": _run_rows, "paged_attn": _run_attn}[state["op"]](state)


def _run_tables(s):
    if own:
        from fp4_kv_cache_mxfp4_b200 import csa2
        csa2.csa2_block_tables(s["args"], s["ws"])
        return [s["table"], s["slots"], s["start"], s["len_out"], s["info"]]
    ln, new, P, table = s["len"].long(), s["new"].long(), s["block"], s["table"]
    B, width = table.shape
    start = torch.zeros(B + 1, dtype=torch.int64, device=DEV)
    start[1:] = torch.cumsum(new, 0)
    have, want = (ln + P - 1) // P, (ln + new + P - 1) // P
    need = want - have
    base = s["free_pos"].long() + torch.cumsum(need, 0) - need
    col = torch.arange(width, device=DEV)
    fresh = (col >= have[:, None]) & (col < want[:, None])
    at = (base[:, None] + col - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], table)
    i = torch.arange(s["max_new"], device=DEV)
    b = torch.searchsorted(start[1:], i, right=True)
    live, b = b < B, b.clamp_max(B - 1)
    pos = ln[b] + i - start[b]
    slots = table[b, (pos // P).clamp_max(width - 1)].long() * P + pos % P
    info = torch.cat([s["free_pos"].long() + need.sum(), torch.zeros(1, dtype=torch.int64, device=DEV)])
    return [table, torch.where(live, slots, -1), start.int(), (ln + new).int(), info.int()]


def _run_rows(s):
    if own:
        from fp4_kv_cache_mxfp4_b200 import csa2
        csa2.csa2_paged_rows(s["pos"], s["table"], s["rows"], block_size=s["block"], n_blocks=s["n_blocks"], n_vis=s["vis"])
        return s["rows"]
    pos, P = s["pos"], s["block"]
    B, Q, K = pos.shape
    ok = (pos >= 0) & (pos < s["vis"][..., None])
    p = torch.where(ok, pos, 0).view(B, Q * K)
    blk = torch.gather(s["table"], 1, (p // P).long())
    return torch.where(ok, (blk * P + p % P).view(B, Q, K), -1)


_FP4_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
_pairs = []


def _dequantise(rows):
    """[n, 288] entries -> [n, 512] float32, both channels of a byte by one lookup."""
    if not _pairs:
        v = torch.tensor(_FP4_VALUES, device=DEV)
        byte = torch.arange(256, device=DEV)
        _pairs.append(torch.stack([v[byte & 15], v[byte >> 4]], 1))
    n = rows.shape[0]
    x = torch.index_select(_pairs[0], 0, rows[:, :256].reshape(-1).int()).view(n, 32, 16)
    return (x * rows[:, 256:].contiguous().view(torch.float8_e4m3fn).float()[..., None]).view(n, D)


def _keys(s, b, a, e):
    """Entries [a, e) of request b in float32."""
    p = torch.arange(a, e, device=DEV)
    rows = s["table"][b, p // s["block"]].long() * s["block"] + p % s["block"]
    got = s["pool"].view(-1, s["pool"].shape[2])[rows]
    return _dequantise(got) if got.dtype == torch.uint8 else got.float()


_CHUNK = 1 << 16


def _run_attn(s):
    if own:
        from fp4_kv_cache_mxfp4_b200 import csa2
        csa2.csa2_paged_attn(s["args"], s["ws"])
        return [s["out"], s["lse"]]
    outs, lses = [], []
    Q, W = s["Q"], s["W"]
    for b, n in enumerate(s["lens"]):
        q = s["q"][b].float().view(Q * H, D) * (D ** -0.5)
        parts = [_keys(s, b, a, min(n, a + _CHUNK)) for a in range(0, n, _CHUNK)] if n <= 4 * _CHUNK else None
        spans = [(a, min(n, a + _CHUNK)) for a in range(0, n, _CHUNK)]
        z = [q @ (parts[i] if parts else _keys(s, b, a, e)).T for i, (a, e) in enumerate(spans)]
        z = torch.cat(z, 1).view(Q, H, n)
        z = torch.where(torch.arange(n, device=DEV) < s["vis"][b][:, None, None], z, -math.inf)
        if W:
            win = s["swa"][b].float() if s["swa_scale"] is None else \
                s["swa"][b].view(torch.float8_e4m3fn).float() * s["swa_scale"][b][:, None]
            zw = (q @ win.T).view(Q, H, W + Q - 1)
            r, i = torch.arange(W + Q - 1, device=DEV), torch.arange(Q, device=DEV)[:, None, None]
            z = torch.cat([z, torch.where((r >= i) & (r < i + W), zw, -math.inf)], 2)
        m = z.amax(2, keepdim=True)
        p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
        total = p.sum(2, keepdim=True)
        p = p.view(Q * H, -1)
        o = torch.zeros(Q * H, D, device=DEV)
        for i, (a, e) in enumerate(spans):
            o += p[:, a:e] @ (parts[i] if parts else _keys(s, b, a, e))
        if W:
            o += p[:, n:] @ win
        o = o.view(Q, H, D) / torch.where(total == 0, 1.0, total)
        outs.append(o.to(torch.bfloat16))
        lses.append((m + torch.log(total))[..., 0])
    return [torch.stack(outs), torch.stack(lses)]


# ----------------------------------------------------------------------------------------------------------------------
# exact values: the definition in 64 bits
# ----------------------------------------------------------------------------------------------------------------------

def _e2m1(code):
    """The value of E2M1 codes: sign, two exponent bits (bias 1), one mantissa bit."""
    e, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1))
    return torch.where(code >= 8, -mag, mag)


def _e4m3(code):
    """The value of E4M3 scale codes: four exponent bits (bias 7), three mantissa bits."""
    e, m = ((code >> 3) & 15).double(), (code & 7).double()
    mag = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e - 7))
    return torch.where(code >= 128, -mag, mag)


def _entries64(raw):
    if raw.dtype != torch.uint8:
        return raw.double()
    raw = raw.int()
    vals = torch.empty(raw.shape[0], D, dtype=torch.float64, device=raw.device)
    vals[:, 0::2] = _e2m1(raw[:, :256] & 15)
    vals[:, 1::2] = _e2m1(raw[:, :256] >> 4)
    return vals * _e4m3(raw[:, 256:]).repeat_interleave(16, 1)


def exact(case, seed):
    if case["op"] != "paged_attn":
        return None
    s = prepare(case, seed)
    B, Q, block, W = case["B"], case["Q"], case["block"], case["W"]
    out = torch.zeros(B, Q, H, D, dtype=torch.float64, device=DEV)
    lse = torch.full((B, Q, H), -math.inf, dtype=torch.float64, device=DEV)
    step = 1 << 15
    for b in range(B):
        n = case_n = _lens(case)[b]
        order = s["table"][b, : _blocks(n, block)].long()
        # running maximum, sum and weighted sum per (query, head)
        m = torch.full((Q, H, 1), -math.inf, dtype=torch.float64, device=DEV)
        l = torch.zeros(Q, H, 1, dtype=torch.float64, device=DEV)
        acc = torch.zeros(Q, H, D, dtype=torch.float64, device=DEV)
        pieces = []
        per = max(1, step // block)
        for j in range(0, order.numel(), per):
            keys = s["pool"][order[j: j + per]].flatten(0, 1)[: case_n - j * block]
            at = torch.arange(keys.shape[0], device=DEV) + j * block
            seen = torch.stack([at < n - Q + 1 + i for i in range(Q)])
            pieces.append((keys, None, seen))
        if W:
            at = torch.arange(W + Q - 1, device=DEV)
            pieces.append((s["swa"][b], s["swa_scale"], torch.stack([(at >= i) & (at < i + W) for i in range(Q)])))
        for keys, scale, seen in pieces:
            k = _e4m3(keys.int()) * scale[b].double()[:, None] if scale is not None else _entries64(keys)
            z = torch.einsum("qhd,nd->qhn", s["q"][b].double(), k) / math.sqrt(D)
            z = z.masked_fill(~seen[:, None], -math.inf)
            top = torch.maximum(m, z.amax(2, keepdim=True))
            safe = top.masked_fill(top == -math.inf, 0.0)
            w, old = torch.exp(z - safe), torch.exp(m - safe)
            l = l * old + w.sum(2, keepdim=True)
            acc = acc * old + torch.einsum("qhn,nd->qhd", w, k)
            m = top
        out[b] = acc / l.masked_fill(l == 0, 1.0)
        lse[b] = (m + torch.log(l))[..., 0]
    return [out, lse]
