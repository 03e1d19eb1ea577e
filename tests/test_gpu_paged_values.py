"""GPU tests of the paged attention on the values at its borders: absent keys
beside rows that are not finite.  Cases and tolerances as in test_gpu_paged."""

import math

import torch
import pytest

from fp4_kv_cache_mxfp4_b200 import csa2
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
    assert torch.all(torch.isfinite(out)) and torch.all(out[1::2] == 0)
    # float32: log2 and a product, half a unit in the last place each, log2 with one more
    assert torch.all((lse[::2] - 27 * math.log(2)).abs() <= 2.0 ** -22 * 27 * math.log(2)) and torch.all(lse[1::2] == -math.inf)
