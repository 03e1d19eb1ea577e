"""Host-side checks of the paged-cache calls, without a GPU: struct layouts,
refusals before any device work, workspace sizes, and the binding's own
checks of types, shapes, strides and devices."""

import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

from fp4_kv_cache_mxfp4_b200 import build, csa2

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000          # 16-byte aligned stand-in pointer, never dereferenced
ARG, SHAPE, ALIGN, WS = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    build.build()
    return csa2.load()


def test_struct_layouts_match_the_header():
    structs = {"csa2_block_table_args": csa2.BlockTableArgs, "csa2_paged_rows_args": csa2.PagedRowsArgs,
               "csa2_paged_attn_args": csa2.PagedAttnArgs}
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "csa2.h"', "int main(void) {"]
    for s, t in structs.items():
        lines.append(f'printf("{s} %zu\\n", sizeof({s}));')
        lines += [f'printf("{s}.{f} %zu\\n", offsetof({s}, {f}));' for f, _ in t._fields_]
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(src, "w").write("\n".join(lines + ["return 0; }"]))
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", exe, src], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    c = dict(line.split() for line in out.strip().splitlines())
    for s, t in structs.items():
        assert int(c[s]) == ctypes.sizeof(t)
        for f, _ in t._fields_:
            assert int(c[f"{s}.{f}"]) == getattr(t, f).offset, (s, f)


def _tables(**kw):
    a = dict(B=4, block_size=16, max_blocks=8, ld_table=8, len=FAKE, n_new=FAKE, free_blocks=FAKE, n_free=10, free_pos=None,
             block_table=FAKE, len_out=FAKE, start=FAKE, slots=FAKE, max_new=64, info=FAKE)
    return csa2.BlockTableArgs(**{**a, **kw})


def _rows(**kw):
    a = dict(B=2, Q=3, K=512, block_size=16, max_blocks=8, ld_table=8, n_blocks=100, positions=FAKE, n_vis=FAKE,
             block_table=FAKE, rows=FAKE)
    return csa2.PagedRowsArgs(**{**a, **kw})


def _attn(**kw):
    a = dict(B=2, Q=3, W=128, block_size=16, max_blocks=8, ld_table=8, n_blocks=100, block_stride=16 * 288, q=FAKE, kv=FAKE,
             kv_format=csa2.FMT_NVFP4, block_table=FAKE, n_vis=FAKE, swa=FAKE, swa_rows=130, swa_step=1,
             swa_format=csa2.FMT_BF16, swa_scale=None, scale=0.0, out=FAKE, lse=FAKE)
    return csa2.PagedAttnArgs(**{**a, **kw})


TABLE_REFUSALS = [
    (dict(B=0), SHAPE), (dict(B=65536), SHAPE), (dict(block_size=0), SHAPE), (dict(max_blocks=0), SHAPE),
    (dict(ld_table=7), SHAPE), (dict(block_size=1 << 20, max_blocks=1 << 11, ld_table=1 << 11), SHAPE),
    (dict(n_free=-1), SHAPE), (dict(max_new=-1), SHAPE), (dict(max_new=1 << 31), SHAPE),
    (dict(len=None), ARG), (dict(n_new=None), ARG), (dict(free_blocks=None), ARG), (dict(block_table=None), ARG),
    (dict(len_out=None), ARG), (dict(start=None), ARG), (dict(slots=None), ARG), (dict(info=None), ARG),
    (dict(len=FAKE + 4), ALIGN), (dict(free_pos=FAKE + 8), ALIGN), (dict(slots=FAKE + 8), ALIGN),
]
ROW_REFUSALS = [
    (dict(B=0), SHAPE), (dict(Q=0), SHAPE), (dict(B=40000, Q=2), SHAPE), (dict(K=0), SHAPE),
    (dict(B=1, Q=65535, K=32769), SHAPE), (dict(n_blocks=0), SHAPE), (dict(block_size=32, n_blocks=1 << 26), SHAPE),
    (dict(ld_table=7), SHAPE), (dict(positions=None), ARG), (dict(block_table=None), ARG), (dict(rows=None), ARG),
    (dict(rows=FAKE + 4), ALIGN), (dict(n_vis=FAKE + 4), ALIGN),
]
ATTN_REFUSALS = [
    (dict(B=0), SHAPE), (dict(Q=0), SHAPE), (dict(B=40000, Q=2), SHAPE), (dict(W=-1), SHAPE), (dict(W=1025, swa_rows=5000), SHAPE),
    (dict(block_size=0), SHAPE), (dict(max_blocks=0), SHAPE), (dict(ld_table=7), SHAPE), (dict(n_blocks=0), SHAPE),
    (dict(n_blocks=1 << 31), SHAPE), (dict(block_stride=16 * 288 - 16), SHAPE), (dict(swa_step=-1), SHAPE),
    (dict(swa_rows=129), SHAPE), (dict(kv_format=csa2.FMT_BF16), SHAPE),          # bf16 rows need 16 x 1024 bytes
    (dict(block_size=1 << 20, max_blocks=1 << 11, ld_table=1 << 11, block_stride=288 << 20), SHAPE),
    (dict(kv_format=csa2.FMT_FP8), ARG), (dict(swa_format=csa2.FMT_MXFP4), ARG),
    (dict(swa_format=csa2.FMT_FP8), ARG), (dict(q=None), ARG), (dict(kv=None), ARG), (dict(block_table=None), ARG),
    (dict(n_vis=None), ARG), (dict(swa=None), ARG), (dict(out=None), ARG),
    (dict(block_stride=16 * 288 + 8), ALIGN), (dict(q=FAKE + 8), ALIGN), (dict(kv=FAKE + 8), ALIGN),
    (dict(n_vis=FAKE + 4), ALIGN), (dict(lse=FAKE + 4), ALIGN), (dict(swa=FAKE + 2), ALIGN),
    (dict(swa_format=csa2.FMT_FP8, swa_scale=FAKE + 2), ALIGN),
]


@pytest.mark.parametrize("kw,status", TABLE_REFUSALS)
def test_block_tables_refusals(L, kw, status):
    a = _tables(**kw)
    assert L.csa2_block_tables(ctypes.byref(a), FAKE, 1 << 30, None) == status
    assert csa2.csa2_workspace_size(a, csa2.WS_BLOCK_TABLES) == 0


@pytest.mark.parametrize("kw,status", ROW_REFUSALS)
def test_paged_rows_refusals(L, kw, status):
    assert L.csa2_paged_rows(ctypes.byref(_rows(**kw)), None) == status


@pytest.mark.parametrize("kw,status", ATTN_REFUSALS)
def test_paged_attn_refusals(L, kw, status):
    a = _attn(**kw)
    assert L.csa2_paged_attn(ctypes.byref(a), FAKE, 1 << 40, None) == status
    assert csa2.csa2_workspace_size(a, csa2.WS_PAGED_ATTN) == 0


def test_null_arguments_and_workspaces(L):
    assert L.csa2_block_tables(None, FAKE, 1 << 30, None) == ARG
    assert L.csa2_paged_rows(None, None) == ARG
    assert L.csa2_paged_attn(None, FAKE, 1 << 30, None) == ARG
    for call, a, which in ((L.csa2_block_tables, _tables(), csa2.WS_BLOCK_TABLES),
                           (L.csa2_paged_attn, _attn(), csa2.WS_PAGED_ATTN)):
        n = csa2.csa2_workspace_size(a, which)
        assert n > 0
        assert call(ctypes.byref(a), None, n, None) == WS
        assert call(ctypes.byref(a), FAKE, n - 1, None) == WS
        assert call(ctypes.byref(a), FAKE + 8, n, None) == WS


def test_workspace_sizes():
    """The attention's workspace is bounded by the SMs, not by the batch."""
    small = csa2.csa2_workspace_size(_attn(B=1, Q=1, max_blocks=1), csa2.WS_PAGED_ATTN)
    large = csa2.csa2_workspace_size(_attn(B=60000, Q=1, swa_rows=128), csa2.WS_PAGED_ATTN)
    assert small < 1 << 20 < large < 40 << 20


def test_binding_checks():
    """Wrong types, shapes, strides and devices are refused before the library sees a pointer."""
    i32 = dict(dtype=torch.int32)
    q, out = torch.zeros(2, 1, 64, 512, dtype=torch.bfloat16), torch.zeros(2, 1, 64, 512, dtype=torch.bfloat16)
    kv, table, vis = torch.zeros(6, 4, 288, dtype=torch.uint8), torch.zeros(2, 3, **i32), torch.zeros(2, 1, **i32)
    ok = csa2.paged_attn_args(q, kv, table, vis, out)
    assert (ok.block_size, ok.max_blocks, ok.ld_table, ok.n_blocks, ok.block_stride) == (4, 3, 3, 6, 4 * 288)
    for bad in ((q.float(), kv, table, vis, out), (q, kv.to(torch.int8), table, vis, out), (q, kv[..., :287], table, vis, out),
                (q, kv[:, ::2], table, vis, out), (q, kv, table.long(), vis, out), (q, kv, table.t(), vis, out),
                (q, kv, table, vis.long(), out), (q, kv, table, vis, out[:1]), (q, kv, table, vis, out.transpose(2, 3)),
                (q, kv, table, vis.to("meta"), out)):
        with pytest.raises(ValueError):
            csa2.paged_attn_args(*bad)
    with pytest.raises(ValueError):
        csa2.paged_attn_args(q, kv, table, vis, out, W=8)
    with pytest.raises(ValueError):
        csa2.paged_attn_args(q, kv, table, vis, out, W=8, swa=torch.zeros(2, 8, 512))
    # an expanded pool or table has no distance between its blocks or rows: the library refuses it
    for a in (csa2.paged_attn_args(q, kv[:1].expand(6, 4, 288), table, vis, out),
              csa2.paged_attn_args(q, kv, table[:1].expand(2, 3), vis, out)):
        assert csa2.csa2_workspace_size(a, csa2.WS_PAGED_ATTN) == 0
    # blocks and table rows that lie apart are passed on with their distance
    wide = torch.zeros(6, 3, 4, 288, dtype=torch.uint8)[:, 1]
    apart = csa2.paged_attn_args(q, wide, torch.zeros(2, 10, **i32)[:, :3], vis, out)
    assert (apart.block_stride, apart.ld_table, apart.max_blocks) == (3 * 4 * 288, 10, 3)
    # tensors that are not on a GPU never reach a launch
    with pytest.raises(ValueError):
        csa2.csa2_paged_attn(ok, torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError):
        csa2.csa2_paged_rows(torch.zeros(2, 1, 8, **i32), table, torch.zeros(2, 1, 8, **i32), block_size=4, n_blocks=6)
    with pytest.raises(ValueError):
        csa2.csa2_paged_rows(torch.zeros(2, 1, 8, **i32), table, torch.zeros(2, 8, 1, **i32), block_size=4, n_blocks=6)
    z = lambda n, t=torch.int32: torch.zeros(n, dtype=t)
    t = csa2.block_table_args(z(2), z(2), z(5), table, z(9, torch.int64), z(3), z(2), z(2), block_size=4)
    assert (t.B, t.n_free, t.max_new) == (2, 5, 9)
    with pytest.raises(ValueError):
        csa2.csa2_block_tables(t, torch.zeros(1024, dtype=torch.uint8))
    for bad in ((z(2), z(3), z(5), table, z(9, torch.int64), z(3), z(2), z(2)),
                (z(2), z(2), z(5), table, z(9), z(3), z(2), z(2)),
                (z(2), z(2), z(5), table, z(9, torch.int64), z(2), z(2), z(2)),
                (z(2), z(2), z(5), table, z(9, torch.int64), z(3), z(2), z(1))):
        with pytest.raises(ValueError):
            csa2.block_table_args(*bad, block_size=4)


def test_output_over_the_queries_is_refused():
    q = torch.zeros(2, 1, 64, 512, dtype=torch.bfloat16)
    kv, table = torch.zeros(6, 4, 288, dtype=torch.uint8), torch.zeros(2, 3, dtype=torch.int32)
    vis = torch.zeros(2, 1, dtype=torch.int32)
    csa2.paged_attn_args(q, kv, table, vis, torch.zeros_like(q))
    with pytest.raises(ValueError, match="out must not be q"):
        csa2.paged_attn_args(q, kv, table, vis, q)


def test_outputs_that_share_bytes_with_inputs_are_refused():
    """Anywhere, not only at the start; what lies between a pool's blocks is not the pool."""
    buf = torch.zeros(1 << 21, dtype=torch.uint8)
    at = lambda first, dtype, *shape: buf[first: first + torch.Size(shape).numel() * dtype.itemsize].view(dtype).view(shape)
    n = 2 * 64 * 512 * 2                                 # bytes of q and of out
    q, table, vis = at(0, torch.bfloat16, 2, 1, 64, 512), at(n, torch.int32, 2, 3), at(n + 32, torch.int32, 2, 1)
    kv = at(4 * n, torch.uint8, 6, 4, 288)
    far = lambda: torch.zeros(2, 1, 64, 512, dtype=torch.bfloat16)
    lse = lambda: torch.zeros(2, 1, 64)
    args = csa2.paged_attn_args
    args(q, kv, table, vis, at(n + 48, torch.bfloat16, 2, 1, 64, 512), at(4 * n - 512, torch.float32, 2, 1, 64))
    for first, what in ((n - 16, "q"), (16, "q"), (n + 16, "block_table"), (n + 32, "n_vis"), (4 * n - 16, "kv"),
                        (4 * n + 6 * 4 * 288 - 16, "kv")):
        with pytest.raises(ValueError, match=f"out must not be {what}"):
            args(q, kv, table, vis, at(first, torch.bfloat16, 2, 1, 64, 512))
    for first, what in ((n - 16, "q"), (n + 16, "block_table"), (4 * n - 16, "kv")):
        with pytest.raises(ValueError, match=f"lse must not be {what}"):
            args(q, kv, table, vis, far(), at(first, torch.float32, 2, 1, 64))
    out = far()
    with pytest.raises(ValueError, match="out must not be lse"):
        args(q, kv, table, vis, out, out.view(-1).view(torch.float32)[64:192].view(2, 1, 64))
    swa = torch.zeros(2, 128, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="out must not be swa"):
        args(q, kv, table, vis, swa[:1].view(2, 1, 64, 512), swa=swa, W=128)
    codes, scale = torch.zeros(2, 128, 512, dtype=torch.uint8), torch.zeros(2, 128)
    with pytest.raises(ValueError, match="lse must not be swa_scale"):
        args(q, kv, table, vis, far(), scale.view(-1)[128:].view(2, 1, 64), swa=codes, W=128, swa_scale=scale)
    # blocks of two layers in one pool, and a log-sum-exp in the gap
    wide = torch.zeros(6, 2, 4, 288, dtype=torch.uint8)
    gap = lambda i, first: wide[i].view(-1)[first: first + 512].view(torch.float32).view(2, 1, 64)
    args(q, wide[:, 0], table, vis, far(), gap(2, 4 * 288))
    args(q, wide[:, 0], table, vis, far(), gap(5, 4 * 288 + 512))
    args(q, wide[:, 1], table, vis, far(), gap(0, 0))
    for i, first in ((0, 4 * 288 - 16), (2, 4 * 288 - 512), (5, 0)):
        with pytest.raises(ValueError, match="lse must not be kv"):
            args(q, wide[:, 0], table, vis, far(), gap(i, first))
