// paged_attention.cuh -- attention of each request's query positions over all
// its visible entries in a block-paged cache plus its layer's window rows,
// one softmax (csa2_paged_attn).
//
// Work unit: a tile of 128 keys of one query (its 64 heads).  A query has
// ceil(n_vis / 128) tiles of cache entries and ceil(W / 128) tiles of window
// rows.  The tiles of all queries, in order, are cut into one equal range
// per CTA (one CTA per SM), whatever the lengths: a long query is split over
// many CTAs, a CTA may serve several short queries.  The ranges come from
// n_vis on the device, so a captured launch serves growing lengths.
//   query inside one CTA's range   normalised and written as bf16
//   query cut by a range boundary  each CTA leaves an unnormalised fp32
//                                  partial and its per-head (max, sum);
//                                  paged_attn_join_kernel merges them in
//                                  CTA order (a fixed order: results do not
//                                  depend on timing)
// A CTA has at most two partials: its first query (when that began in an
// earlier range) and its last (when that goes on).
//
// Tile mathematics as in attention_tc.cuh: S^T[key, head] = K . Q^T
// (M = 128 keys, N = 64), weights exp2(S^T - ref) in bf16 against a running
// reference, O^T[dim, head] += V^T . P^T with the same key tile.
#pragma once
#include "common.cuh"
#include "quantize.cuh"
#include "attention_tc.cuh"

namespace csa2 {

constexpr int kPagedThreads = 512;
constexpr int kPagedKeys = 128;                        // keys per tile (MMA M)
constexpr int kPagedMaxCtas = 148;                     // one per SM of a B200
constexpr uint32_t kPagedSmem = kTcAttnSmem;

struct PagedAttnParams {
  int BQ, Q, W;
  int w_tiles;               // ceil(W / 128)
  uint32_t block_size, max_blocks;
  int64_t ld_table, n_blocks, block_stride;            // block_stride in bytes
  const uint8_t* kv;
  int kv_bf16;               // cache rows: 0 FP4 entries (288 B), 1 bf16 (1024 B)
  const int32_t* table;
  const int32_t* n_vis;      // [B][Q]
  const uint8_t* swa;        // bf16 rows or E4M3 codes
  const float* swa_scale;    // FP8 window: [B][swa_rows]
  int swa_fp8, swa_rows, swa_step;
  float scale_log2;
  __nv_bfloat16* out;        // [BQ][64][512]
  float* lse;                // optional [BQ][64]
  float* opart;              // [2 * CTAs][64][512] unnormalised partials
  float* ml;                 // [2 * CTAs][64][2]: reference (log2 units), sum
  int32_t* first_row;        // [CTAs]: the query a CTA's range begins inside of, -1 if it begins with a new one
};

// Tiles of query r: at least one, so that a query without any key is written too.
__device__ __forceinline__ int64_t paged_tiles(const PagedAttnParams& p, int r, int* keys) {
  const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.block_size;
  const int64_t n = min(static_cast<int64_t>(max(p.n_vis[r], 0)), cap);
  *keys = static_cast<int>(n);
  return max((n + kPagedKeys - 1) / kPagedKeys + p.w_tiles, static_cast<int64_t>(1));
}

// This CTA's tile range [lo, hi) of the total, the query that lo lies in and
// lo's offset inside it.  Every CTA sums the tiles of all queries (4 bytes
// each from L2); every thread calls it.
struct PagedRange { int64_t lo, hi; int row; int64_t offset; };
__device__ __forceinline__ PagedRange paged_range(const PagedAttnParams& p, int64_t* warp_s, PagedRange* range_s) {
  const int per = (p.BQ + blockDim.x - 1) / blockDim.x;
  const int r0 = min(p.BQ, static_cast<int>(threadIdx.x) * per), r1 = min(p.BQ, r0 + per);
  int64_t mine = 0, total = 0;
  int keys;
  for (int r = r0; r < r1; ++r) mine += paged_tiles(p, r, &keys);
  int64_t at = block_exclusive_sum(mine, warp_s, &total);
  // no CTA without a tile between two that have one (the join looks at neighbours)
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);
  if (blockIdx.x >= ctas) return PagedRange{0, 0, 0, 0};
  const int64_t lo = total * blockIdx.x / ctas, hi = total * (blockIdx.x + 1) / ctas;
  if (lo >= at && lo < at + mine) {
    for (int r = r0; r < r1; ++r) {
      const int64_t t = paged_tiles(p, r, &keys);
      if (lo < at + t) { *range_s = PagedRange{lo, hi, r, lo - at}; break; }
      at += t;
    }
  }
  __syncthreads();
  return *range_s;
}

// Address of entry `pos` of a request's cache; nullptr where the table names no block of the pool.
__device__ __forceinline__ const uint8_t* paged_row(const PagedAttnParams& p, const int32_t* table, uint32_t pos,
                                                    uint32_t row_bytes) {
  const uint32_t blk = pos / p.block_size;
  const int32_t id = table[blk];
  if (id < 0 || id >= p.n_blocks) return nullptr;
  return p.kv + id * p.block_stride + static_cast<int64_t>(pos - blk * p.block_size) * row_bytes;
}

__global__ void __launch_bounds__(kPagedThreads, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap tmap_q, PagedAttnParams p) {
  extern __shared__ __align__(1024) uint8_t paged_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(paged_smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* kt = smem;
  uint8_t* qt = smem + kTcKeyTileBytes;
  uint8_t* pt = qt + kTcQTileBytes;
  uint8_t* misc = pt + kTcPTileBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(misc);   // [0] Q TMA, [1] MMA 1 done, [2] MMA 2 done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 48);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 52);
  int* rescale_flag = reinterpret_cast<int*>(misc + 56);
  float* red_s = reinterpret_cast<float*>(misc + 576);
  float* ref_s = reinterpret_cast<float*>(misc + 2624);
  float* sum_s = reinterpret_cast<float*>(misc + 2880);
  float* fac_s = reinterpret_cast<float*>(misc + 3136);
  float* wsc_s = reinterpret_cast<float*>(misc + 3392);               // [128] FP8 window: row scale per key
  const uint8_t** row_s = reinterpret_cast<const uint8_t**>(misc + 4096);   // [128] key addresses, null = no key
  int64_t* warp_s = reinterpret_cast<int64_t*>(misc + 5632);          // [33]
  PagedRange* range_s = reinterpret_cast<PagedRange*>(misc + 6016);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < 3; ++i) mbar_init(&bars[i], 1);
    *abort_flag = 0;
    *rescale_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmap_q);
  }
  if (warp == 1) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  pdl_launch_dependents();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const PagedRange range = paged_range(p, warp_s, range_s);
  if (tid == 0) p.first_row[blockIdx.x] = (range.lo < range.hi && range.offset > 0) ? range.row : -1;

  uint32_t ph_q = 0, ph_mma = 0;
  int row = range.row;
  int64_t offset = range.offset;
  for (int64_t at = range.lo; at < range.hi; ++row) {
    int keys;
    const int64_t tiles = paged_tiles(p, row, &keys);
    const int kv_tiles = (keys + kPagedKeys - 1) / kPagedKeys;
    const int64_t t0 = offset, t1 = min(tiles, offset + (range.hi - at));
    const int b = row / p.Q, qi = row - b * p.Q;
    const int32_t* table = p.table + b * p.ld_table;
    if (tid == 0) {
      mbar_arrive_expect_tx(&bars[0], kTcQTileBytes);
      const uint64_t pol = l2_policy_evict_last();
      for (int c = 0; c < 8; ++c) tma_load_2d(qt + c * 8192, &tmap_q, &bars[0], 64 * c, row * 64, pol);
    }
    if (tid < 64) { ref_s[tid] = -INFINITY; sum_s[tid] = 0.0f; }
    for (int64_t t = t0; t < t1; ++t) {
      const bool window = t >= kv_tiles;
      const int key0 = static_cast<int>((window ? t - kv_tiles : t) * kPagedKeys);
      const int nkeys = max(0, min(kPagedKeys, (window ? p.W : keys) - key0));
      const bool win8 = window && p.swa_fp8;
      const bool bf16_rows = window ? !p.swa_fp8 : p.kv_bf16 != 0;
      if (tid < kPagedKeys) {
        const uint8_t* a = nullptr;
        float s = 0.0f;
        if (tid < nkeys) {
          if (window) {
            const int64_t r = static_cast<int64_t>(b) * p.swa_rows + qi * p.swa_step + key0 + tid;
            a = p.swa + r * (p.swa_fp8 ? 512 : 1024);
            if (p.swa_fp8) s = p.swa_scale[r];
          } else {
            a = paged_row(p, table, static_cast<uint32_t>(key0 + tid), p.kv_bf16 ? 1024 : 288);
          }
        }
        row_s[tid] = a;
        wsc_s[tid] = s;
      }
      __syncthreads();
      // warp w loads keys 8w..8w+7; a key that is not there becomes zeros
      if (bf16_rows) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = 8 * warp + j;
          const uint4* src = reinterpret_cast<const uint4*>(row_s[r]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int u = lane + 32 * h;
            const uint4 v = src ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(kt + (u >> 3) * 16384 + sw128_off(r, u & 7)) = v;
          }
        }
      } else if (win8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = 8 * warp + j;
          const uint4* src = reinterpret_cast<const uint4*>(row_s[r]);
          const uint4 raw = src ? __ldg(src + lane) : make_uint4(0, 0, 0, 0);
          uint32_t o[8];
          e4m3x4_to_bf16(raw.x, o[0], o[1]);
          e4m3x4_to_bf16(raw.y, o[2], o[3]);
          e4m3x4_to_bf16(raw.z, o[4], o[5]);
          e4m3x4_to_bf16(raw.w, o[6], o[7]);
          uint8_t* chunk = kt + (lane >> 2) * 16384;
          *reinterpret_cast<uint4*>(chunk + sw128_off(r, 2 * (lane & 3))) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(chunk + sw128_off(r, 2 * (lane & 3) + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      } else {
        // FP4: half a row (16 lanes x 16 nibble bytes) of two keys per load
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 8 * warp + 2 * j + (lane >> 4), c = lane & 15;
          const uint8_t* src = row_s[r];
          const uint4 nib = src ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0, 0, 0, 0);
          const uint32_t sc = src ? __ldg(reinterpret_cast<const uint16_t*>(src + 256) + c) : 0;
          const float s0 = e4m3_code_to_float(sc & 0xFF), s1 = e4m3_code_to_float(sc >> 8);
          const __nv_bfloat162 S0 = __floats2bfloat162_rn(s0, s0), S1 = __floats2bfloat162_rn(s1, s1);
          uint32_t o[4][4];
          e2m1x8_to_bf16(nib.x, S0, o[0]);
          e2m1x8_to_bf16(nib.y, S0, o[1]);
          e2m1x8_to_bf16(nib.z, S1, o[2]);
          e2m1x8_to_bf16(nib.w, S1, o[3]);
          uint8_t* chunk = kt + (c >> 1) * 16384;
#pragma unroll
          for (int u = 0; u < 4; ++u)
            *reinterpret_cast<uint4*>(chunk + sw128_off(r, 4 * (c & 1) + u)) = make_uint4(o[u][0], o[u][1], o[u][2], o[u][3]);
        }
      }
      fence_async_smem();
      __syncthreads();

      // S^T = K . Q^T
      if (warp == 1 && lane == 0) {
        if (mbar_wait(&bars[0], ph_q, kErrWaitOperand, abort_flag)) {
          tc_fence_after();
          constexpr uint32_t idesc = umma_idesc_bf16_f32(128, 64);
          const uint32_t ka = smem_u32(kt), qa = smem_u32(qt);
#pragma unroll
          for (int kk = 0; kk < 32; ++kk)
            umma_bf16(tmem, umma_desc_sw128_kmajor(ka + (kk >> 2) * 16384 + (kk & 3) * 32),
                      umma_desc_sw128_kmajor(qa + (kk >> 2) * 8192 + (kk & 3) * 32), idesc, kk > 0);
        }
        umma_commit(&bars[1]);
      }
      const bool first = t == t0;
      {
        const int quarter = warp & 3, hg = warp >> 2;
        const int key = quarter * 32 + lane;
        float sv[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) sv[j] = -INFINITY;
        const bool ok = mbar_wait(&bars[1], ph_mma, kErrWaitTmemFull, abort_flag);
        if (__all_sync(0xffffffffu, ok)) {
          tc_fence_after();
          const bool there = row_s[key] != nullptr;
          const float ls = p.scale_log2 * (win8 ? wsc_s[key] : 1.0f);
          uint32_t r[16];
          tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + 16 * hg, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) sv[j] = there ? __uint_as_float(r[j]) * ls : -INFINITY;
        }
        const float m = warp_reduce_heads16<true>(sv, lane);
        if ((lane & 1) == 0) red_s[quarter * 64 + 16 * hg + (lane >> 1)] = m;
        __syncthreads();
        float lj[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int h = 16 * hg + j;
          const float mt = fmaxf(fmaxf(red_s[h], red_s[64 + h]), fmaxf(red_s[128 + h], red_s[192 + h]));
          const float ref = ref_s[h];
          const float nref = (mt > ref + kTcRefSlack) ? mt : ref;
          lj[j] = exp2f(sv[j] - ((nref == -INFINITY) ? 0.0f : nref));
        }
        // an FP8 window key's row scale goes into the weight that multiplies
        // its codes; the sum takes the weights that the rounded products stand for
        const float rs = win8 ? wsc_s[key] : 1.0f, inv = rs != 0.0f ? 1.0f / rs : 0.0f;
        uint32_t pk[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const __nv_bfloat162 v2 = __floats2bfloat162_rn(lj[2 * j] * rs, lj[2 * j + 1] * rs);
          pk[j] = *reinterpret_cast<const uint32_t*>(&v2);
          const float2 f = __bfloat1622float2(v2);
          if (rs != 0.0f) { lj[2 * j] = f.x * inv; lj[2 * j + 1] = f.y * inv; }
        }
        *reinterpret_cast<uint4*>(pt + sw128_off(key, 2 * hg)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
        *reinterpret_cast<uint4*>(pt + sw128_off(key, 2 * hg + 1)) = make_uint4(pk[4], pk[5], pk[6], pk[7]);
        const float l = warp_reduce_heads16<false>(lj, lane);
        if ((lane & 1) == 0) red_s[256 + quarter * 64 + 16 * hg + (lane >> 1)] = l;
        fence_async_smem();
        __syncthreads();
        if (tid < 64) {
          const int h = tid;
          const float mt = fmaxf(fmaxf(red_s[h], red_s[64 + h]), fmaxf(red_s[128 + h], red_s[192 + h]));
          const float ls = (red_s[256 + h] + red_s[320 + h]) + (red_s[384 + h] + red_s[448 + h]);
          const float ref = ref_s[h];
          const float nref = (mt > ref + kTcRefSlack) ? mt : ref;
          const float f = (nref == ref || ref == -INFINITY) ? 1.0f : exp2f(ref - nref);
          fac_s[h] = f;
          if (f != 1.0f && !first) *rescale_flag = 1;
          ref_s[h] = nref;
          sum_s[h] = sum_s[h] * f + ls;
        }
        tc_fence_before();
        __syncthreads();
      }
      if (*rescale_flag) {
        const int quarter = warp & 3, tt = warp >> 2;
#pragma unroll 1
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t r[32];
          const uint32_t taddr = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + 64 + 64 * tt + 32 * hh;
          tc_fence_after();
          tmem_ld_32x32b_x32(taddr, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * fac_s[32 * hh + j]);
          tmem_st_32x32b_x32(taddr, r);
          tmem_st_wait();
        }
        tc_fence_before();
        __syncthreads();
        if (tid == 0) *rescale_flag = 0;
      }
      // O^T += V^T . P^T
      if (warp == 1 && lane == 0) {
        tc_fence_after();
        if (!*abort_flag) {
          constexpr uint32_t idesc = umma_idesc_bf16_f32(128, 64) | (1u << 15) | (1u << 16);
          const uint32_t ka = smem_u32(kt), pa = smem_u32(pt);
#pragma unroll
          for (int tt = 0; tt < 4; ++tt) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_bf16(tmem + 64 + 64 * tt, umma_desc_sw128_mnmajor(ka + (2 * tt) * 16384 + kk * 2048, 16384),
                        umma_desc_sw128_mnmajor(pa + kk * 2048, 16384), idesc, (!first || kk > 0) ? 1u : 0u);
          }
        }
        umma_commit(&bars[2]);
      }
      // the key tile and P^T are free once MMA 2 is done
      mbar_wait(&bars[2], ph_mma, kErrWaitTmemFull, abort_flag);
      tc_fence_after();
      ph_mma ^= 1;
      __syncthreads();
    }
    ph_q ^= 1;

    // the query's result, or this CTA's partial of it
    const bool whole = t0 == 0 && t1 == tiles;
    const int slot = 2 * blockIdx.x + (t0 == 0 ? 1 : 0);
    float* obuf = reinterpret_cast<float*>(kt);
    if (!*abort_flag) {
      const int quarter = warp & 3, tt = warp >> 2;
      const int d = 128 * tt + 32 * quarter + lane;
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + 64 + 64 * tt + 32 * hh, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float l = sum_s[32 * hh + j];
          obuf[(32 * hh + j) * 512 + d] = whole ? (l > 0.0f ? __uint_as_float(r[j]) / l : 0.0f) : __uint_as_float(r[j]);
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!*abort_flag) {
      if (whole) {
        uint4* op = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(row) * 64 * 512);
#pragma unroll 4
        for (int j = tid; j < 64 * 512 / 8; j += kPagedThreads) {
          const float4 a = reinterpret_cast<const float4*>(obuf)[2 * j];
          const float4 c = reinterpret_cast<const float4*>(obuf)[2 * j + 1];
          op[j] = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(c.x, c.y), pack_bf16x2(c.z, c.w));
        }
        if (p.lse && tid < 64) {
          const float l = sum_s[tid];
          p.lse[static_cast<int64_t>(row) * 64 + tid] = l > 0.0f ? (ref_s[tid] + log2f(l)) * 0.69314718055994531f : -INFINITY;
        }
      } else {
        float4* op = reinterpret_cast<float4*>(p.opart + static_cast<int64_t>(slot) * 64 * 512);
        const float4* src = reinterpret_cast<const float4*>(obuf);
#pragma unroll 4
        for (int j = tid; j < 64 * 512 / 4; j += kPagedThreads) op[j] = src[j];
        if (tid < 64) {
          p.ml[(slot * 64 + tid) * 2] = ref_s[tid];
          p.ml[(slot * 64 + tid) * 2 + 1] = sum_s[tid];
        }
      }
    }
    fence_async_smem();
    __syncthreads();
    at += t1 - t0;
    offset = 0;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) { tc_fence_after(); tmem_dealloc(tmem, 512); }
}

// Merge of the queries that range boundaries cut.  CTA column c looks at the
// boundary before CTA c of the attention: when that CTA's range begins
// inside a query and the one before it begins elsewhere, the query's
// partials are CTA c-1's last and the first ones of CTAs c, c+1, ... as long
// as they begin inside the same query.  One head per CTA, 4 dims per thread.
__global__ void __launch_bounds__(128)
paged_attn_join_kernel(PagedAttnParams p, int ctas) {
  pdl_launch_dependents();
  pdl_wait();
  const int h = blockIdx.x, c = blockIdx.y + 1, t = threadIdx.x;
  const int row = p.first_row[c];
  if (row < 0 || p.first_row[c - 1] == row) return;
  int last = c;
  while (last + 1 < ctas && p.first_row[last + 1] == row) ++last;
  const int first_slot = 2 * (c - 1) + 1;
  float M = p.ml[(first_slot * 64 + h) * 2];
  for (int k = c; k <= last; ++k) M = fmaxf(M, p.ml[(2 * k * 64 + h) * 2]);
  float L = 0.0f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (M != -INFINITY) {
    for (int k = c - 1; k <= last; ++k) {
      const int slot = k < c ? first_slot : 2 * k;
      const float m = p.ml[(slot * 64 + h) * 2];
      if (m == -INFINITY) continue;
      const float f = exp2f(m - M);
      const float4 o = __ldcg(reinterpret_cast<const float4*>(p.opart + (static_cast<int64_t>(slot) * 64 + h) * 512) + t);
      L += f * p.ml[(slot * 64 + h) * 2 + 1];
      acc.x += f * o.x; acc.y += f * o.y; acc.z += f * o.z; acc.w += f * o.w;
    }
  }
  const float inv = (L > 0.0f) ? 1.0f / L : 0.0f;
  uint2 packed;
  packed.x = pack_bf16x2(acc.x * inv, acc.y * inv);
  packed.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(row) * 64 + h) * 512 + 4 * t) = packed;
  if (p.lse && t == 0)
    p.lse[static_cast<int64_t>(row) * 64 + h] = (L > 0.0f) ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace csa2
