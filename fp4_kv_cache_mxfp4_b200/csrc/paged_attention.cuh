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
// earlier range) and its last (when that goes on).  Runs of one part of a query
// (kPagedRun) are merged in the same two places.
//
// Mathematics of a tile, as in attention_tc.cuh: S^T[key, head] = K . Q^T
// (tcgen05, M = 128 keys, N = 64 heads, K = 512 dims), weights
// P^T = exp2(S^T - ref) in bf16 against a running reference per head that
// moves only when a logit passes it by 2^8, O^T[dim, head] += V^T . P^T
// (M = 128 dims x 4, N = 64, K = 128 keys) with the same bf16 key tile read
// along its other axis.  The weights are the one thing rounded before the end:
// an MMA's operands have one type, and as TF32 keys and weights would take
// twice the shared memory and half the rate.  A weight is off by up to 2^-8 of itself,
// the output by 2.3e-3 of its norm at most (1.7e-3 for the bf16 result alone);
// the sums that divide it are of the unrounded weights, in float32.
//
// What bounds it: the data path of shared memory and L1.  A tile's 64 MMAs
// read 6 KB of operands each at 128 B per cycle, 48 cycles (measured; the MMA
// rate alone would allow 32), half of a tile; beside them the expanded keys are
// written (1024 cycles) and raw keys, weights and addresses pass, 3100
// load/store wavefronts per tile in all (counted; 1400 of them are not shared
// memory: scales read two bytes at a time, prefetches of rows).  One key tile (128 KB), Q
// (64 KB) and P^T (16 KB) fill the shared memory, so there is no second tile to work on while the
// softmax runs (some 1300 cycles, 512 of them the exponentials' rate); the
// tile is filled in slabs of 128 dims instead: MMA 2 releases slab t when its
// output rows t are done, and the next tile's slab t is expanded while MMA 2
// runs on the others.  Measured, a tile takes some 6000 cycles: MMA 2 2250,
// MMA 1 2450, softmax 1300.  Four sequences of 131,072 entries take 109 us (42 at
// the bf16 rate), one of 1,048,576 201 us (84), both with the join.
// Tried and slower: a second issuing warp for MMA 1 (its MMAs and MMA 2's
// then took 100 cycles each, 10 % in all), whole or half slabs expanded
// before the wait for their place (7 and 4 %), one lane or one warp polling
// for the others (11 and 1 %).  Roles:
//   warp 0       MMA issue (the scheduler prefers older warps: as the last warp
//                it lost hundreds of cycles per tile to the loaders)
//   warp 1       row addresses of the tiles to come (block table, window),
//                up to three tiles ahead, and their prefetch to L2
//   warps 2-3    Q (TMA, then the channel order below; warp 2 alone in bf16 pools)
//   warps 4-11   loaders: rows -> bf16 slabs (FP4 entries of the next tile
//                wait in registers; bf16 rows go by cp.async)
//   warps 12-27  softmax: S^T from tensor memory, weights to P^T, and the
//                epilogue; warp w has keys 32 (w % 4).. and heads 16 (w / 4 - 3)..
// Every role about fits in the 72 registers that 28 warps leave each thread (32
// bytes are spilled).  Spills in the loops cost (58 bytes: 11 %): with the whole
// shared memory taken, L1 is too small for spilled values to stay, and each
// reload then costs an L2 round trip.
//
// FP4 to bf16 in 9 logic, 4 multiply-add and 4 half-precision instructions
// per 8 channels (the ALU rate, half the FMA rate, is what bounds the
// loaders; a table look-up by byte permutes takes 26 logic ones and made the
// conversion of a tile 5600 cycles): the nibble pair (j, j + 4) of a word,
// times 2^12 + 2^6, has each sign at bit 15 and each magnitude at bits 6..8
// of its half, which read as bf16 is the value times 2^-126 (subnormals
// included, as in E2M1).  One multiplication by scale * 2^118 leaves the
// entry times 2^-8 (2^126 * 448 would overflow), exactly.  So in a pool of FP4 entries
//   - every 16-byte unit of an operand holds channels 0 4 1 5 2 6 3 7 of its
//     eight: Q and the window rows are permuted alike, and the epilogue
//     writes each dim to its channel;
//   - logits of cache tiles are multiplied by 2^8, weights of window keys by
//     2^-8 and the result by 2^8.
#pragma once
#include "common.cuh"
#include "quantize.cuh"
#include "attention_tc.cuh"
#include "paged_tables.cuh"
#include "topk.cuh"

namespace csa2 {

constexpr int kPagedLoaders = 8, kPagedSoftmax = 16, kPagedQWarps = 2;      // warps
constexpr int kPagedQWarp0 = 2, kPagedLoader0 = kPagedQWarp0 + kPagedQWarps, kPagedSoftmax0 = kPagedLoader0 + kPagedLoaders;
constexpr int kPagedThreads = 32 * (kPagedSoftmax0 + kPagedSoftmax);
static_assert(kPagedLoader0 % 4 == 0 && kPagedSoftmax0 % 4 == 0, "roles are whole warpgroups");
// Registers per thread: 72 at launch (896 threads); warps 0-3 hand some to the loaders: 256 x 88 + 128 x 40 = 384 x 72.
constexpr int kPagedLoaderRegs = 88, kPagedOtherRegs = 40;
static_assert(256 * kPagedLoaderRegs + 128 * kPagedOtherRegs <= 384 * 72, "register split");
constexpr int kPagedStages = 3;                        // tiles whose row addresses are kept
constexpr uint32_t kPagedPolls = 1u << 24;            // of a wait, before it gives up
constexpr int kPagedEndBar = 5;                         // named barriers: 1-4 the softmax quarters, 5 the end
// Minus the reference of a head that has none yet.  Finite: a logit of -inf
// (finite entries may reach it in float32) then has weight 0, where -inf + inf
// would be NaN; any other logit passes it and moves the reference.
constexpr float kPagedNoRef = 3.0e38f;
constexpr float kPagedFp4Up = 256.0f, kPagedFp4Down = 0.00390625f;
constexpr int kPagedKeys = 128;                        // keys per tile (MMA M)
// Tiles summed in tensor memory.  The tensor core drops what of a product lies
// below the last bit of its accumulator, and the loss grows with the keys
// that one accumulator takes: with keys of one sign, 5e-4 of the output after
// 131,072 keys, 6e-3 after 1,048,576, half after 2^27.  So a longer part is summed in
// runs of so many tiles (2e-4 at any length, measured; the bf16 weights are
// off by up to 2^-8 each), merged in float32 in the CTA's own partial slot.
// 148 requests of 1,048,576 entries take 25.1 ms with and without.
constexpr int kPagedRun = 256;
constexpr int kPagedMaxCtas = 148;                     // one per SM of a B200
constexpr uint32_t kPagedSmem = kTcAttnSmem;

struct PagedAttnParams {
  int BQ, Q, W;
  int w_tiles;               // ceil(W / 128)
  uint32_t block_size, max_blocks;
  DivBy by_block;
  int64_t ld_table, n_blocks, block_stride;            // block_stride in bytes
  const uint8_t* kv;
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
  int2* cut;                 // [CTAs]: (query, partials) where a CTA's range is the first to begin inside a query, else (-1, 0)
};

// Tiles of query r: at least one, so that a query without any key is written too.
__device__ __forceinline__ int paged_tiles(const PagedAttnParams& p, int r, int* keys) {
  // max_blocks * block_size <= 2^30
  *keys = min(max(p.n_vis[r], 0), static_cast<int>(p.max_blocks * p.block_size));
  return max((*keys + kPagedKeys - 1) / kPagedKeys + p.w_tiles, 1);
}

// This CTA's tile range [lo, hi) of the total, the query that lo lies in and
// lo's offset inside it.  Every CTA sums the tiles of all queries (4 bytes
// each from L2); every thread calls it.
struct PagedRange { int64_t lo, hi; int row, offset, parts; };   // parts: partials of the query, as in cut[]
__device__ __forceinline__ PagedRange paged_range(const PagedAttnParams& p, int64_t* warp_s, PagedRange* range_s) {
  const int per = (p.BQ + blockDim.x - 1) / blockDim.x;
  const int r0 = min(p.BQ, static_cast<int>(threadIdx.x) * per), r1 = min(p.BQ, r0 + per);
  int64_t mine = 0, total = 0;
  int keys;
  for (int r = r0; r < r1; ++r) mine += paged_tiles(p, r, &keys);
  int64_t at = block_exclusive_sum(mine, warp_s, &total);
  // no CTA without a tile between two that have one (the join looks at neighbours)
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);
  if (blockIdx.x >= ctas) return PagedRange{0, 0, 0, 0, 0};
  const int64_t lo = total * blockIdx.x / ctas, hi = total * (blockIdx.x + 1) / ctas;
  if (lo >= at && lo < at + mine) {
    for (int r = r0; r < r1; ++r) {
      const int t = paged_tiles(p, r, &keys);
      if (lo < at + t) {
        // tile x lies in the range of CTA ((x + 1) ctas - 1) / total
        const int first = static_cast<int>(((at + 1) * ctas - 1) / total);
        const int last = static_cast<int>(((at + t) * ctas - 1) / total);
        const bool cuts = lo > at && static_cast<int>(blockIdx.x) == first + 1;
        *range_s = PagedRange{lo, hi, r, static_cast<int>(lo - at), cuts ? last - first + 1 : 0};
        break;
      }
      at += t;
    }
  }
  __syncthreads();
  return *range_s;
}

// Walks the tiles of a CTA's range: runs [t, t1) of query `row`'s tiles, then the next query's.
struct PagedCursor {
  uint32_t left;             // tiles of the range from tile t on (below 2^32 / 148 queries' worth each)
  int t, t1;                 // this tile, the end of its run
  int row, keys, kv_tiles;
};
// The query's tiles.
__device__ __forceinline__ int paged_all(const PagedAttnParams& p, const PagedCursor& c) { return max(c.kv_tiles + p.w_tiles, 1); }
__device__ __forceinline__ void paged_run(const PagedAttnParams& p, PagedCursor& c) {
  c.t1 = min(paged_all(p, c), c.t + static_cast<int>(min(c.left, static_cast<uint32_t>(kPagedRun))));
}
// At a run's last tile: is it the last of the range's part of the query?
__device__ __forceinline__ bool paged_part_ends(const PagedAttnParams& p, const PagedCursor& c) {
  return c.left == 1 || c.t1 == paged_all(p, c);
}
__device__ __forceinline__ void paged_enter(const PagedAttnParams& p, PagedCursor& c, int row, int offset) {
  c.row = row;
  paged_tiles(p, row, &c.keys);
  c.kv_tiles = (c.keys + kPagedKeys - 1) / kPagedKeys;
  c.t = offset;
  paged_run(p, c);
}
// The cursor at the range's first tile.
__device__ __forceinline__ PagedCursor paged_begin(const PagedAttnParams& p, const volatile PagedRange* r) {
  PagedCursor c;
  c.left = static_cast<uint32_t>(r->hi - r->lo);
  paged_enter(p, c, r->row, r->offset);
  return c;
}
// To the next tile; false behind the last.
__device__ __forceinline__ bool paged_next(const PagedAttnParams& p, PagedCursor& c) {
  if (--c.left == 0) return false;
  if (++c.t == c.t1) {
    if (c.t == paged_all(p, c)) paged_enter(p, c, c.row + 1, 0);
    else paged_run(p, c);
  }
  return true;
}

// Address of entry `pos` of a request's cache; nullptr where the table names no block of the pool.
__device__ __forceinline__ const uint8_t* paged_row(const PagedAttnParams& p, const int32_t* table, uint32_t pos,
                                                    uint32_t row_bytes) {
  const uint32_t blk = p.by_block(pos);
  const int32_t id = table[blk];
  if (id < 0 || id >= p.n_blocks) return nullptr;
  return p.kv + id * p.block_stride + static_cast<int64_t>(pos - blk * p.block_size) * row_bytes;
}

// Wait of a whole warp.  Every lane polls: with one lane polling for the
// others, the warp could go on in two parts, and what all lanes must execute
// together (tcgen05, named barriers) then happened twice.
__device__ __forceinline__ bool paged_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool paged_wait(uint32_t bar, uint32_t parity, int err, volatile int* abort) {
  if (__all_sync(0xffffffffu, paged_try_wait(bar, parity))) return true;
  // bounded by polls, which take some 140 cycles each: a second or two
#pragma unroll 1
  for (uint32_t n = 0; n < kPagedPolls && !*abort; ++n)
    if (__all_sync(0xffffffffu, paged_try_wait(bar, parity))) return true;
  __syncwarp();
  if (!*abort) {
    record_error(err);
    *abort = 1;
  }
  __syncwarp();
  return false;
}
// For warps that end where a wait fails and owe nothing to others then.  By an
// instruction, not a branch out of the role's loop, which made a tile 2 % slower
// (148 requests of 1,048,576 entries: 25.7 against 25.1 ms).
__device__ __forceinline__ void paged_wait_or_exit(uint32_t bar, uint32_t parity, int err, volatile int* abort) {
  if (!paged_wait(bar, parity, err, abort)) asm volatile("exit;" ::: "memory");
}
// Before a role ends: waits, with the same limit whatever gave up before, for its own copy or MMAs.
__device__ __forceinline__ void paged_drain(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (uint32_t n = 0; n < kPagedPolls; ++n)
    if (__all_sync(0xffffffffu, paged_try_wait(bar, parity))) return;
}
__device__ __forceinline__ void paged_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" :: "r"(bar) : "memory");
  __syncwarp();
}
__device__ __forceinline__ void paged_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void paged_bar(int id, int nthreads) {
  __syncwarp();
  named_bar_sync(id, nthreads);
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      :: "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
         "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
template <int N>
__device__ __forceinline__ void regs_up() { __syncwarp(); asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { __syncwarp(); asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N)); }
__device__ __forceinline__ void sts(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void sts(uint32_t a, float v) { asm volatile("st.shared.f32 [%0], %1;" :: "r"(a), "f"(v) : "memory"); }
__device__ __forceinline__ void sts(uint32_t a, int v) { asm volatile("st.shared.b32 [%0], %1;" :: "r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ void sts(uint32_t a, const uint8_t* v) { asm volatile("st.shared.b64 [%0], %1;" :: "r"(a), "l"(v) : "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float lds_f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ int lds_i(uint32_t a) {
  int v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ const uint8_t* lds_ptr(uint32_t a) {
  const uint8_t* v;
  asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
// Wait for the end of a query's part, which may be millions of tiles: it
// gives up only when, for as many polls, no tile's addresses were written either.
__device__ __forceinline__ bool paged_wait_part(uint32_t bar, uint32_t parity, uint32_t progress, int err, volatile int* abort) {
  int seen = -1;
  while (true) {
#pragma unroll 1
    for (uint32_t n = 0; n < kPagedPolls && !*abort; ++n)
      if (__all_sync(0xffffffffu, paged_try_wait(bar, parity))) return true;
    const int now = __shfl_sync(0xffffffffu, lds_i(progress), 0);
    if (now == seen || __any_sync(0xffffffffu, *abort)) break;
    seen = now;
  }
  if (!*abort) {
    record_error(err);
    *abort = 1;
  }
  __syncwarp();
  return false;
}
// (volatile: stays before the barrier that it is meant to hide)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Waits for tensor-memory loads; naming the registers keeps their uses behind it.
__device__ __forceinline__ void paged_ld_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]) :: "memory");
}
__device__ __forceinline__ void tmem_ld_32x32b_x4(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(taddr) : "memory");
}
__device__ __forceinline__ void paged_ld_wait(uint32_t (&r)[4]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]) :: "memory");
}
// umma_bf16 with the descriptors' high words apart: only the low ones (the
// addresses) change from one MMA to the next.
__device__ __forceinline__ void paged_mma(uint32_t tmem_d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}"
      :: "r"(tmem_d), "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate) : "memory");
}
// True in one lane of a converged warp; which one is the hardware's choice.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  __syncwarp();
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// Barrier `id` over n threads that also ORs a predicate over them.
__device__ __forceinline__ bool named_bar_or(int id, int n, bool pred) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r) : "r"(id), "r"(n), "r"(static_cast<uint32_t>(pred)) : "memory");
  return r != 0;
}

// Eight natural-order bf16 channels to the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ uint4 paged_order(uint4 v) {
  return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                    __byte_perm(v.y, v.w, 0x7632));
}
// Channel (0..7) of position i of such a unit.
__device__ __forceinline__ int paged_channel(int i) { return (i >> 1) + 4 * (i & 1); }

// Two E4M3 scale codes (bytes 0, 1 of w) to bf16, times 2^118: bits of an
// E4M3 code at the bottom of a bf16 read as its value times 2^-120.
__device__ __forceinline__ __nv_bfloat162 paged_scales(uint32_t w) {
  const uint32_t a = __byte_perm(w, 0u, 0x4140);
  const uint32_t m = ((a & 0x007F007Fu) << 4) | ((a & 0x00800080u) << 8);
  const __nv_bfloat162 up1 = __floats2bfloat162_rn(1.329227995784916e36f, 1.329227995784916e36f);   // 2^120
  const __nv_bfloat162 up2 = __floats2bfloat162_rn(3.323069989462290e35f, 3.323069989462290e35f);   // 2^118
  return __hmul2(__hmul2(*reinterpret_cast<const __nv_bfloat162*>(&m), up1), up2);
}
// Eight E2M1 codes to the unit's eight bf16 values (order as above), times scale * 2^-126.
__device__ __forceinline__ uint4 paged_expand8(uint32_t w, __nv_bfloat162 scale) {
  const uint32_t h = w >> 8;
  uint32_t o[4] = {(w & 0x000F000Fu) * 0x1040u, (w & 0x00F000F0u) * 0x0104u, (h & 0x000F000Fu) * 0x1040u,
                   (h & 0x00F000F0u) * 0x0104u};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    o[j] &= 0x81C081C0u;
    const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&o[j]), scale);
    o[j] = *reinterpret_cast<const uint32_t*>(&x);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

constexpr int kPagedPool = 0, kPagedBf16 = 1, kPagedFp8 = 2;       // kinds of tiles: cache entries, window rows

// Loader threads and keys (w counts the loader warps).  Warps 0-3 fill slabs
// 0 and 2, warps 4-7 slabs 1 and 3: two slabs in work at a time, so that one's expansion covers the
// other's stores and hand-over.  FP4 entries: keys 32 (w % 4) + 8 i + kk
// (i = 0..3) with kk from lane bits 1, 2 and 4 and the 16-byte unit of a
// 64-byte slab piece from bits 0 and 3, so that 8 lanes of a store phase hit
// 8 different bank groups of the swizzled tile and every global sector is
// used whole.  bf16 and FP8 rows: keys 32 (w % 4) + 4 i + lane / 8
// (i = 0..7), unit lane % 8.

template <bool KVB>
__global__ void __launch_bounds__(kPagedThreads, 1)
paged_attn_kernel(const __grid_constant__ CUtensorMap tmap_q, PagedAttnParams p) {
  extern __shared__ __align__(1024) uint8_t paged_smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(paged_smem_raw) + 1023) & ~uintptr_t(1023));
  // The tiles and what is read per tile go by 32-bit shared addresses: the
  // pointers below are generic (twice the registers, and slower accesses).
  const uint32_t kt = smem_u32(smem);                   // key tile: 8 chunks of [128 keys][64 dims], 2 per slab
  const uint32_t qt = kt + kTcKeyTileBytes;
  const uint32_t pt = qt + kTcQTileBytes;
  const uint32_t misc32 = pt + kTcPTileBytes;
  uint8_t* misc = smem + kTcKeyTileBytes + kTcQTileBytes + kTcPTileBytes;
  const uint32_t full = misc32;                         // [4] slab filled (4 loader warps)
  const uint32_t freed = misc32 + 32;                   // [4] slab read by MMA 2
  const uint32_t q_full = misc32 + 64;
  const uint32_t s_full = misc32 + 72;                  // MMA 1 done (and every MMA before it)
  const uint32_t p_full = misc32 + 80;                  // P^T written, O^T rescaled (16 softmax warps)
  const uint32_t o_full = misc32 + 88;                  // the run's last MMA 2 done
  const uint32_t q_tma = misc32 + 96;                   // Q arrived, in natural order (FP4 pools)
  const uint32_t q_free = misc32 + 104;                 // the query part's last MMA 1 done
  const uint32_t rows_full = misc32 + 112;              // [3] row addresses written
  const uint32_t rows_free = misc32 + 136;              // [3] ... and read (16 softmax warps)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 160);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 164);
  const uint32_t tiles_s = misc32 + 168;                              // int: tiles whose addresses were written
  const uint32_t all_done = misc32 + 192;               // after a wait gave up: every MMA done
  const uint32_t kind_s = misc32 + 176;                               // int [3]
  float* red_s = reinterpret_cast<float*>(misc + 256);                // [4 quarters][64 heads]
  const uint32_t nref_s = misc32 + 1280;                              // float [64] minus the reference
  const uint32_t fac_s = misc32 + 1536;                               // float [64] rescale factor, later 1 / sum
  int64_t* warp_s = reinterpret_cast<int64_t*>(misc + 1792);          // [33]
  PagedRange* range_s = reinterpret_cast<PagedRange*>(misc + 2064);
  const uint32_t row_s = misc32 + 2304;                               // [3][128] row address, null: no such key
  const uint32_t wsc_s = misc32 + 5376;                               // float [3][128] FP8 row scales
  const uint32_t ref0_s = misc32 + 6912;                              // float [64] reference of the part's earlier runs
  const uint32_t sum0_s = misc32 + 7168;                              // float [64] ... their sum
  const uint32_t fac0_s = misc32 + 7424;                              // float [64] ... and their factor in the merge

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 32) {
    uint64_t* bars = reinterpret_cast<uint64_t*>(misc);  // in the order above
    for (int i = 0; i < 20; ++i)
      mbar_init(bars + i, i < 4 ? kPagedLoaders / 2 : i == 8 ? (KVB ? 1 : kPagedQWarps) : i == 10 || i >= 17 ? kPagedSoftmax : 1);
    mbar_init(bars + 24, 1);                            // all_done
    *abort_flag = 0;
    sts(tiles_s, 0);
    fence_barrier_init();
    tma_prefetch_desc(&tmap_q);
  }
  if (warp == 0) { tmem_alloc(tmem_slot, 512); tmem_relinquish(); }
  pdl_launch_dependents();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (read by asm: only asm writes it, which a plain load might not be told)
  const uint32_t tmem = lds_i(misc32 + 160);
  const PagedRange range = paged_range(p, warp_s, range_s);
  if (tid == 0) p.cut[blockIdx.x] = range.parts > 0 ? make_int2(range.row, range.parts) : make_int2(-1, 0);

  // Every role walks the same tiles.  Waits are bounded; after one gave up
  // the others return at once.  The MMA warp and the softmax warps, which share
  // named barriers, then walk to their end and leave NaN for every query that
  // was not finished, in partials too (the join runs all the same); the row
  // addresses and the loaders stop, so that no address is followed that
  // was not written for its tile.
  if (range.lo < range.hi) {
    if (warp < kPagedLoader0) {
      regs_down<kPagedOtherRegs>();
      PagedCursor c = paged_begin(p, range_s);
      if (warp == 0) {
        // ---------------------------------------------------------- MMA
        // The whole warp walks along and one elected lane issues: the
        // descriptors then live in uniform registers, and an MMA costs a few
        // issue slots among busy warps.
        const bool issuer = elect_one();
        uint32_t ph_q = 0;
        bool first = true, fresh = true;                // of a run, of a query's part
        // descriptors of the tiles' first bytes; an offset adds to the 16-byte address field
        const uint64_t kd = umma_desc_sw128_kmajor(kt), qd = umma_desc_sw128_kmajor(qt);
        const uint64_t vd = umma_desc_sw128_mnmajor(kt, 16384), pd = umma_desc_sw128_mnmajor(pt, 16384);
        constexpr uint32_t idesc1 = umma_idesc_bf16_f32(128, 64);
        constexpr uint32_t idesc2 = umma_idesc_bf16_f32(128, 64) | (1u << 15) | (1u << 16);   // both MN-major
        // The walk to the next tile is done while the softmax runs: between MMA 2
        // and the next MMA 1 every instruction costs (28 warps share the
        // instruction cache).
        bool last = c.t + 1 == c.t1, ends = last && paged_part_ends(p, c);
        for (uint32_t ph = 0;; ph ^= 1) {
          bool ok = true;
          if (fresh) {
            ok = paged_wait(q_full, ph_q, kErrWaitOperand, abort_flag);
            ph_q ^= 1;
          }
          uint32_t da = static_cast<uint32_t>(kd), db = static_cast<uint32_t>(qd);
#pragma unroll 1
          for (int t = 0; t < 4; ++t) {
            ok = paged_wait(full + 8 * t, ph, kErrWaitTmaFull, abort_flag) && ok;
            tc_fence_after();
            if (ok && issuer) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                paged_mma(tmem, da + ((kk >> 2) * 16384 + (kk & 3) * 32 >> 4), kd >> 32,
                          db + ((kk >> 2) * 8192 + (kk & 3) * 32 >> 4), qd >> 32, idesc1, (t > 0 || kk > 0) ? 1u : 0u);
            }
            __syncwarp();
            da += 2 * 16384 >> 4;
            db += 2 * 8192 >> 4;
          }
          if (issuer) {
            paged_commit(s_full);
            if (ends) paged_commit(q_free);
          }
          __syncwarp();
          const bool more = paged_next(p, c), next_last = c.t + 1 == c.t1, next_ends = next_last && paged_part_ends(p, c);
          ok = paged_wait(p_full, ph, kErrWaitOperand, abort_flag) && ok;
          tc_fence_after();
          da = static_cast<uint32_t>(vd);
#pragma unroll 1
          for (int t = 0; t < 4; ++t) {
            if (ok && issuer) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                paged_mma(tmem + 64 + 64 * t, da + (kk * 2048 >> 4), vd >> 32, static_cast<uint32_t>(pd) + (kk * 2048 >> 4), pd >> 32,
                          idesc2, (!first || kk > 0) ? 1u : 0u);
            }
            if (issuer) paged_commit(freed + 8 * t);
            __syncwarp();
            da += 2 * 16384 >> 4;
          }
          if (issuer && last) paged_commit(o_full);
          __syncwarp();
          if (!more) break;
          first = last;
          fresh = ends;
          last = next_last;
          ends = next_ends;
        }
        paged_bar(kPagedEndBar, 32 * (kPagedSoftmax + 1));
        if (__any_sync(0xffffffffu, *abort_flag)) {
          if (issuer) paged_commit(all_done);
          paged_drain(all_done, 0);
        }
        tc_fence_after();
        tmem_dealloc(lds_i(misc32 + 160), 512);
      } else if (warp == 1) {
        // ---------------------------------------------------------- row addresses, 4 keys per lane
        int stage = 0, tiles = 0;
        uint32_t ph = 1;
        while (true) {
          // (after any wait gave up, rows_free no longer says that the loaders are through)
          if (!paged_wait(rows_free + 8 * stage, ph, kErrWaitSmemEmpty, abort_flag) || __any_sync(0xffffffffu, *abort_flag)) break;
          const bool window = c.t >= c.kv_tiles;
          const int b = c.row / p.Q;
          const int key0 = (window ? c.t - c.kv_tiles : c.t) * kPagedKeys + lane;
          const int bytes = window ? (p.swa_fp8 ? 512 : 1024) : (KVB ? 1024 : 288);
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
            const int key = key0 + 32 * i;
            const uint8_t* row = nullptr;
            if (window) {
              const int64_t r = static_cast<int64_t>(b) * p.swa_rows + static_cast<int64_t>(c.row - b * p.Q) * p.swa_step + key;
              if (key < p.W) row = p.swa + r * bytes;
              // (of absent keys too: their weight of 0 is multiplied by it)
              if (p.swa_fp8) sts(wsc_s + 4 * (stage * 128 + lane + 32 * i), row ? p.swa_scale[r] : 0.0f);
            } else if (key < c.keys) {
              row = paged_row(p, p.table + b * p.ld_table, static_cast<uint32_t>(key), bytes);
            }
            sts(row_s + 8 * (stage * 128 + lane + 32 * i), row);
            if (row)
              for (int o = 0; o < bytes; o += 128) prefetch_l2(row + o);
          }
          if (lane == 0) {
            sts(kind_s + 4 * stage, window ? (p.swa_fp8 ? kPagedFp8 : kPagedBf16) : kPagedPool);
            sts(tiles_s, ++tiles);
          }
          paged_arrive(rows_full + 8 * stage);
          if (!paged_next(p, c)) break;
          if (++stage == kPagedStages) { stage = 0; ph ^= 1; }
        }
      } else if (!KVB || warp == kPagedQWarp0) {
        // ---------------------------------------------------------- Q
        // (bf16 pools: the copy alone, one warp.  A warp whose work no one waits
        // for could fall a phase behind on q_free.)
        const int qtid = tid - 32 * kPagedQWarp0;
        uint32_t sent = 0;                              // copies, one per part
        while (true) {
          if (!paged_wait_part(q_free, (sent & 1) ^ 1, tiles_s, kErrWaitOperand, abort_flag)) break;
          if (qtid == 0) {
            uint64_t* arrived = reinterpret_cast<uint64_t*>(misc + (KVB ? 64 : 96));   // q_full or q_tma
            mbar_arrive_expect_tx(arrived, kTcQTileBytes);
            const uint64_t pol = l2_policy_evict_first();
            for (int k = 0; k < 8; ++k) tma_load_2d(smem + kTcKeyTileBytes + k * 8192, &tmap_q, arrived, 64 * k, c.row * 64, pol);
          }
          ++sent;
          if (!KVB) {
            if (!paged_wait(q_tma, (sent & 1) ^ 1, kErrWaitOperand, abort_flag)) break;
            for (int i = qtid; i < static_cast<int>(kTcQTileBytes / 16); i += 4 * 32 * kPagedQWarps) {
              uint4 v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int j = i + k * 32 * kPagedQWarps;
                if (j < static_cast<int>(kTcQTileBytes / 16)) v[k] = lds128(qt + 16 * j);
              }
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int j = i + k * 32 * kPagedQWarps;
                if (j < static_cast<int>(kTcQTileBytes / 16)) sts(qt + 16 * j, paged_order(v[k]));
              }
            }
            fence_async_smem();
            paged_arrive(q_full);
          }
          c.left -= min(c.left, static_cast<uint32_t>(paged_all(p, c) - c.t));
          if (c.left == 0) break;
          paged_enter(p, c, c.row + 1, 0);
        }
        if (sent > 0) paged_drain(KVB ? q_full : q_tma, (sent & 1) ^ 1);
      }
    } else if (warp < kPagedSoftmax0) {
      // ------------------------------------------------------------ loaders
      regs_up<kPagedLoaderRegs>();
      uint32_t left = static_cast<uint32_t>(range_s->hi - range_s->lo);
      const int kk = ((lane >> 1) & 3) | ((lane >> 2) & 4), u = (lane & 1) | ((lane >> 2) & 2);
      const int key0 = 32 * (warp & 3), t0 = (warp - kPagedLoader0) >> 2;  // first key; slabs t0, t0 + 2
      uint4 raw[2][4];                                  // FP4: [slab][key] 32 channels ...
      uint16_t rsc[2][4];                               // ... and their two scales
      int kind;
      auto fetch = [&](int stage) {                     // the tile's kind and, of cache entries, their bytes
        kind = lds_i(kind_s + 4 * stage);
        if (!KVB && kind == kPagedPool) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint8_t* row = lds_ptr(row_s + 8 * (stage * 128 + key0 + 8 * i + kk));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int t = t0 + 2 * k;
              raw[k][i] = make_uint4(0, 0, 0, 0);
              rsc[k][i] = 0;
              if (row) {
                raw[k][i] = __ldg(reinterpret_cast<const uint4*>(row + 64 * t + 16 * u));
                rsc[k][i] = __ldg(reinterpret_cast<const uint16_t*>(row + 256 + 8 * t + 2 * u));
              }
            }
          }
        }
      };
      auto publish = [&](int t) {
        fence_async_smem();
        paged_arrive(full + 8 * t);
      };
      int stage = 0;
      uint32_t ph_rows = 0;
      // Addresses are followed only if they were written.
      paged_wait_or_exit(rows_full + 8 * 0, 0, kErrWaitOperand, abort_flag);
      fetch(0);
      for (uint32_t ph = 1;; ph ^= 1) {                 // ph: MMA 2 of the tile before has released the slab
        if (!KVB && kind == kPagedPool) {
          // (rolled: the kernel's hot code should stay in the instruction cache)
          uint32_t chunk = kt + (2 * t0 + (u >> 1)) * 16384 + sw128_off(key0 + kk, 4 * (u & 1));
#pragma unroll 1
          for (int t = t0; t < 4; t += 2) {
            paged_wait(freed + 8 * t, ph, kErrWaitSmemEmpty, abort_flag);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 sc = paged_scales(rsc[0][i]);
              const __nv_bfloat162 s0 = __low2bfloat162(sc), s1 = __high2bfloat162(sc);
              const uint32_t w[4] = {raw[0][i].x, raw[0][i].y, raw[0][i].z, raw[0][i].w};
              // unit q of the row: the swizzle XORs bits 4, 5 of the address
#pragma unroll
              for (int q = 0; q < 4; ++q) sts((chunk ^ (16 * q)) + 1024 * i, paged_expand8(w[q], q < 2 ? s0 : s1));
            }
            publish(t);
            chunk += 4 * 16384;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              raw[0][i] = raw[1][i];
              rsc[0][i] = rsc[1][i];
            }
          }
        } else if (KVB && kind == kPagedPool) {
          const uint8_t* row[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) row[i] = lds_ptr(row_s + 8 * (stage * 128 + key0 + 4 * i + (lane >> 3)));
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = t0 + 2 * k;
            paged_wait(freed + 8 * t, ph, kErrWaitSmemEmpty, abort_flag);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint8_t* src = row[i] ? row[i] + 256 * t + 16 * (lane & 7) : p.kv;
#pragma unroll
              for (int h = 0; h < 2; ++h)
                cp_async16(kt + (2 * t + h) * 16384 + sw128_off(key0 + 4 * i + (lane >> 3), lane & 7),
                           src + (row[i] ? 128 * h : 0), row[i] != nullptr);
            }
            cp_async_commit();
          }
          cp_async_wait<1>();
          publish(t0);
          cp_async_wait<0>();
          publish(t0 + 2);
        } else {
          // window rows, in the pool's channel order, four keys of a thread at
          // a time, the first four read before the wait for the slab (in the registers of
          // the FP4 bytes, which are then known to be dead: others cost spills)
          const bool fp8 = kind == kPagedFp8;
#pragma unroll 1
          for (int t = t0; t < 4; t += 2) {
#pragma unroll 1
            for (int i = 0; i < 8; i += 4) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint8_t* row = lds_ptr(row_s + 8 * (stage * 128 + key0 + 4 * (i + k) + (lane >> 3)));
                raw[0][k] = raw[1][k] = make_uint4(0, 0, 0, 0);
                if (row) {
                  const uint4* src = reinterpret_cast<const uint4*>(row + (fp8 ? 128 : 256) * t) + (lane & 7);
                  raw[0][k] = __ldg(src);
                  if (!fp8) raw[1][k] = __ldg(src + 8);
                }
              }
              if (i == 0) paged_wait(freed + 8 * t, ph, kErrWaitSmemEmpty, abort_flag);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int r = key0 + 4 * (i + k) + (lane >> 3);
                uint4 lo = raw[0][k], hi = raw[1][k];
                uint32_t at = 2 * t * 16384 + sw128_off(r, lane & 7), at2 = at + 16384;
                if (fp8) {
                  e4m3x4_to_bf16(raw[0][k].x, lo.x, lo.y);
                  e4m3x4_to_bf16(raw[0][k].y, lo.z, lo.w);
                  e4m3x4_to_bf16(raw[0][k].z, hi.x, hi.y);
                  e4m3x4_to_bf16(raw[0][k].w, hi.z, hi.w);
                  const uint32_t chunk = (2 * t + ((lane >> 2) & 1)) * 16384;
                  at = chunk + sw128_off(r, 2 * (lane & 3));
                  at2 = chunk + sw128_off(r, 2 * (lane & 3) + 1);
                }
                sts(kt + at, KVB ? lo : paged_order(lo));
                sts(kt + at2, KVB ? hi : paged_order(hi));
              }
            }
            publish(t);
          }
        }
        if (--left == 0) break;
        if (++stage == kPagedStages) { stage = 0; ph_rows ^= 1; }
        paged_wait_or_exit(rows_full + 8 * stage, ph_rows, kErrWaitOperand, abort_flag);
        fetch(stage);                                   // behind the tile's last fence, which would wait for the loads
      }
    } else {
      // ------------------------------------------------------------ softmax
      PagedCursor c = paged_begin(p, range_s);
      const int quarter = warp & 3, hg = (warp - kPagedSoftmax0) >> 2, bar = 1 + hg;
      const int key = 32 * quarter + lane, head0 = 16 * hg;
      const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
      uint32_t ph_o = 0;
      int stage = 0;
      float sum[16];                                    // this key's weights, summed over the tiles, per head
      bool first = true, merge = false, part_begins = false;     // merge: the part has earlier runs
      for (uint32_t it = 0;; ++it) {
        if (first) {
          if (!merge) part_begins = c.t == 0;
          if (quarter == 0 && lane < 16) sts(nref_s + 4 * (head0 + lane), kPagedNoRef);
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[j] = 0.0f;
          paged_bar(bar, 128);
        }
        const bool window = c.t >= c.kv_tiles;
        paged_wait(full + 8 * 0, it & 1, kErrWaitSmemEmpty, abort_flag);      // a loader has seen the tile's addresses
        const bool there = lds_ptr(row_s + 8 * (stage * 128 + key)) != nullptr;
        float rs = (window && p.swa_fp8) ? lds_f(wsc_s + 4 * (stage * 128 + key)) : 1.0f;
        const float ls = p.scale_log2 * (KVB || window ? rs : kPagedFp4Up);
        if (!KVB && window) rs *= kPagedFp4Down;
        paged_wait(s_full, it & 1, kErrWaitTmemFull, abort_flag);
        tc_fence_after();
        // y = exp2(logit - reference) in log2 units.  The weights go to P^T before
        // the vote on whether some reference must move (then they are made again),
        // and into the sums after the hand-over: both off the path from S^T to MMA 2.
        float y[16];
        float over = -INFINITY;
        auto weights = [&]() {
          uint32_t r[16];
          tmem_ld_32x32b_x16(tmem + lanes + head0, r);
          float4 nr[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) nr[j] = lds_f4(nref_s + 4 * (head0 + 4 * j));
          paged_ld_wait(r);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            y[j] = fmaf(__uint_as_float(r[j]), ls, nr[j / 4].x);
            y[j + 1] = fmaf(__uint_as_float(r[j + 1]), ls, nr[j / 4].y);
            y[j + 2] = fmaf(__uint_as_float(r[j + 2]), ls, nr[j / 4].z);
            y[j + 3] = fmaf(__uint_as_float(r[j + 3]), ls, nr[j / 4].w);
          }
          if (!__all_sync(0xffffffffu, there)) {
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = there ? y[j] : -INFINITY;
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t pk[4];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              const int i = 8 * q + j;
              over = fmaxf(over, fmaxf(y[i], y[i + 1]));
              y[i] = ex2(y[i]);
              y[i + 1] = ex2(y[i + 1]);
              // an FP8 window key's row scale goes into the weight that multiplies its codes
              pk[j / 2] = window ? pack_bf16x2(y[i] * rs, y[i + 1] * rs) : pack_bf16x2(y[i], y[i + 1]);
            }
            sts(pt + sw128_off(key, 2 * hg + q), make_uint4(pk[0], pk[1], pk[2], pk[3]));
          }
          fence_async_smem();
        };
        weights();
        if (named_bar_or(bar, 128, over > kTcRefSlack)) {
          // some reference moves: the tile's maximum per head, over the lanes and the four quarters
          {
            float v[16];
            uint32_t r[16];
            tmem_ld_32x32b_x16(tmem + lanes + head0, r);
            paged_ld_wait(r);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = there ? __uint_as_float(r[j]) * ls : -INFINITY;
            const float m = warp_reduce_heads16<true>(v, lane);
            if ((lane & 1) == 0) red_s[quarter * 64 + head0 + (lane >> 1)] = m;
          }
          paged_bar(bar, 128);
          if (quarter == 0) {                           // every lane, so that the warp stays together; 16 write
            const int h = head0 + (lane & 15);
            const float mt = fmaxf(fmaxf(red_s[h], red_s[64 + h]), fmaxf(red_s[128 + h], red_s[192 + h]));
            const float ref = -lds_f(nref_s + 4 * h);
            const bool move = mt > ref + kTcRefSlack;
            const float f = ex2(ref - mt), fac = move ? f : 1.0f;
            __syncwarp();
            if (lane < 16) {
              sts(fac_s + 4 * h, fac);
              sts(nref_s + 4 * h, move ? -mt : -ref);
            }
          }
          paged_bar(bar, 128);
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[j] *= lds_f(fac_s + 4 * (head0 + j));
          if (!first) {
            // earlier tiles are in the accumulator, and their MMAs are done (s_full)
#pragma unroll 1
            for (int t = 0; t < 4; ++t) {
              uint32_t r[16];
              const uint32_t ta = tmem + lanes + 64 + 64 * t + head0;
              tmem_ld_32x32b_x16(ta, r);
              paged_ld_wait(r);
#pragma unroll
              for (int j = 0; j < 16; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * lds_f(fac_s + 4 * (head0 + j)));
              tmem_st_32x32b_x16(ta, r);
              tmem_st_wait();
            }
          }
          weights();
        }
        tc_fence_before();
        paged_arrive(p_full);
        // (the loaders are through with the addresses too; a tcgen05.commit for
        // this would hold the MMA warp up until its queue has drained)
        paged_arrive(rows_free + 8 * stage);
        if (++stage == kPagedStages) stage = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) sum[j] += y[j];    // unrounded: the log-sum-exp keeps float32
        first = false;

        if (c.t + 1 == c.t1) {
          // -------------------------------------- the run is complete
          const int row = c.row;
          const bool ends = paged_part_ends(p, c), whole = part_begins && c.t1 == paged_all(p, c);
          const int slot = 2 * blockIdx.x + (part_begins ? 1 : 0);
          {
            const float l = warp_reduce_heads16<false>(sum, lane);
            if ((lane & 1) == 0) red_s[quarter * 64 + head0 + (lane >> 1)] = l;
          }
          paged_bar(bar, 128);
          if (quarter == 0) {
            const int h = head0 + (lane & 15);
            float l = (red_s[h] + red_s[64 + h]) + (red_s[128 + h] + red_s[192 + h]);
            float ref = -lds_f(nref_s + 4 * h), f = KVB ? 1.0f : kPagedFp4Up, f0 = 0.0f;
            if (merge) {
              const float ref0 = lds_f(ref0_s + 4 * h), top = fmaxf(ref0, ref);
              f0 = ref0 == top ? 1.0f : ex2(ref0 - top);
              const float f1 = ref == top ? 1.0f : ex2(ref - top);
              l = lds_f(sum0_s + 4 * h) * f0 + l * f1;
              f *= f1;
              ref = top;
            }
            if (*abort_flag) f = l = NAN;
            if (whole) {
              const float inv = l > 0.0f ? 1.0f / l : 0.0f;
              f *= inv;
              f0 *= inv;
            }
            const float v = l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.69314718055994531f;   // (NaN stays NaN)
            __syncwarp();
            if (lane < 16) {
              sts(fac_s + 4 * h, f);
              sts(fac0_s + 4 * h, f0);
              sts(ref0_s + 4 * h, ref);
              sts(sum0_s + 4 * h, l);
              if (ends && !whole) {
                *reinterpret_cast<float2*>(p.ml + (slot * 64 + h) * 2) = make_float2(ref, l);
              } else if (ends && p.lse) {
                p.lse[static_cast<int64_t>(row) * 64 + h] = v;
              }
            }
          }
          paged_bar(bar, 128);
          paged_wait(o_full, ph_o, kErrWaitTmemFull, abort_flag);
          tc_fence_after();
          ph_o ^= 1;
          if (*abort_flag) sts(fac_s + 4 * (head0 + (lane & 15)), NAN);
          __syncwarp();
          // the channel of this lane's dim, and the lane with the next one (its partner)
          const int ch = KVB ? lane : (lane & ~7) + paged_channel(lane & 7);
          constexpr int kPair = KVB ? 1 : 2;
          const int odd = ch & 1;
          // lanes pair up: the even one writes dims d, d + 1 of head j, the odd one of head j + 1
          auto put = [&](int d, int j, float a, float b) {
            const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, kPair);
            const uint32_t v = odd ? pack_bf16x2(got, b) : pack_bf16x2(a, got);
            *reinterpret_cast<uint32_t*>(p.out + (static_cast<int64_t>(row) * 64 + head0 + odd + j) * 512 + (d & ~1)) = v;
          };
          float* part = p.opart + (static_cast<int64_t>(slot) * 64 + head0) * 512 + 32 * quarter + ch;
          if (!merge) {
            float fac[16];
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              const float4 f = lds_f4(fac_s + 4 * (head0 + j));
              fac[j] = f.x; fac[j + 1] = f.y; fac[j + 2] = f.z; fac[j + 3] = f.w;
            }
#pragma unroll 1
            for (int t = 0; t < 4; ++t) {
              uint32_t r[16];
              tmem_ld_32x32b_x16(tmem + lanes + 64 + 64 * t + head0, r);
              paged_ld_wait(r);
              if (whole) {
#pragma unroll
                for (int j = 0; j < 16; j += 2)
                  put(128 * t + 32 * quarter + ch, j, __uint_as_float(r[j]) * fac[j], __uint_as_float(r[j + 1]) * fac[j + 1]);
              } else {
#pragma unroll
                for (int j = 0; j < 16; ++j) part[j * 512 + 128 * t] = __uint_as_float(r[j]) * fac[j];
              }
            }
          } else {
            // each thread adds to what it wrote itself (rolled: seldom run, and few registers)
#pragma unroll 1
            for (int i = 0; i < 16; ++i) {
              const int t = i >> 2, j = 4 * (i & 3);
              uint32_t r[4];
              float o[4];
              float* at = part + j * 512 + 128 * t;
#pragma unroll
              for (int k = 0; k < 4; ++k) o[k] = at[k * 512];
              tmem_ld_32x32b_x4(tmem + lanes + 64 + 64 * t + head0 + j, r);
              const float4 f = lds_f4(fac_s + 4 * (head0 + j)), f0 = lds_f4(fac0_s + 4 * (head0 + j));
              paged_ld_wait(r);
              o[0] = fmaf(o[0], f0.x, __uint_as_float(r[0]) * f.x);
              o[1] = fmaf(o[1], f0.y, __uint_as_float(r[1]) * f.y);
              o[2] = fmaf(o[2], f0.z, __uint_as_float(r[2]) * f.z);
              o[3] = fmaf(o[3], f0.w, __uint_as_float(r[3]) * f.w);
              if (whole) {
                put(128 * t + 32 * quarter + ch, j, o[0], o[1]);
                put(128 * t + 32 * quarter + ch, j + 2, o[2], o[3]);
              } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) at[k * 512] = o[k];
              }
            }
          }
          tc_fence_before();
          paged_bar(bar, 128);                     // nref_s and fac_s are free
          merge = !ends;
          first = true;
        }
        if (!paged_next(p, c)) break;
      }
      tc_fence_before();
      paged_bar(kPagedEndBar, 32 * (kPagedSoftmax + 1));           // tensor memory is no longer read
    }
  } else if (warp == 0) {
    tmem_dealloc(lds_i(misc32 + 160), 512);
  }
}

// Merge of the queries that range boundaries cut.  A query that CTA c-1
// begins and CTAs c, c+1, ... go on with left its partials in slots
// 2(c-1)+1, 2c, 2(c+1), ...; cut[c] names it and counts them.  Partials are
// added in a fixed order whatever the timing.
//
// CTAs (., y) take the y-th cut query, or, where there are as many queries as
// boundaries, boundary y + 1 if a query is first cut there.  SPLIT = 0 (many
// queries, few partials each): a CTA's four groups of 128 threads take one
// head each.  SPLIT = 1 (fewer queries): a CTA takes one head, its four groups
// every fourth partial each.  SPLIT = 2 (one query or two): a CTA takes half
// of a head's dims, its eight groups of 64 threads every eighth partial each.  A thread owns 4 dims and keeps kFlight
// 16-byte loads in flight, the first of them over the reading of maxima and
// sums: the chain of dependent reads bounds the kernel, not the bytes.
//
// Where the rule lies, attention and join of 262,144 entries in all (us):
//   queries      1     2     4     8    12    16    20
//   SPLIT 2   68.2  65.9  67.6  74.5  83.2  89.0  95.3
//   SPLIT 1   71.2  66.8  64.7  67.8  74.5  77.0  80.4
//   SPLIT 0  118.1  91.6  77.3  71.7  73.0  71.3  71.4
constexpr int kPagedJoinThreads = 512;
constexpr int kPagedHalfJoin = 2, kPagedSplitJoin = 10;            // queries up to which SPLIT is 2, 1
template <int SPLIT>
__global__ void __launch_bounds__(kPagedJoinThreads)
paged_attn_join_kernel(PagedAttnParams p, int ctas) {
  __shared__ int c0_s, count_s[kPagedJoinThreads / 32];
  __shared__ int slot_s[kPagedMaxCtas + 1];              // slot of each partial
  __shared__ float w_s[SPLIT ? 1 : 4][kPagedMaxCtas + 1];  // and its factor, per head of the CTA
  constexpr int kGroup = SPLIT == 2 ? 64 : 128, kGroups = kPagedJoinThreads / kGroup, kFlight = SPLIT ? 8 : 4;
  __shared__ float4 acc_s[SPLIT ? kGroups - 1 : 1][kGroup];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = tid / kGroup, t = tid % kGroup;
  const int h = SPLIT ? blockIdx.x / SPLIT : 4 * blockIdx.x + g;
  const int d = SPLIT == 2 ? 4 * (t + kGroup * (blockIdx.x & 1)) : 4 * t;     // first of the thread's dims
  pdl_launch_dependents();
  if (tid == 0) c0_s = 0;
  pdl_wait();
  int c0 = blockIdx.y + 1;
  if (static_cast<int>(gridDim.y) < ctas - 1) {          // fewer queries than boundaries
    const bool begins = tid + 1 < ctas && __ldcg(&p.cut[tid + 1].y) > 0;
    const uint32_t vote = __ballot_sync(0xffffffffu, begins);
    if (lane == 0) count_s[warp] = __popc(vote);
    __syncthreads();
    int rank = __popc(vote & ((1u << lane) - 1u));
    for (int w = 0; w < warp; ++w) rank += count_s[w];
    if (begins && rank == static_cast<int>(blockIdx.y)) c0_s = tid + 1;
    __syncthreads();
    c0 = c0_s;
    if (c0 == 0) return;
  }
  const int2 cut = __ldcg(p.cut + c0);
  const int row = cut.x, n = cut.y;
  if (n == 0) return;
  if (tid < n) slot_s[tid] = tid == 0 ? 2 * (c0 - 1) + 1 : 2 * (c0 + tid - 1);
  __syncthreads();
  const float* op = p.opart + static_cast<int64_t>(h) * 512 + d;
  constexpr int kStep = SPLIT ? kGroups : 1;
  int i = SPLIT ? g : 0;
  float4 o[kFlight];
#pragma unroll
  for (int j = 0; j < kFlight; ++j)                     // behind the last partial: the last one again, with factor 0
    o[j] = __ldcg(reinterpret_cast<const float4*>(op + static_cast<int64_t>(slot_s[min(i + j * kStep, n - 1)]) * (64 * 512)));
  // every warp: joint maximum and sum of its head, and the partials' factors
  const float2* ml = reinterpret_cast<const float2*>(p.ml) + h;
  constexpr int kMl = (kPagedMaxCtas + 1 + 31) / 32;
  float2 v[kMl];
  float M = -INFINITY, L = 0.0f;
#pragma unroll
  for (int j = 0; j < kMl; ++j) {
    v[j] = make_float2(-INFINITY, 0.0f);
    if (lane + 32 * j < n) v[j] = __ldcg(ml + slot_s[lane + 32 * j] * 64);
  }
#pragma unroll
  for (int j = 0; j < kMl; ++j) M = fmaxf(M, v[j].x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
#pragma unroll
  for (int j = 0; j < kMl; ++j) {
    const float f = exp2f(v[j].x - M);
    L += f * v[j].y;
    if (t < 32 && lane + 32 * j < n) w_s[SPLIT ? 0 : g][lane + 32 * j] = f;        // (SPLIT: the groups write the same)
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xffffffffu, L, d);
  __syncthreads();
  const float* w = w_s[SPLIT ? 0 : g];
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  while (true) {
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      const int k = i + j * kStep;
      const float f = k < n ? w[k] : 0.0f;
      acc.x += f * o[j].x; acc.y += f * o[j].y; acc.z += f * o[j].z; acc.w += f * o[j].w;
    }
    i += kFlight * kStep;
    if (i >= n) break;
#pragma unroll
    for (int j = 0; j < kFlight; ++j)
      o[j] = __ldcg(reinterpret_cast<const float4*>(op + static_cast<int64_t>(slot_s[min(i + j * kStep, n - 1)]) * (64 * 512)));
  }
  if (SPLIT) {
    if (g > 0) acc_s[g - 1][t] = acc;
    __syncthreads();
    if (g > 0) return;
#pragma unroll
    for (int k = 0; k < kGroups - 1; ++k) {
      const float4 q = acc_s[k][t];
      acc.x += q.x; acc.y += q.y; acc.z += q.z; acc.w += q.w;
    }
  }
  const float inv = (L > 0.0f) ? 1.0f / L : 0.0f;
  uint2 packed;
  packed.x = pack_bf16x2(acc.x * inv, acc.y * inv);
  packed.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(row) * 64 + h) * 512 + d) = packed;
  if (p.lse && d == 0)
    p.lse[static_cast<int64_t>(row) * 64 + h] = L == 0.0f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

}  // namespace csa2
