// paged_tables.cuh -- block tables and pool rows of a block-paged cache,
// made on the device from request lengths (csa2_block_tables) and from
// selected positions (csa2_paged_rows).
//
// Request b holds len entries in ceil(len / P) blocks of P entries; a step
// appends n_new.  With have = ceil(len / P) and want = ceil((len + n_new) / P)
// it takes want - have blocks from the free list, at the exclusive sum of
// the earlier requests' needs; new entry i sits at position len + i, in block
// table[pos / P], row table[pos / P] * P + pos % P.  A new block begins
// exactly at a position divisible by P, so the thread that makes that
// position's row also writes the block's table entry, and no second pass
// over the tables is needed.
//
// Bytes: 16 per request, 8 per block taken, 8 per row written.  Small steps
// are bound by latency, two block-wide scans and one binary search per row:
// 3.0 us for 4 requests, 5.8 us for 1024 with one entry each.  512 requests
// with up to 4096 new entries each (310,000 rows) take 13 us, 0.4 of them
// for the bytes; the row kernel's searches and reads are the rest.
#pragma once
#include "common.cuh"

namespace csa2 {

constexpr int kTablesThreads = 1024;
constexpr int kRowsPerBlock = 1024;            // fill: rows per CTA, one per thread
// Up to this many rows, one per thread, the scanning CTA writes the rows itself
// and saves a launch (us, against two launches: 4 rows 3.0 and 4.3; 256 rows
// 4.0 and 5.1; 1024 rows 6.2 and 7.3; 2048 rows 8.2 and 7.3)
constexpr int64_t kTablesOneLaunch = kTablesThreads;
// Up to this many requests the row kernel's CTAs copy the starts to shared
// memory, for the dependent reads of the search (13.7 against 14.6 us in the case above)
constexpr int kStartsShared = 4096;

// Division by a launch's constant (Granlund and Montgomery, "Division by
// invariant integers using multiplication"): with l = ceil(log2 d) and
// m = floor(2^32 (2^l - d) / d) + 1, n / d = (mulhi(m, n) + n) >> l.  The sum
// needs n < 2^31.  Divisions by run-time values bounded paged_rows_kernel
// (three per position: 4096 x 512 positions took 9.4 us, now 6.4).
struct DivBy {
  uint32_t m, l;
  static DivBy of(uint32_t d) {
    uint32_t l = 0;
    while ((uint64_t(1) << l) < d) ++l;
    return {static_cast<uint32_t>((((uint64_t(1) << l) - d) << 32) / d + 1), l};
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(m, n) + n) >> l; }
};

struct TablesParams {
  int B;
  uint32_t P;                  // entries per block
  DivBy by_P;
  int64_t cap;                 // entries that a table row can name: max_blocks * P
  int64_t ld_table;
  const int32_t* len;
  const int32_t* n_new;
  const int32_t* free_blocks;
  int n_free;
  const int32_t* free_pos;     // optional
  int32_t* table;
  int32_t* len_out;            // may be len
  int32_t* start;              // [B + 1]
  int64_t* slots;
  int64_t max_new;
  int32_t* info;               // info[0] may be free_pos
  int32_t* base;               // workspace [B]: index in the free list of the request's first new block, -1 refused
};

// Exclusive sum over the CTA of one value per thread; *total gets the sum.
// `warp_s` holds one value per warp plus the total.
__device__ __forceinline__ int64_t block_exclusive_sum(int64_t v, int64_t* warp_s, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) warp_s[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int64_t w = (lane < n_warps) ? warp_s[lane] : 0;
    int64_t s = w;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += o;
    }
    if (lane < n_warps) warp_s[lane] = s - w;
    if (lane == 31) warp_s[32] = s;
  }
  __syncthreads();
  const int64_t r = warp_s[warp] + incl - v;
  *total = warp_s[32];
  __syncthreads();                              // warp_s may be used again
  return r;
}

// Row of new entry i (and, where the entry opens a block, its table entry).
// start and len_out are the call's own results, written before; start may be
// a copy in shared memory.  (Four rows per thread, neighbours or a CTA's
// stride apart, saved searches but lengthened the chain of reads: 13.8 and
// 18.3 us against 13.0 for 512 requests with up to 4096 new entries each.)
__device__ __forceinline__ void write_row(const TablesParams& p, const int32_t* start, int64_t i) {
  // the request with start[b] <= i < start[b + 1]: the last b with start[b] <= i
  // (requests without new entries share their successor's start)
  int64_t slot = -1;
  if (i < start[p.B]) {
    int lo = 0, hi = p.B;                       // start[lo] <= i < start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= i) lo = mid; else hi = mid;
    }
    const int32_t base = p.base[lo];
    if (base >= 0) {
      const uint32_t len = static_cast<uint32_t>(p.len_out[lo] - p.n_new[lo]);
      const uint32_t pos = len + static_cast<uint32_t>(i - start[lo]);
      const uint32_t have = p.by_P(len + p.P - 1), j = p.by_P(pos), r = pos - j * p.P;
      int32_t* row = p.table + lo * p.ld_table;
      const int32_t id = (j < have) ? row[j] : p.free_blocks[base + static_cast<int32_t>(j - have)];
      if (r == 0) row[j] = id;
      if (id >= 0) slot = static_cast<int64_t>(id) * p.P + r;
    }
  }
  p.slots[i] = slot;
}

// One CTA: the two scans over the requests (rows of the step, then blocks of
// the requests that fit), and with `fill` the rows themselves.
__global__ void __launch_bounds__(kTablesThreads)
block_tables_kernel(TablesParams p, int fill) {
  __shared__ int64_t warp_s[33];
  __shared__ int refused_s;
  __shared__ int64_t taken_s;
  const int tid = threadIdx.x;
  pdl_launch_dependents();
  if (tid == 0) { refused_s = 0; taken_s = 0; }
  pdl_wait();
  const int per = (p.B + kTablesThreads - 1) / kTablesThreads;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  // a thread's first request, usually its only one, is read once, in one go
  const int32_t len0 = b0 < b1 ? p.len[b0] : 0, add0 = b0 < b1 ? p.n_new[b0] : 0;
  const int64_t pos0 = p.free_pos ? p.free_pos[0] : 0;
  auto len_of = [&](int b) -> int32_t { return b == b0 ? len0 : p.len[b]; };
  auto add_of = [&](int b) -> int32_t { return b == b0 ? add0 : p.n_new[b]; };
  int64_t rows = 0, total = 0;
  for (int b = b0; b < b1; ++b) rows += max(add_of(b), 0);
  const int64_t row0 = block_exclusive_sum(rows, warp_s, &total);
  const int64_t all_rows = total;
  // a request that its table row or the row list cannot hold takes nothing
  int64_t at = row0, need_sum = 0;
  auto need_of = [&](int b, int64_t first, bool& fits) -> int64_t {
    const int64_t len = len_of(b), add = add_of(b);
    fits = len >= 0 && add >= 0 && len + add <= p.cap && first + add <= p.max_new;
    // (entries and P are at most 2^30 each)
    return fits ? p.by_P(static_cast<uint32_t>(len + add) + p.P - 1) - p.by_P(static_cast<uint32_t>(len) + p.P - 1) : 0;
  };
  for (int b = b0; b < b1; ++b) {
    bool fits;
    need_sum += need_of(b, at, fits);
    at += max(add_of(b), 0);
  }
  int64_t base = block_exclusive_sum(need_sum, warp_s, &total) + pos0;
  int refused = 0;
  int64_t taken = 0;
  at = row0;
  for (int b = b0; b < b1; ++b) {
    bool fits;
    const int64_t need = need_of(b, at, fits);
    const bool ok = fits && (need == 0 || (pos0 >= 0 && base + need <= p.n_free));
    const int32_t add = add_of(b), len = len_of(b);
    p.start[b] = static_cast<int32_t>(min(at, p.max_new));
    p.len_out[b] = ok ? len + add : len;
    p.base[b] = ok ? (need ? static_cast<int32_t>(base) : 0) : -1;
    if (ok) taken += need; else ++refused;
    base += need;
    at += max(add, 0);
  }
  if (refused) atomicAdd(&refused_s, refused);
  if (taken) atomicAdd(reinterpret_cast<unsigned long long*>(&taken_s), static_cast<unsigned long long>(taken));
  if (tid == 0) p.start[p.B] = static_cast<int32_t>(min(all_rows, p.max_new));
  __syncthreads();
  if (tid == 0) {
    p.info[0] = static_cast<int32_t>(pos0 + taken_s);
    p.info[1] = refused_s;
  }
  if (fill && tid < p.max_new) write_row(p, p.start, tid);
}

// One thread per row of the list.
__global__ void __launch_bounds__(kRowsPerBlock)
block_rows_kernel(TablesParams p) {
  __shared__ int32_t start_s[kStartsShared + 1];
  pdl_launch_dependents();
  pdl_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRowsPerBlock + threadIdx.x;
  const int32_t* start = p.start;
  if (p.B <= kStartsShared) {
    for (int b = threadIdx.x; b <= p.B; b += kRowsPerBlock) start_s[b] = p.start[b];
    __syncthreads();
    start = start_s;
  }
  if (i < p.max_new) write_row(p, start, i);
}

// ---------------------------------------------------------------------------
// Pool rows of selected positions: 8 bytes per position and one table entry
// (a row of the table stays in L1 / L2).  Four positions per thread by one
// 16-byte load and store.  4096 x 512 positions: 6.4 us, 2.6 TB/s; 2.6 us at
// the copy rate.
// ---------------------------------------------------------------------------
struct PagedRowsParams {
  const int32_t* pos;          // [R][K]
  const int32_t* n_vis;        // optional [R]
  const int32_t* table;
  int32_t* rows;               // [R][K]; may be pos
  uint32_t n;                  // R * K
  DivBy by_K, by_Q, by_P;
  uint32_t P;
  uint32_t max_blocks, n_blocks;
  int64_t ld_table;
};

__global__ void __launch_bounds__(256)
paged_rows_kernel(PagedRowsParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t i0 = (blockIdx.x * 256u + threadIdx.x) * 4u;
  if (i0 >= p.n) return;
  const uint32_t m = min(4u, p.n - i0);
  int32_t v[4] = {-1, -1, -1, -1};
  if (m == 4) {
    const int4 x = *reinterpret_cast<const int4*>(p.pos + i0);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  } else {
    for (uint32_t j = 0; j < m; ++j) v[j] = p.pos[i0 + j];
  }
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j) {
    if (j >= m || v[j] < 0) { v[j] = -1; continue; }
    const uint32_t r = p.by_K(i0 + j), b = p.by_Q(r);
    const uint32_t pos = static_cast<uint32_t>(v[j]), blk = p.by_P(pos);
    int32_t row = -1;
    if (blk < p.max_blocks && (!p.n_vis || v[j] < p.n_vis[r])) {
      const int32_t id = p.table[b * p.ld_table + blk];
      if (id >= 0 && static_cast<uint32_t>(id) < p.n_blocks) row = static_cast<int32_t>(id * p.P + (pos - blk * p.P));
    }
    v[j] = row;
  }
  if (m == 4) {
    *reinterpret_cast<int4*>(p.rows + i0) = make_int4(v[0], v[1], v[2], v[3]);
  } else {
    for (uint32_t j = 0; j < m; ++j) p.rows[i0 + j] = v[j];
  }
}

}  // namespace csa2
