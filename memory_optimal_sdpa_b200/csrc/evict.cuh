// evict.cuh -- keeping the cache rows that attention weighs most.
//
// sdpa_evict_select_kernel, one block per (sequence, head): of the len rows, the last `rec` are kept; of the
// n = len - rec rows before them the `need` with the largest accumulated weight.  The need-th largest is
// found by a radix selection on the weights' bits as an order-preserving unsigned number (11, 11 and 10 bits; a
// block-wide scan finds each digit), then one ordered pass by ballots writes the kept rows' numbers, which makes the lower
// row win where weights are equal.  Up to EVICT_CACHED weights stay in shared memory, so they are read from HBM once; beyond that
// every pass reads them again (from L2).
// sdpa_evict_rows_kernel moves the rows; it reads and writes each kept row once (the bound: HBM).  Into another
// cache all rows move at once; in place sdpa_evict_rows_in_place_kernel goes through a sequence's rows in order.  Both are
// programmatic dependents of the selection and wait for it first (2 us of 67 for 16 x 8 heads, 8192 -> 2048 rows of 256 bytes).
// A block picks its array's pointers from its parameters at run time, which puts those 120 bytes in local memory.
// In place the rounds of a sequence and head run one after another in a block for each array and 64-byte slice of its rows.
// Whole calls, in place and into another cache: 16 x 8 heads, d = 128, 4001-8192 -> 2048 rows bf16 87 and 69 us, 4 bits 42 and 36 us; 1 x 8 heads,
// 32768 -> 4096 rows bf16 52 and 38 us, 4 bits 52 and 34 us; 1 x 8 heads, d = 64, 4096 -> 1024 rows bf16 20 and 15 us.
#pragma once

#include "kv4.cuh"

namespace sdpa {

struct EvictParams {
  const float* acc;      // [B, H, n_cap]
  float* acc_out;        // [B, H, n_out]
  const int* kv_lens;    // [B]
  int* keep;             // [B, H, budget]
  int* new_lens;         // [B]
  int H, n_cap, n_out, budget, recent;
};

constexpr int EVICT_THREADS = 1024;
constexpr int EVICT_CACHED = 48 * 1024;  // weights in shared memory (192 KB)
constexpr int EVICT_BINS = 2048;

// Larger weights have larger numbers; NaN has the smallest.
__device__ __forceinline__ uint32_t evict_order(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
  if (w != w) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the block's threads.
__device__ __forceinline__ uint32_t evict_scan(uint32_t v, uint32_t* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  uint32_t w = warp_sums[lane];  // 32 warps
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, w, off);
    if (lane >= off) w += y;
  }
  const uint32_t before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
  return (warp ? before : 0u) + x - v;
}

template <bool CACHED>
__global__ void __launch_bounds__(EVICT_THREADS) sdpa_evict_select_kernel(const EvictParams p) {
  extern __shared__ float s_acc[];  // CACHED: all len weights
  __shared__ uint32_t hist[EVICT_BINS];
  __shared__ uint32_t warp_sums[32], warp_eq[32];
  __shared__ uint32_t s_digit, s_left;
  constexpr int WARPS = EVICT_THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t bh = blockIdx.x;
  const int b = blockIdx.x / p.H;
  const int len = cache_len(p.kv_lens, b, p.n_cap);
  const int n_new = min(len, p.budget), rec = min(p.recent, n_new);
  const int n = len - rec, need = n_new - rec;
  const float* acc = p.acc + bh * p.n_cap;
  float* acc_out = p.acc_out + bh * p.n_out;
  int* keep = p.keep + bh * p.budget;
  if (threadIdx.x == 0 && blockIdx.x == b * p.H) p.new_lens[b] = n_new;
  if (CACHED) {
#pragma unroll 4
    for (int j = threadIdx.x; j < len; j += EVICT_THREADS) s_acc[j] = acc[j];
    __syncthreads();
  }
  auto weight = [&](int j) { return CACHED ? s_acc[j] : acc[j]; };

  uint32_t limit = 0;                  // the need-th largest
  uint32_t ties = (uint32_t)max(need, 0);  // how many equal to it are kept (all rows: every number is >= 0)
  if (need > 0 && need < n) {
    uint32_t left = (uint32_t)need;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bins = pass == 2 ? 1024 : 2048;
      const uint32_t mask = pass == 0 ? 0u : 0xFFFFFFFFu << (pass == 1 ? 21 : 10);
      for (int i = threadIdx.x; i < bins; i += EVICT_THREADS) hist[i] = 0;
      __syncthreads();
#pragma unroll 4
      for (int j = threadIdx.x; j < n; j += EVICT_THREADS) {
        const uint32_t u = evict_order(weight(j));
        if ((u & mask) == limit) atomicAdd(&hist[(u >> shift) & (bins - 1)], 1u);
      }
      __syncthreads();
      // bins from the top: thread t has bins top - 2 t and top - 2 t - 1
      const int top = bins - 1 - 2 * (int)threadIdx.x;
      const uint32_t h0 = top >= 0 ? hist[top] : 0u, h1 = top >= 1 ? hist[top - 1] : 0u;
      const uint32_t above = evict_scan(h0 + h1, warp_sums);
      if (above < left && left <= above + h0 + h1) {
        const bool upper = left <= above + h0;
        s_digit = (uint32_t)(upper ? top : top - 1);
        s_left = left - above - (upper ? 0u : h0);
      }
      __syncthreads();
      limit |= s_digit << shift;
      left = s_left;
    }
    ties = left;
  }
  // Ordered pass: each warp has a stretch of the rows; counts first, then places.
  if (need > 0) {
    const int stretch = ((n + WARPS - 1) / WARPS + 31) / 32 * 32, j0 = warp * stretch, j1 = min(n, j0 + stretch);
    uint32_t gt = 0, eq = 0;
    for (int j = j0 + lane; j < j1; j += 32) {
      const uint32_t u = evict_order(weight(j));
      gt += u > limit;
      eq += u == limit;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    __syncthreads();  // the scans' sums have been read
    if (lane == 0) {
      warp_sums[warp] = gt;
      warp_eq[warp] = eq;
    }
    __syncthreads();
    uint32_t gt_before = __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[lane] : 0u);
    uint32_t eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? warp_eq[lane] : 0u);
    const uint32_t lower = (1u << lane) - 1u;
    for (int j = j0; j < j1; j += 32) {
      const float w = j + lane < j1 ? weight(j + lane) : 0.f;
      const uint32_t u = evict_order(w);
      const bool on = j + lane < j1, is_gt = on && u > limit, is_eq = on && u == limit;
      const uint32_t m_gt = __ballot_sync(0xffffffffu, is_gt), m_eq = __ballot_sync(0xffffffffu, is_eq);
      const uint32_t e = eq_before + __popc(m_eq & lower);
      if (is_gt || (is_eq && e < ties)) {
        const uint32_t to = gt_before + __popc(m_gt & lower) + min(e, ties);
        keep[to] = j + lane;
        if (CACHED) acc_out[to] = w;
      }
      gt_before += __popc(m_gt);
      eq_before += __popc(m_eq);
    }
  }
  for (int i = threadIdx.x; i < rec; i += EVICT_THREADS) {
    keep[need + i] = n + i;
    if (CACHED) acc_out[need + i] = s_acc[n + i];
  }
  if (!CACHED) {
    // In order, as acc_out may be acc: a kept row only moves down, and a round's weights are read before they are written.
    __syncthreads();
    for (int i0 = 0; i0 < n_new; i0 += EVICT_THREADS) {
      const int i = i0 + threadIdx.x;
      const float w = i < n_new ? acc[keep[i]] : 0.f;
      __syncthreads();
      if (i < n_new) acc_out[i] = w;
    }
    __syncthreads();
  }
  for (int i = n_new + threadIdx.x; i < p.budget; i += EVICT_THREADS) keep[i] = -1;
  for (int i = n_new + threadIdx.x; i < p.n_out; i += EVICT_THREADS) acc_out[i] = 0.f;
}

struct EvictRowsParams {
  const uint8_t* src[4];
  uint8_t* dst[4];
  int row_bytes[4];
  const int* keep;      // [B, H, budget]
  const int* kv_lens;
  int H, n_cap, n_out, budget;
  int n_bh;             // B H
};

constexpr int EVICT_ROW_THREADS = 256;
constexpr int EVICT_ROW_UNROLL = 8;    // rows a thread has in flight, into another cache
constexpr int EVICT_SHIFT_UNROLL = 4;  // and in place

// Words of W bytes, into another cache.  A block takes every gridDim.x-th stretch of rows, the next stretch's loads ahead
// of this one's stores.  Measured with the selection (14 us), 16 x 8 heads, 8192 -> 2048 rows of 256 bytes: blocks of one
// stretch each 108 / 82 / 74 us with 2 / 4 / 8 rows a thread (they spend their time starting), this form 86 / 67 us with
// 4 / 8 rows; 8 and 16 blocks an SM 69 us (all before the overlapped launch).  Kept rows lie about 1 KB apart there, so the reads are short DRAM bursts.
template <class W>
__device__ __forceinline__ void evict_copy(const EvictRowsParams& p, const uint8_t* src, uint8_t* dst, int row_bytes) {
  constexpr int U = EVICT_ROW_UNROLL;
  const int wpr = row_bytes / (int)sizeof(W), rpp = EVICT_ROW_THREADS / wpr;  // words per row, rows per pass
  const int r = threadIdx.x / wpr, w = threadIdx.x - r * wpr;
  const int per_bh = (p.budget + U * rpp - 1) / (U * rpp);  // stretches per (sequence, head)
  const uint32_t total = (uint32_t)per_bh * p.n_bh;
  struct Stretch {
    W x[U];
    W* to;  // of this thread's first row
    int left;  // rows from there on
  };
  auto load = [&](uint32_t item, Stretch& s) {
    s.left = 0;
    if (item >= total) return;
    const uint32_t bh = item / (uint32_t)per_bh;
    const int i0 = (int)(item - bh * per_bh) * (U * rpp) + r;
    s.left = min(cache_len(p.kv_lens, (int)bh / p.H, p.n_cap), p.budget) - i0;
    const int* keep = p.keep + (size_t)bh * p.budget + i0;
    const uint8_t* from = src + (size_t)bh * p.n_cap * row_bytes + w * sizeof(W);
    s.to = reinterpret_cast<W*>(dst + ((size_t)bh * p.n_out + i0) * row_bytes) + w;
    int at[U];
#pragma unroll
    for (int u = 0; u < U; ++u) at[u] = u * rpp < s.left ? keep[u * rpp] : 0;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u * rpp < s.left) s.x[u] = __ldcs(reinterpret_cast<const W*>(from + (size_t)at[u] * row_bytes));
  };
  Stretch s, next;
  load(blockIdx.x, s);
  for (uint32_t item = blockIdx.x; item < total; item += gridDim.x) {
    load(item + gridDim.x, next);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u * rpp < s.left) s.to[(size_t)u * rpp * wpr] = s.x[u];
    s = next;
  }
}

// Grid: x blocks that share the stretches, y array.  Row sizes are powers of two from 8 to 256 bytes.
__global__ void __launch_bounds__(EVICT_ROW_THREADS) sdpa_evict_rows_kernel(const EvictRowsParams p) {
  cudaGridDependencySynchronize();
  const int a = blockIdx.y, rb = p.row_bytes[a];
  if (rb >= 16)
    evict_copy<uint4>(p, p.src[a], p.dst[a], rb);
  else
    evict_copy<uint2>(p, p.src[a], p.dst[a], rb);
}

// In place, a slice of `bytes` of every row at a time.  Rounds of rows in order: a round's rows are in registers
// of the whole block before any of them is written, and a kept row only moves down, so what later rounds
// read lies above everything written so far; their loads may start early.  Rows that stay where they are are not written.
template <class W>
__device__ __forceinline__ void evict_shift(uint8_t* rows, const int* keep, int n, int row_bytes, int bytes, int slice) {
  const int wps = bytes / (int)sizeof(W), rpp = EVICT_ROW_THREADS / wps;
  const int r = threadIdx.x / wps, w = threadIdx.x - r * wps;
  uint8_t* col = rows + (size_t)slice * bytes + w * sizeof(W);
  constexpr int U = EVICT_SHIFT_UNROLL;
  W x[U], y[U];
  int from[U], from_next[U];
  auto load = [&](int i0, W* to, int* at) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * rpp + r;
      at[u] = i < n ? keep[i] : i;
      if (at[u] != i) to[u] = *reinterpret_cast<const W*>(col + (size_t)at[u] * row_bytes);
    }
  };
  load(0, x, from);
  for (int i0 = 0; i0 < n; i0 += U * rpp) {
    load(i0 + U * rpp, y, from_next);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * rpp + r;
      if (from[u] != i) *reinterpret_cast<W*>(col + (size_t)i * row_bytes) = x[u];
      x[u] = y[u];
      from[u] = from_next[u];
    }
  }
}

// Grid: x (sequence, head), y slice of 64 bytes, z array.
__global__ void __launch_bounds__(EVICT_ROW_THREADS) sdpa_evict_rows_in_place_kernel(const EvictRowsParams p) {
  cudaGridDependencySynchronize();
  const int a = blockIdx.z, len = cache_len(p.kv_lens, blockIdx.x / p.H, p.n_cap), n = min(len, p.budget);
  const size_t bh = blockIdx.x;
  const int rb = p.row_bytes[a], bytes = min(rb, 64);
  if ((int)blockIdx.y * bytes >= rb) return;
  uint8_t* rows = p.dst[a] + bh * p.n_cap * rb;
  if (bytes >= 16)
    evict_shift<uint4>(rows, p.keep + bh * p.budget, n, rb, bytes, blockIdx.y);
  else
    evict_shift<uint2>(rows, p.keep + bh * p.budget, n, rb, bytes, blockIdx.y);
}

}  // namespace sdpa
