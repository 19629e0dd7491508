// evict.cuh -- keeping the cache rows that attention weighs most.
//
// sdpa_evict_select_kernel, one block per (sequence, head): of the len rows, the last `rec` are kept; of the
// n = len - rec rows before them the `need` with the largest accumulated weight.  The need-th largest is
// found by a radix selection on the weights' bits (four passes over eight bits each, as an order-preserving
// unsigned number), then one ordered pass writes the kept rows' numbers by prefix sums, which makes the
// lower row win where weights are equal.  The weights are moved in the same pass.
// sdpa_evict_rows_kernel moves the rows: it reads and writes each kept row once (the bound: HBM).
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

constexpr int EVICT_THREADS = 512;

// Larger weights have larger numbers; NaN has the smallest.
__device__ __forceinline__ uint32_t evict_order(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as 0
  if (w != w) return 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the block of v (two 32-bit counts packed in 64 bits); total: the whole sum.
__device__ __forceinline__ unsigned long long evict_scan(unsigned long long v, unsigned long long& total,
                                                         unsigned long long* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  unsigned long long before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < EVICT_THREADS / 32; ++i) {
    if (i < warp) before += warp_sums[i];
    all += warp_sums[i];
  }
  __syncthreads();
  total = all;
  return before + x - v;
}

__global__ void __launch_bounds__(EVICT_THREADS) sdpa_evict_select_kernel(const EvictParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_prefix, s_need;
  __shared__ unsigned long long warp_sums[EVICT_THREADS / 32];
  const size_t bh = blockIdx.x;
  const int b = blockIdx.x / p.H;
  const int len = cache_len(p.kv_lens, b, p.n_cap);
  const int n_new = min(len, p.budget), rec = min(p.recent, n_new);
  const int n = len - rec, need = n_new - rec;
  const float* acc = p.acc + bh * p.n_cap;
  float* acc_out = p.acc_out + bh * p.n_out;
  int* keep = p.keep + bh * p.budget;
  if (threadIdx.x == 0 && blockIdx.x == b * p.H) p.new_lens[b] = n_new;

  uint32_t limit = 0;      // the need-th largest
  uint32_t ties = 0;       // how many equal to it are kept
  if (need > 0 && need < n) {
    uint32_t prefix = 0, left = (uint32_t)need;
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += EVICT_THREADS) hist[i] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
      for (int j = threadIdx.x; j < n; j += EVICT_THREADS) {
        const uint32_t u = evict_order(acc[j]);
        if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        uint32_t above = 0;
        int d = 255;
        while (above + hist[d] < left) above += hist[d--];
        s_prefix = prefix | ((uint32_t)d << shift);
        s_need = left - above;
      }
      __syncthreads();
      prefix = s_prefix;
      left = s_need;
    }
    limit = prefix;
    ties = left;
  } else if (need > 0) {  // all of them: every number is >= 0, take all ties
    ties = (uint32_t)n;
  }
  // Ordered pass.  Row j goes to (kept rows before it) <= j, and every earlier chunk has been read, so
  // acc_out may be acc.
  unsigned long long run = 0;  // (larger, equal) counts of the chunks before
  if (need > 0) {
    for (int j0 = 0; j0 < n; j0 += EVICT_THREADS) {
      const int j = j0 + threadIdx.x;
      const float w = j < n ? acc[j] : 0.f;
      const uint32_t u = evict_order(w);
      const bool gt = j < n && u > limit, eq = j < n && u == limit;
      unsigned long long total;
      const unsigned long long pre = run + evict_scan(((unsigned long long)gt << 32) | (uint32_t)eq, total, warp_sums);
      const uint32_t eq_before = (uint32_t)pre, gt_before = (uint32_t)(pre >> 32);
      if (gt || (eq && eq_before < ties)) {
        const uint32_t to = gt_before + min(eq_before, ties);
        keep[to] = j;
        acc_out[to] = w;
      }
      run += total;
    }
  }
  for (int j0 = 0; j0 < rec; j0 += EVICT_THREADS) {
    const int i = j0 + threadIdx.x;
    const float w = i < rec ? acc[n + i] : 0.f;
    __syncthreads();
    if (i < rec) {
      keep[need + i] = n + i;
      acc_out[need + i] = w;
    }
  }
  __syncthreads();
  for (int i = n_new + threadIdx.x; i < p.budget; i += EVICT_THREADS) keep[i] = -1;
  for (int i = n_new + threadIdx.x; i < p.n_out; i += EVICT_THREADS) acc_out[i] = 0.f;
}

struct EvictRowsParams {
  const uint8_t* src[4];
  uint8_t* dst[4];
  int row_bytes[4];
  const int* keep;      // [B, H, budget]
  const int* kv_lens;
  int n_arrays, H, n_cap, n_out, budget;
};

// Words of W bytes.  Grid: x (sequence, head), y array.  In place is safe: the rows of a chunk are read
// before they are written, and a kept row only moves down, so later chunks' sources lie above this chunk.
template <class W>
__device__ __forceinline__ void evict_move(const uint8_t* src, uint8_t* dst, const int* keep, int n, int row_bytes) {
  const int wpr = row_bytes / (int)sizeof(W), rpc = 256 / wpr;
  const int r = threadIdx.x / wpr, w = threadIdx.x % wpr;
  for (int i0 = 0; i0 < n; i0 += rpc) {
    const int i = i0 + r;
    const bool on = r < rpc && i < n;
    W x;
    if (on) x = reinterpret_cast<const W*>(src + (size_t)keep[i] * row_bytes)[w];
    __syncthreads();
    if (on) reinterpret_cast<W*>(dst + (size_t)i * row_bytes)[w] = x;
  }
}

__global__ void __launch_bounds__(256) sdpa_evict_rows_kernel(const EvictRowsParams p) {
  const int a = blockIdx.y;
  const size_t bh = blockIdx.x;
  const int len = cache_len(p.kv_lens, blockIdx.x / p.H, p.n_cap);
  const int n = min(len, p.budget), rb = p.row_bytes[a];
  const uint8_t* src = p.src[a] + bh * p.n_cap * rb;
  uint8_t* dst = p.dst[a] + bh * p.n_out * rb;
  if (rb >= 32)
    evict_move<uint4>(src, dst, p.keep + bh * p.budget, n, rb);
  else
    evict_move<uint2>(src, dst, p.keep + bh * p.budget, n, rb);
}

}  // namespace sdpa
