// decode_cache.cuh -- one query row per head against a bounded cache: bf16 or 4-bit rows, with the
// attention weights of every key added to an accumulator where asked for.
//
// CTA (split s, key/value head, b) reduces keys [s chunk, s chunk + chunk) of the valid prefix to a
// normalised partial output and a log-sum-exp (base 2) per query head.  With weights it also writes the
// scores (base 2, fp32): a key's weight needs the log-sum-exp over all splits, and reading 4 bytes a
// score back is far cheaper than reading the keys again.  sdpa_cache_finish_kernel joins the splits,
// sdpa_cache_weights_kernel adds sum_h 2^(score_h - LSE_h) per key.
#pragma once

#include "kv4.cuh"

namespace sdpa {

struct CacheDecodeParams {
  const __nv_bfloat16* Q;       // [B, Hq, D]
  const __nv_bfloat16* rows[2]; // bf16 cache K, V
  Kv4Cache cache[2];            // or 4-bit cache K, V
  const int* kv_lens;
  float* part_o;    // [B, Hq, S, D]
  float* part_lse;  // [B, Hq, S], base 2
  float* lse2;      // [B, Hq], base 2
  float* scores;    // [B, Hq, n_cap], base 2, or null
  const float* acc;
  float* acc_out;   // [B, Hkv, n_cap]
  __nv_bfloat16* O;
  float* LSE;
  int H_q, H_kv, group, n_cap, chunk, n_split;
  float scale_log2;
};

constexpr int CACHE_HEADS = 8;   // query heads per CTA
constexpr int CACHE_CHUNK = 256; // keys per split
constexpr int CACHE_THREADS = 128;

template <int D, bool KV4>
__device__ __forceinline__ float cache_value(const CacheDecodeParams& p, int which, size_t row, int e) {
  if (!KV4) return __bfloat162float(p.rows[which][row * D + e]);
  constexpr int NG = D / 32;
  const int g = e >> 5, r = (e >> 2) & 7;
  const uint32_t byte = p.cache[which].codes[row * (D / 2) + 2 * (r * NG + g) + ((e >> 1) & 1)];
  const uint32_t sm = p.cache[which].scales[row * NG + g];
  return fmaf(__uint_as_float(sm << 16), (float)((byte >> (4 * (e & 1))) & 15u), __uint_as_float(sm & 0xFFFF0000u));
}

template <int D, bool KV4>
__global__ void __launch_bounds__(CACHE_THREADS) sdpa_cache_split_kernel(const CacheDecodeParams p) {
  __shared__ float s_q[CACHE_HEADS][D];
  __shared__ float s_p[CACHE_HEADS][CACHE_CHUNK];
  __shared__ float s_m[CACHE_HEADS], s_l[CACHE_HEADS];
  const int hb = (p.group + CACHE_HEADS - 1) / CACHE_HEADS;
  const int s = blockIdx.x, kvh = blockIdx.y / hb, h0 = (blockIdx.y % hb) * CACHE_HEADS, b = blockIdx.z;
  const int nh = min(CACHE_HEADS, p.group - h0);
  const int len = cache_len(p.kv_lens, b, p.n_cap);
  const int k0 = s * p.chunk;
  if (k0 >= len) return;
  const int n = min(p.chunk, len - k0);
  const size_t row0 = ((size_t)b * p.H_kv + kvh) * p.n_cap + k0;
  const size_t head0 = (size_t)b * p.H_q + kvh * p.group + h0;
  for (int i = threadIdx.x; i < nh * D; i += CACHE_THREADS)
    s_q[i / D][i % D] = __bfloat162float(p.Q[head0 * D + i]) * p.scale_log2;
  __syncthreads();
  for (int j = threadIdx.x; j < n; j += CACHE_THREADS) {
    float d[CACHE_HEADS] = {};
    for (int e = 0; e < D; ++e) {
      const float x = cache_value<D, KV4>(p, 0, row0 + j, e);
      for (int h = 0; h < nh; ++h) d[h] = fmaf(x, s_q[h][e], d[h]);
    }
    for (int h = 0; h < nh; ++h) {
      s_p[h][j] = d[h];
      if (p.scores) p.scores[(head0 + h) * p.n_cap + k0 + j] = d[h];
    }
  }
  __syncthreads();
  for (int h = threadIdx.x >> 5; h < nh; h += CACHE_THREADS / 32) {
    const int lane = threadIdx.x & 31;
    float m = -__int_as_float(0x7f800000), l = 0.f;
    for (int j = lane; j < n; j += 32) m = fmaxf(m, s_p[h][j]);
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    for (int j = lane; j < n; j += 32) {
      const float e = exp2f(s_p[h][j] - m);
      s_p[h][j] = e;
      l += e;
    }
    for (int off = 16; off; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
    if (lane == 0) {
      s_l[h] = l;
      p.part_lse[(head0 + h) * p.n_split + s] = m + log2f(l);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += CACHE_THREADS) {
    float o[CACHE_HEADS] = {};
    for (int j = 0; j < n; ++j) {
      const float x = cache_value<D, KV4>(p, 1, row0 + j, e);
      for (int h = 0; h < nh; ++h) o[h] = fmaf(s_p[h][j], x, o[h]);
    }
    for (int h = 0; h < nh; ++h) p.part_o[((head0 + h) * p.n_split + s) * D + e] = o[h] / s_l[h];
  }
}

template <int D>
__global__ void __launch_bounds__(D) sdpa_cache_finish_kernel(const CacheDecodeParams p) {
  const size_t bh = blockIdx.x;
  const int len = cache_len(p.kv_lens, blockIdx.x / p.H_q, p.n_cap);
  const int ns = (len + p.chunk - 1) / p.chunk;
  const float* lse = p.part_lse + bh * p.n_split;
  const float NEG_INF = -__int_as_float(0x7f800000);
  float M = NEG_INF, L = 0.f, a = 0.f;
  for (int s = 0; s < ns; ++s) M = fmaxf(M, lse[s]);
  for (int s = 0; s < ns; ++s) {
    const float w = exp2f(lse[s] - M);
    L += w;
    a = fmaf(w, p.part_o[(bh * p.n_split + s) * D + threadIdx.x], a);
  }
  p.O[bh * D + threadIdx.x] = __float2bfloat16_rn(ns ? a / L : 0.f);
  if (threadIdx.x == 0) {
    const float l2 = ns ? M + log2f(L) : NEG_INF;
    p.lse2[bh] = l2;
    if (p.LSE) p.LSE[bh] = l2 * 0.69314718055994531f;
  }
}

__global__ void __launch_bounds__(256) sdpa_cache_weights_kernel(const CacheDecodeParams p) {
  const int kvh = blockIdx.y, b = blockIdx.z, j = blockIdx.x * 256 + threadIdx.x;
  if (j >= cache_len(p.kv_lens, b, p.n_cap)) return;
  const size_t head0 = (size_t)b * p.H_q + kvh * p.group;
  float w = 0.f;
  for (int h = 0; h < p.group; ++h) w += exp2f(p.scores[(head0 + h) * p.n_cap + j] - p.lse2[head0 + h]);
  const size_t at = ((size_t)b * p.H_kv + kvh) * p.n_cap + j;
  p.acc_out[at] = (p.acc ? p.acc[at] : 0.f) + w;
}

}  // namespace sdpa
