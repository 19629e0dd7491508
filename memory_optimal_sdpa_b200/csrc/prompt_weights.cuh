// prompt_weights.cuh -- the attention weights of a prompt, summed over its queries.
#pragma once

#include "kv4.cuh"

namespace sdpa {

struct PromptWeightsParams {
  const __nv_bfloat16* Q;  // [B, Hq, n_q, D]
  const __nv_bfloat16* K;  // [B, Hkv, n_kv, D]
  const float* LSE;        // [B, Hq, n_q]
  const float* acc;        // [B, Hkv, n_acc] or null
  float* acc_out;
  int H_q, H_kv, group, n_q, n_kv, n_acc, causal;
  float scale_log2;
};

// One thread per key, query rows staged in shared memory.
template <int D>
__global__ void __launch_bounds__(128) sdpa_prompt_weights_kernel(const PromptWeightsParams p) {
  constexpr int TILE = 32;
  __shared__ float s_q[TILE][D];
  __shared__ float s_lse[TILE];
  const int b = blockIdx.y / p.H_kv, kvh = blockIdx.y % p.H_kv;
  const int j = blockIdx.x * 128 + threadIdx.x;
  const size_t bkv = blockIdx.y;
  float k[D];
  for (int e = 0; e < D; ++e) k[e] = j < p.n_kv ? __bfloat162float(p.K[(bkv * p.n_kv + j) * D + e]) * p.scale_log2 : 0.f;
  float w = 0.f;
  for (int h = 0; h < p.group; ++h) {
    const size_t head = (size_t)b * p.H_q + kvh * p.group + h;
    for (int i0 = 0; i0 < p.n_q; i0 += TILE) {
      const int n = min(TILE, p.n_q - i0);
      __syncthreads();
      for (int i = threadIdx.x; i < n * D; i += 128)
        s_q[i / D][i % D] = __bfloat162float(p.Q[(head * p.n_q + i0) * D + i]);
      if (threadIdx.x < n) s_lse[threadIdx.x] = p.LSE[head * p.n_q + i0 + threadIdx.x];
      __syncthreads();
      float part = 0.f;
      for (int i = 0; i < n; ++i) {
        if (p.causal && j > i0 + i + p.n_kv - p.n_q) continue;
        if (fabsf(s_lse[i]) == __int_as_float(0x7f800000)) continue;
        float d = 0.f;
        for (int e = 0; e < D; ++e) d = fmaf(k[e], s_q[i][e], d);
        part += exp2f(d - s_lse[i] * 1.4426950408889634f);
      }
      w += part;
    }
  }
  if (j < p.n_kv) p.acc_out[bkv * p.n_acc + j] = (p.acc ? p.acc[bkv * p.n_acc + j] : 0.f) + w;
}

}  // namespace sdpa
