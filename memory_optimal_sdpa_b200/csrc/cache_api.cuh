// cache_api.cuh -- the C ABI of include/sdpa_cache.h: argument checks and launches (part of sdpa_api.cu's
// translation unit, whose helpers it uses).
#pragma once

#include <atomic>
#include <type_traits>

#include "sdpa_cache.h"
#include "decode_cache.cuh"
#include "evict.cuh"
#include "kv4.cuh"
#include "prompt_weights.cuh"

namespace {

bool cache_head_dim(int d) { return d == 64 || d == 128; }

// batch, heads and batch * heads * rows within what the kernels index with 32 bits.  They round row numbers up to whole
// blocks of 4096 at most, and step on by one more, before they compare them with a length.
bool cache_sizes_fit(long long batch, long long heads, long long rows) {
  return batch <= 65535 && heads <= 65535 && batch * heads * rows <= (1LL << 31) - 8192;
}

int launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SDPA_OK : cuda_fail(what, e);
}

// A programmatic dependent of the launch before it: its own launch overlaps that one's last wave, and the kernel waits for it
// (cudaGridDependencySynchronize) before it reads anything.
template <class Params>
int launch_dependent(const char* what, void (*kern)(Params), dim3 grid, int threads, cudaStream_t s,
                     const std::remove_const_t<Params>& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  return e == cudaSuccess ? SDPA_OK : cuda_fail(what, e);
}

template <bool LOAD>
int launch_kv4_rows(const sdpa::Kv4RowsParams& p, int d, cudaStream_t s) {
  const long long slots = (long long)p.B * p.H * p.n_rows;
  const int per_block = sdpa::KV4_THREADS / (d / 8) * sdpa::KV4_UNROLL;
  const dim3 grid((unsigned)((slots + per_block - 1) / per_block), 2);
  if (d == 64)
    sdpa::sdpa_kv4_rows_kernel<64, LOAD><<<grid, sdpa::KV4_THREADS, 0, s>>>(p);
  else
    sdpa::sdpa_kv4_rows_kernel<128, LOAD><<<grid, sdpa::KV4_THREADS, 0, s>>>(p);
  return launched(LOAD ? "kv4 load launch" : "kv4 append launch");
}

// Allow `kern` this much dynamic shared memory on the current device, once per device (a bit of `ready` each).
template <class Kernel>
int allow_smem(Kernel kern, int bytes, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (e == cudaSuccess && dev < 64 && (ready.load(std::memory_order_acquire) & bit)) return SDPA_OK;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return cuda_fail("cudaFuncSetAttribute(max dynamic smem, cache)", e);
  ready.fetch_or(bit, std::memory_order_release);
  return SDPA_OK;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  return (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}

// A running sum goes into its own place or elsewhere: an array that overlaps it partly would be read after it was written.
bool sums_fit(const float* acc, const float* acc_out, size_t n) {
  return !acc || acc == acc_out || !overlap(acc, n * sizeof(float), acc_out, n * sizeof(float));
}

bool cache_arrays_aligned(const void* kc, const void* ks, const void* vc, const void* vs) {
  return aligned16(kc) && aligned16(ks) && aligned16(vc) && aligned16(vs);
}

}  // namespace

extern "C" int sdpa_kv4_append(const void* K, const void* V, const int* kv_lens, const int* n_new, void* k_codes,
                               void* k_scales, void* v_codes, void* v_scales, void* k_read, void* v_read, int batch,
                               int heads, int n_rows, int n_kv_cap, int d, void* stream) {
  if (batch < 0 || heads < 0 || n_rows < 0 || n_kv_cap < 1) return SDPA_ERR_INVALID_ARG;
  if (!cache_head_dim(d)) return SDPA_ERR_UNSUPPORTED;
  if (batch == 0 || heads == 0 || n_rows == 0) return SDPA_OK;
  if (!K || !V || !kv_lens || !k_codes || !k_scales || !v_codes || !v_scales || !k_read != !v_read)
    return SDPA_ERR_INVALID_ARG;
  if (!aligned16(K) || !aligned16(V) || !cache_arrays_aligned(k_codes, k_scales, v_codes, v_scales) ||
      !aligned16(k_read) || !aligned16(v_read) || !aligned4(kv_lens) || !aligned4(n_new))
    return SDPA_ERR_MISALIGNED;
  if (!cache_sizes_fit(batch, heads, n_rows) || !cache_sizes_fit(batch, heads, n_kv_cap)) return SDPA_ERR_UNSUPPORTED;
  const size_t bytes = (size_t)batch * heads * n_rows * d * 2;
  for (const void* read : {k_read, v_read})  // the inputs are read through the non-coherent path
    if (read && (overlap(read, bytes, K, bytes) || overlap(read, bytes, V, bytes))) return SDPA_ERR_INVALID_ARG;
  if (k_read && overlap(k_read, bytes, v_read, bytes)) return SDPA_ERR_INVALID_ARG;
  if (int e = check_device()) return e;
  sdpa::Kv4RowsParams p = {};
  p.cache[0] = {(uint8_t*)k_codes, (uint32_t*)k_scales};
  p.cache[1] = {(uint8_t*)v_codes, (uint32_t*)v_scales};
  p.rows[0] = (__nv_bfloat16*)K;
  p.rows[1] = (__nv_bfloat16*)V;
  p.read[0] = (__nv_bfloat16*)k_read;
  p.read[1] = (__nv_bfloat16*)v_read;
  p.kv_lens = kv_lens;
  p.n_new = n_new;
  p.B = batch;
  p.H = heads;
  p.n_rows = n_rows;
  p.n_cap = n_kv_cap;
  p.by_rows = sdpa::FastDiv::of((uint32_t)n_rows);
  p.by_heads = sdpa::FastDiv::of((uint32_t)heads);
  return launch_kv4_rows<false>(p, d, (cudaStream_t)stream);
}

extern "C" int sdpa_kv4_load(const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                             const int* kv_lens, void* K, void* V, int batch, int heads, int n_rows, int n_kv_cap,
                             int d, void* stream) {
  if (batch < 0 || heads < 0 || n_rows < 0 || n_kv_cap < 1) return SDPA_ERR_INVALID_ARG;
  if (!cache_head_dim(d)) return SDPA_ERR_UNSUPPORTED;
  if (batch == 0 || heads == 0 || n_rows == 0) return SDPA_OK;
  if (!K || !V || !kv_lens || !k_codes || !k_scales || !v_codes || !v_scales) return SDPA_ERR_INVALID_ARG;
  if (!aligned16(K) || !aligned16(V) || !cache_arrays_aligned(k_codes, k_scales, v_codes, v_scales) ||
      !aligned4(kv_lens))
    return SDPA_ERR_MISALIGNED;
  if (!cache_sizes_fit(batch, heads, n_rows) || !cache_sizes_fit(batch, heads, n_kv_cap)) return SDPA_ERR_UNSUPPORTED;
  if (int e = check_device()) return e;
  sdpa::Kv4RowsParams p = {};
  p.cache[0] = {(uint8_t*)k_codes, (uint32_t*)k_scales};
  p.cache[1] = {(uint8_t*)v_codes, (uint32_t*)v_scales};
  p.rows[0] = (__nv_bfloat16*)K;
  p.rows[1] = (__nv_bfloat16*)V;
  p.kv_lens = kv_lens;
  p.B = batch;
  p.H = heads;
  p.n_rows = n_rows;
  p.n_cap = n_kv_cap;
  p.by_rows = sdpa::FastDiv::of((uint32_t)n_rows);
  p.by_heads = sdpa::FastDiv::of((uint32_t)heads);
  return launch_kv4_rows<true>(p, d, (cudaStream_t)stream);
}

// ------------------------------------------------------------------ decode over a bounded cache
namespace {

long long cache_score_stride(long long n_cap) { return (n_cap + 3) / 4 * 4; }

// Query heads per unit of work: up to 8, or up to 16 where the group has more.
int cache_unit_heads(int group) { return group > 8 ? 16 : 8; }

// CTAs that share the work: what fits on the 148 SMs of a B200 at once, as workspace sizes have to be known without a GPU.  No CTA
// waits for another, so fewer SMs only take more than one wave.
template <int D, bool KV4, bool WIDE>
constexpr int kCacheCtas = 148 * sdpa::CacheCfg<D, KV4, WIDE>::MIN_BLOCKS;

template <int D, bool KV4>
int cache_ctas_for(bool wide) {
  return wide ? kCacheCtas<D, KV4, true> : kCacheCtas<D, KV4, false>;
}
int cache_ctas(int d, bool kv4, bool wide) {
  if (d == 64) return kv4 ? cache_ctas_for<64, true>(wide) : cache_ctas_for<64, false>(wide);
  return kv4 ? cache_ctas_for<128, true>(wide) : cache_ctas_for<128, false>(wide);
}

// Partial results of the segments (at most one per unit and one more per CTA).
struct CacheParts {
  long long heads, rows;  // query heads per unit; rows of all segments
};
CacheParts cache_parts(long long batch, int heads_q, int heads_kv, int d, bool kv4) {
  const int group = heads_q / heads_kv, rows = cache_unit_heads(group);
  const long long units = batch * heads_kv * ((group + rows - 1) / rows);
  return {rows, (units + cache_ctas(d, kv4, rows == 16)) * rows};
}

// Floats: d outputs, a maximum and a sum per row of the partial results (a multiple of 8 rows), and the scores per (head,
// cache row); then one 64-bit number per sequence and one more.
size_t cache_ws_size(int batch, int heads_q, int heads_kv, int n_cap, int d, bool kv4, bool with_acc) {
  if (batch <= 0 || heads_q <= 0 || heads_kv <= 0 || heads_q % heads_kv != 0 || n_cap <= 0 || !cache_head_dim(d)) return 0;
  const CacheParts parts = cache_parts(batch, heads_q, heads_kv, d, kv4);
  const long long scores = with_acc ? (long long)batch * heads_q * cache_score_stride(n_cap) : 0;
  return (size_t)(parts.rows * (d + 2) + scores) * sizeof(float) + (size_t)(batch + 2) / 2 * 2 * sizeof(long long);
}

template <int D, bool KV4, bool WIDE>
int launch_cache_split(const sdpa::CacheDecodeParams& p, cudaStream_t s) {
  using Cfg = sdpa::CacheCfg<D, KV4, WIDE>;
  auto kern = sdpa::sdpa_cache_split_kernel<D, KV4, WIDE>;
  static std::atomic<uint64_t> ready{0};
  if (int e = allow_smem(kern, Cfg::SMEM_BYTES, ready)) return e;
  kern<<<(unsigned)p.n_cta, Cfg::THREADS, Cfg::SMEM_BYTES, s>>>(p);
  return launched("cache decode launch");
}

template <int D, bool KV4>
int launch_cache_decode(sdpa::CacheDecodeParams p, cudaStream_t s) {
  const bool wide = p.rows == 16;
  p.block = wide ? sdpa::CacheCfg<D, KV4, true>::BLOCK : sdpa::CacheCfg<D, KV4, false>::BLOCK;
  p.n_cta = cache_ctas_for<D, KV4>(wide);
  // no more CTAs than blocks of work in a full cache
  const long long most = (long long)p.B * p.H_kv * p.head_blocks * ((p.n_cap + p.block - 1) / p.block);
  if (most < p.n_cta) p.n_cta = (int)most;
  const int rc = wide ? launch_cache_split<D, KV4, true>(p, s) : launch_cache_split<D, KV4, false>(p, s);
  if (rc != SDPA_OK) return rc;
  const int key_blocks = p.scores ? (p.n_cap + sdpa::CACHE_FINISH_KEYS - 1) / sdpa::CACHE_FINISH_KEYS : 0;
  return launch_dependent("cache decode finish launch", sdpa::sdpa_cache_finish_kernel<D>,
                          dim3((unsigned)(p.head_blocks + key_blocks), (unsigned)p.H_kv, (unsigned)p.B),
                          sdpa::CACHE_FINISH_THREADS, s, p);
}

// The part that both decodes share: p holds the cache; everything else is checked and filled in here.
int cache_decode(sdpa::CacheDecodeParams p, bool kv4, const void* Q, const int* kv_lens, void* O, float* LSE,
                 const float* acc, float* acc_out, int batch, int heads_q, int heads_kv, int n_cap, int d, float scale,
                 void* workspace, size_t workspace_bytes, void* stream) {
  if (!aligned16(Q) || !aligned16(O) || !aligned4(kv_lens) || !aligned4(LSE) || !aligned4(acc) || !aligned4(acc_out))
    return SDPA_ERR_MISALIGNED;
  if (!cache_sizes_fit(batch, heads_q, 1) || !cache_sizes_fit(batch, heads_kv, n_cap)) return SDPA_ERR_UNSUPPORTED;
  if (!sums_fit(acc, acc_out, (size_t)batch * heads_kv * n_cap)) return SDPA_ERR_INVALID_ARG;
  const size_t need = cache_ws_size(batch, heads_q, heads_kv, n_cap, d, kv4, acc_out != nullptr);
  if (!workspace || workspace_bytes < need) return SDPA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return SDPA_ERR_MISALIGNED;
  if (int e = check_device()) return e;
  p.Q = (const __nv_bfloat16*)Q;
  p.kv_lens = kv_lens;
  p.acc = acc;
  p.acc_out = acc_out;
  p.O = (__nv_bfloat16*)O;
  p.LSE = LSE;
  p.H_q = heads_q;
  p.H_kv = heads_kv;
  p.group = heads_q / heads_kv;
  p.n_cap = n_cap;
  const CacheParts parts = cache_parts(batch, heads_q, heads_kv, d, kv4);
  p.B = batch;
  p.rows = (int)parts.heads;
  p.head_blocks = (p.group + p.rows - 1) / p.rows;
  p.score_stride = (int)cache_score_stride(n_cap);
  const float size = std::fabs(scale);
  p.scale_exp = size > 0x1p126f ? 2 : size < 0x1p-100f ? -64 : 0;
  p.scale_log2 = std::ldexp(scale, -p.scale_exp) * 1.4426950408889634f;
  p.part_o = (float*)workspace;
  p.scores = acc_out ? p.part_o + (size_t)parts.rows * d : nullptr;  // 16-byte rows: the stride is a multiple of 4
  p.part_stat = (float2*)(p.part_o + (size_t)parts.rows * d + (acc_out ? (size_t)batch * heads_q * p.score_stride : 0));
  p.seq_at = (long long*)(p.part_stat + parts.rows);
  cudaStream_t s = (cudaStream_t)stream;
  if (d == 64) return kv4 ? launch_cache_decode<64, true>(p, s) : launch_cache_decode<64, false>(p, s);
  return kv4 ? launch_cache_decode<128, true>(p, s) : launch_cache_decode<128, false>(p, s);
}

}  // namespace

extern "C" size_t sdpa_decode_kv4_workspace_size(int batch, int heads_q, int heads_kv, int n_kv_cap, int d, int with_acc) {
  return cache_ws_size(batch, heads_q, heads_kv, n_kv_cap, d, true, with_acc != 0);
}

extern "C" size_t sdpa_decode_acc_workspace_size(int batch, int heads_q, int heads_kv, int n_kv_cap, int d) {
  return cache_ws_size(batch, heads_q, heads_kv, n_kv_cap, d, false, true);
}

extern "C" int sdpa_decode_kv4(const void* Q, const void* k_codes, const void* k_scales, const void* v_codes,
                               const void* v_scales, const int* kv_lens, void* O, float* LSE, const float* acc,
                               float* acc_out, int batch, int heads_q, int heads_kv, int n_kv_cap, int d, float scale,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (batch < 0 || heads_q < 0 || heads_kv < 1 || n_kv_cap < 1 || heads_q % heads_kv != 0 || !std::isfinite(scale))
    return SDPA_ERR_INVALID_ARG;
  if (!cache_head_dim(d)) return SDPA_ERR_UNSUPPORTED;
  if (batch == 0 || heads_q == 0) return SDPA_OK;
  if (!Q || !k_codes || !k_scales || !v_codes || !v_scales || !kv_lens || !O || (acc && !acc_out))
    return SDPA_ERR_INVALID_ARG;
  if (!cache_arrays_aligned(k_codes, k_scales, v_codes, v_scales)) return SDPA_ERR_MISALIGNED;
  sdpa::CacheDecodeParams p = {};
  p.cache[0] = {(uint8_t*)k_codes, (uint32_t*)k_scales};
  p.cache[1] = {(uint8_t*)v_codes, (uint32_t*)v_scales};
  return cache_decode(p, true, Q, kv_lens, O, LSE, acc, acc_out, batch, heads_q, heads_kv, n_kv_cap, d, scale, workspace,
                      workspace_bytes, stream);
}

extern "C" int sdpa_decode_acc(const void* Q, const void* K, const void* V, const int* kv_lens, void* O, float* LSE,
                               const float* acc, float* acc_out, int batch, int heads_q, int heads_kv, int n_kv_cap,
                               int d, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  if (batch < 0 || heads_q < 0 || heads_kv < 1 || n_kv_cap < 1 || heads_q % heads_kv != 0 || !std::isfinite(scale))
    return SDPA_ERR_INVALID_ARG;
  if (!cache_head_dim(d)) return SDPA_ERR_UNSUPPORTED;
  if (batch == 0 || heads_q == 0) return SDPA_OK;
  if (!Q || !K || !V || !kv_lens || !O || !acc_out) return SDPA_ERR_INVALID_ARG;
  if (!aligned16(K) || !aligned16(V)) return SDPA_ERR_MISALIGNED;
  sdpa::CacheDecodeParams p = {};
  p.kv[0] = (const __nv_bfloat16*)K;
  p.kv[1] = (const __nv_bfloat16*)V;
  return cache_decode(p, false, Q, kv_lens, O, LSE, acc, acc_out, batch, heads_q, heads_kv, n_kv_cap, d, scale,
                      workspace, workspace_bytes, stream);
}

// ------------------------------------------------------------------ weights of a prompt
namespace {

// Units of 256 keys unless the heaviest one, which sees all queries, is more than 15 % above an SM's share of the 128 x 128
// tiles: then of 128 (both measured at the head of prompt_weights.cuh).
bool prompt_wide(const sdpa::PromptWeightsParams& p) {
  const long long n_kt = (p.n_kv + 127) / 128, n_qt = (p.n_q + 127) / 128;
  long long tiles = n_kt * n_qt;  // of a head
  if (p.causal) {                 // key tile k loses max(0, k - k0) query tiles
    const long long off = (long long)p.n_kv - p.n_q, k0 = off >= 0 ? (off + 127) / 128 : -(-off / 128);
    const long long most = n_kt - 1 - k0, least = k0 < 0 ? -k0 : 0;
    if (most > 0) tiles -= (most * (most + 1) - least * (least - 1)) / 2;
  }
  return 2.0 * (double)n_qt * sm_count() <= 1.15 * (double)tiles * p.bkv;
}

template <int D, int MT>
int launch_prompt_weights(const void* Q, const void* K, sdpa::PromptWeightsParams p, int batch, cudaStream_t stream) {
  using Cfg = sdpa::PromptCfg<D, MT>;
  auto kern = sdpa::sdpa_prompt_weights_kernel<D, MT>;
  static std::atomic<uint64_t> ready{0};
  if (int e = allow_smem(kern, Cfg::SMEM_BYTES, ready)) return e;
  CUtensorMap mq, mk;
  if (!make_map(&mk, K, D, p.n_kv, p.bkv)) return SDPA_ERR_CUDA;
  if (p.n_q == 0)
    mq = mk;  // not read
  else if (!make_map(&mq, Q, D, p.n_q, batch * p.heads_q))
    return SDPA_ERR_CUDA;
  p.n_kt = (p.n_kv + 128 * MT - 1) / (128 * MT);
  long long grid = (long long)p.bkv * p.n_kt;
  if (grid > sm_count()) grid = sm_count();
  kern<<<(unsigned)grid, Cfg::THREADS, Cfg::SMEM_BYTES, stream>>>(mq, mk, p);
  return launched("prompt weights launch");
}

}  // namespace

extern "C" int sdpa_fwd_acc(const void* Q, const void* K, const float* LSE, const float* acc, float* acc_out, int batch,
                            int heads_q, int heads_kv, int n_q, int n_kv, int n_acc, int d, float scale, int causal,
                            void* stream) {
  if (batch < 0 || heads_q < 0 || heads_kv < 1 || n_q < 0 || n_kv < 1 || n_acc < n_kv || (causal != 0 && causal != 1) ||
      heads_q % heads_kv != 0 || !std::isfinite(scale))
    return SDPA_ERR_INVALID_ARG;
  if (!cache_head_dim(d)) return SDPA_ERR_UNSUPPORTED;
  if (batch == 0 || heads_q == 0) return SDPA_OK;
  if (!K || !acc_out || (n_q > 0 && (!Q || !LSE))) return SDPA_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned4(LSE) || !aligned4(acc) || !aligned4(acc_out)) return SDPA_ERR_MISALIGNED;
  if (!cache_sizes_fit(batch, heads_q, n_q) || !cache_sizes_fit(batch, heads_kv, n_acc)) return SDPA_ERR_UNSUPPORTED;
  if (!sums_fit(acc, acc_out, (size_t)batch * heads_kv * n_acc)) return SDPA_ERR_INVALID_ARG;
  if (int e = check_device()) return e;
  sdpa::PromptWeightsParams p = {};
  p.LSE = LSE;
  p.acc = acc;
  p.acc_out = acc_out;
  p.heads_q = heads_q;
  p.heads_kv = heads_kv;
  p.group = heads_q / heads_kv;
  p.n_q = n_q;
  p.n_kv = n_kv;
  p.n_acc = n_acc;
  p.causal = causal;
  p.bkv = batch * heads_kv;
  p.quarter = std::fabs(scale) > 0x1p126f;
  p.scale_log2 = (p.quarter ? 0.25f * scale : scale) * 1.4426950408889634f;
  cudaStream_t s = (cudaStream_t)stream;
  const bool wide = prompt_wide(p);
  if (d == 64) return wide ? launch_prompt_weights<64, 2>(Q, K, p, batch, s) : launch_prompt_weights<64, 1>(Q, K, p, batch, s);
  return wide ? launch_prompt_weights<128, 2>(Q, K, p, batch, s) : launch_prompt_weights<128, 1>(Q, K, p, batch, s);
}

// ------------------------------------------------------------------ eviction
namespace {

struct EvictArray {
  const void* in;
  void* out;
  size_t row_bytes;
};

// arrays[0 .. n) are the cache's rows; the weights are added here.
int evict(const EvictArray* arrays, int n, const float* acc, const int* kv_lens, float* acc_out, int* keep,
          int* new_lens, int batch, int heads, int n_cap, int n_out, int budget, int recent, void* stream) {
  const size_t bh = (size_t)batch * heads;
  EvictArray all[5];
  for (int i = 0; i < n; ++i) all[i] = arrays[i];
  all[n] = {acc, acc_out, 4};
  for (int i = 0; i <= n; ++i) {
    if (!all[i].in || !all[i].out) return SDPA_ERR_INVALID_ARG;
    if (i < n ? !aligned16(all[i].in) || !aligned16(all[i].out) : !aligned4(acc) || !aligned4(acc_out))
      return SDPA_ERR_MISALIGNED;
  }
  if (!kv_lens || !keep || !new_lens) return SDPA_ERR_INVALID_ARG;
  if (!aligned4(kv_lens) || !aligned4(keep) || !aligned4(new_lens)) return SDPA_ERR_MISALIGNED;
  if (!cache_sizes_fit(batch, heads, n_cap) || !cache_sizes_fit(batch, heads, n_out)) return SDPA_ERR_UNSUPPORTED;
  const struct {
    const void* at;
    size_t bytes;
  } results[2] = {{keep, bh * budget * 4}, {new_lens, (size_t)batch * 4}};
  for (const auto& r : results) {  // they overlap nothing
    if (overlap(r.at, r.bytes, kv_lens, (size_t)batch * 4)) return SDPA_ERR_INVALID_ARG;
    for (int i = 0; i <= n; ++i)
      if (overlap(r.at, r.bytes, all[i].in, bh * n_cap * all[i].row_bytes) ||
          overlap(r.at, r.bytes, all[i].out, bh * n_out * all[i].row_bytes))
        return SDPA_ERR_INVALID_ARG;
  }
  if (overlap(keep, results[0].bytes, new_lens, results[1].bytes)) return SDPA_ERR_INVALID_ARG;
  for (int i = 0; i <= n; ++i)  // an output is its own input or apart from every input and output
    for (int j = 0; j <= n; ++j) {
      const bool in_place = i == j && all[i].in == all[i].out && n_out == n_cap;
      if (!in_place && overlap(all[i].out, bh * n_out * all[i].row_bytes, all[j].in, bh * n_cap * all[j].row_bytes))
        return SDPA_ERR_INVALID_ARG;
      if (i != j && overlap(all[i].out, bh * n_out * all[i].row_bytes, all[j].out, bh * n_out * all[j].row_bytes))
        return SDPA_ERR_INVALID_ARG;
    }
  if (int e = check_device()) return e;
  cudaStream_t s = (cudaStream_t)stream;
  sdpa::EvictParams p = {acc, acc_out, kv_lens, keep, new_lens, heads, n_cap, n_out, budget, recent};
  if (n_cap <= sdpa::EVICT_CACHED) {
    static std::atomic<uint64_t> ready{0};
    if (int e = allow_smem(sdpa::sdpa_evict_select_kernel<true>, sdpa::EVICT_CACHED * 4, ready)) return e;
    sdpa::sdpa_evict_select_kernel<true><<<(unsigned)bh, sdpa::EVICT_THREADS, (size_t)n_cap * 4, s>>>(p);
  } else {
    sdpa::sdpa_evict_select_kernel<false><<<(unsigned)bh, sdpa::EVICT_THREADS, 0, s>>>(p);
  }
  if (int e = launched("evict select launch")) return e;
  // Arrays in place and arrays that go elsewhere (a caller may mix them).
  for (int in_place = 0; in_place < 2; ++in_place) {
    sdpa::EvictRowsParams r = {};
    int k = 0;
    size_t largest = 0;
    for (int i = 0; i < n; ++i) {
      if ((arrays[i].in == arrays[i].out) != (in_place == 1)) continue;
      r.src[k] = (const uint8_t*)arrays[i].in;
      r.dst[k] = (uint8_t*)arrays[i].out;
      r.row_bytes[k++] = (int)arrays[i].row_bytes;
      if (arrays[i].row_bytes > largest) largest = arrays[i].row_bytes;
    }
    if (k == 0) continue;
    r.keep = keep;
    r.kv_lens = kv_lens;
    r.H = heads;
    r.n_cap = n_cap;
    r.n_out = n_out;
    r.budget = budget;
    r.n_bh = (int)bh;
    if (in_place) {
      const dim3 grid((unsigned)bh, (unsigned)((largest + 63) / 64), (unsigned)k);
      if (int e = launch_dependent("evict rows launch", sdpa::sdpa_evict_rows_in_place_kernel, grid, sdpa::EVICT_ROW_THREADS, s, r))
        return e;
    } else {
      // four blocks an SM in all, no more than stretches of the array with the longest rows
      const long long rows = sdpa::EVICT_ROW_THREADS * sdpa::EVICT_ROW_UNROLL * 16 / (long long)largest;
      long long blocks = (budget + rows - 1) / rows * (long long)bh;
      if (blocks > 148 * 4 / k) blocks = 148 * 4 / k;
      if (int e = launch_dependent("evict rows launch", sdpa::sdpa_evict_rows_kernel, dim3((unsigned)blocks, (unsigned)k),
                                   sdpa::EVICT_ROW_THREADS, s, r))
        return e;
    }
  }
  return SDPA_OK;
}

int evict_sizes(int batch, int heads, int n_cap, int n_out, int d, int budget, int recent) {
  if (batch < 0 || heads < 0 || n_cap < 1 || n_out < 1 || budget < 1 || budget > n_out || recent < 0 || recent > budget)
    return SDPA_ERR_INVALID_ARG;
  return cache_head_dim(d) ? SDPA_OK : SDPA_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" int sdpa_evict(const void* K, const void* V, const float* acc, const int* kv_lens, void* K_out, void* V_out,
                          float* acc_out, int* keep, int* new_lens, int batch, int heads, int n_kv_cap, int n_out_cap,
                          int d, int budget, int recent, void* stream) {
  if (int e = evict_sizes(batch, heads, n_kv_cap, n_out_cap, d, budget, recent)) return e;
  if (batch == 0 || heads == 0) return SDPA_OK;
  const EvictArray a[2] = {{K, K_out, (size_t)d * 2}, {V, V_out, (size_t)d * 2}};
  return evict(a, 2, acc, kv_lens, acc_out, keep, new_lens, batch, heads, n_kv_cap, n_out_cap, budget, recent, stream);
}

extern "C" int sdpa_kv4_evict(const void* k_codes, const void* k_scales, const void* v_codes, const void* v_scales,
                              const float* acc, const int* kv_lens, void* k_codes_out, void* k_scales_out,
                              void* v_codes_out, void* v_scales_out, float* acc_out, int* keep, int* new_lens,
                              int batch, int heads, int n_kv_cap, int n_out_cap, int d, int budget, int recent,
                              void* stream) {
  if (int e = evict_sizes(batch, heads, n_kv_cap, n_out_cap, d, budget, recent)) return e;
  if (batch == 0 || heads == 0) return SDPA_OK;
  const size_t codes = (size_t)d / 2, scales = (size_t)d / 8;
  const EvictArray a[4] = {{k_codes, k_codes_out, codes},
                           {k_scales, k_scales_out, scales},
                           {v_codes, v_codes_out, codes},
                           {v_scales, v_scales_out, scales}};
  return evict(a, 4, acc, kv_lens, acc_out, keep, new_lens, batch, heads, n_kv_cap, n_out_cap, budget, recent, stream);
}
