// decode_cache.cuh -- one query row per head against a bounded cache: bf16 or 4-bit rows, with the
// attention weights of every key added to an accumulator where asked for.
//
// CTA (split s, key/value head and block of its query heads, b) reduces keys [s chunk, s chunk + chunk) of
// the valid prefix to a normalised partial output and a log-sum-exp (base 2) per query head.  With weights
// it also writes the scores (base 2, fp32): a key's weight needs the log-sum-exp over all splits, and 4
// bytes a score, written and read once, cost far less than reading the keys again.
// sdpa_cache_finish_kernel joins the splits and adds sum_h 2^(score_h - LSE_h) per key.
//
// What bounds it: HBM, if the arithmetic fits under it.  A 4-bit row pair of d = 128 is 160 bytes, 6.9 clocks of an
// SM's share of HBM, in which 256 codes have to become operands.  So the codes never leave registers:
// mma.sync takes its B operand from the registers they were unpacked in, where tcgen05 would need them
// written to shared memory as 16-bit numbers and read back (512 + 512 bytes, 8 clocks).  Measured on this
// part: m16n8k16 one per 2.1 clocks (two a key here), integer operations two warp instructions a clock.
//
// Unpacking: (w & 0x000F000F) is, read as two fp16 numbers, c 2^-24 exactly (subnormal), and
// (w & 0x00F000F0) 16 c 2^-24: one integer operation gives two operands.  The powers of two are put back
// with the group scales.  For that Q enters as fp16, normalised by a power of two per head so that its
// largest element is near 2^14 (the 8 significant bits of bf16 fit in fp16's 11; elements 2^-28 times the
// largest and smaller lose bits, far below the rounding of the 32-bit sums).
//   scores   S[h, j] = sum_g s_jg (sum_{i in g} q_hi c_ji) + m_jg (sum_{i in g} q_hi)
//   output   O[h, i] = sum_j (p_hj s_jg) c_ji + sum_j p_hj m_jg          (g the group of channel i)
// p s is rounded to fp16 (half a step: 2^-12 of it, a sixteenth of the rounding of O to bf16), scaled by a power of
// two that keeps it in range; the sums with m and everything else stay in fp32.
// bf16 caches use the same kernel with bf16 products; there p is split in two bf16 parts (its rounding to one
// would cost as much again as that of O).
//
// Each warp streams tiles of its own (cp.async, two or three tiles in flight, no barrier between warps) with an
// online softmax of its own; the four warps of a CTA are joined at its end.  The softmax reference moves
// only when a score exceeds it by more than 4 (a factor 16).
#pragma once

#include <cuda_fp16.h>

#include "kv4.cuh"

namespace sdpa {

struct CacheDecodeParams {
  const __nv_bfloat16* Q;       // [B, Hq, D]
  const __nv_bfloat16* rows[2]; // bf16 cache K, V
  Kv4Cache cache[2];            // or 4-bit cache K, V
  const int* kv_lens;
  float* part_o;    // [B, Hq, S, D]
  float* part_lse;  // [B, Hq, S], base 2
  float* scores;    // [B, Hq, score_stride], base 2, or null
  const float* acc;
  float* acc_out;   // [B, Hkv, n_cap]
  __nv_bfloat16* O;
  float* LSE;
  int H_q, H_kv, group, n_cap, chunk, n_split;
  int score_stride;  // n_cap rounded up to 4
  float scale_log2;
};

// WIDE: 9 to 16 query heads per CTA, else up to 8.  The MMA has 16 rows either way.
template <int D, bool KV4, bool WIDE>
struct CacheCfg {
  static constexpr int WARPS = 4;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int ROWS = WIDE ? 16 : 8;         // query heads
  static constexpr int TILE = KV4 ? 32 : 16;         // keys per warp tile
  static constexpr int STAGES = 3;
  static constexpr int ROW_BYTES = KV4 ? D / 2 : 2 * D;
  static constexpr int HALF_BYTES = TILE * ROW_BYTES;  // K or V of a tile
  static constexpr int STAGE_BYTES = 2 * HALF_BYTES;
  static constexpr int NG = D / 32;
  static constexpr int SCALE_BYTES = KV4 ? 4 * TILE * NG * 4 : 0;  // s and m of K and V, as fp32
  static constexpr int WARP_BYTES = STAGES * STAGE_BYTES + SCALE_BYTES;
  static constexpr int JOIN_BYTES = (ROWS * D + 2 * ROWS) * 4;  // a warp's O, m, l (over the stages)
  static constexpr int SMEM_BYTES = WARPS * (WARP_BYTES > JOIN_BYTES ? WARP_BYTES : JOIN_BYTES);
  static constexpr int MIN_BLOCKS = WIDE ? 2 : (KV4 ? 3 : 2);
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// C += A B, m16n8k16, fp32 accumulation.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <class T>
__device__ __forceinline__ T lds(uint32_t addr);
template <>
__device__ __forceinline__ uint32_t lds<uint32_t>(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
template <>
__device__ __forceinline__ uint2 lds<uint2>(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
template <>
__device__ __forceinline__ uint4 lds<uint4>(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, float x, float y, float z, float w) {
  asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}
// 2^e as a float, e clamped to the normal range.
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23); }

// ------------------------------------------------------------------------------------------ operands
// A fragments of Q.  4-bit: per group g and step st (channels i = 2 st, 2 st + 1 of the pieces), the pairs
// (32 g + 8 t + i, 32 g + 8 t + 4 + i), those of odd i divided by 16; see the file's head.
template <int D, bool KV4, bool WIDE>
struct CacheQuery {
  static constexpr int NG = D / 32, NR = WIDE ? 2 : 1;
  uint32_t a[D / 16][2 * NR];  // a0, a2 (row r), then a1, a3 (row r + 8)
  float sum[NR][KV4 ? NG : 1]; // group sums of the normalised q, times 2^-24
  float norm[NR];              // what scores are multiplied by at the end (a power of two)

  __device__ __forceinline__ void load(const __nv_bfloat16* q, int heads, int lane) {
    const int r = lane >> 2, t = lane & 3;
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      const bool on = r + 8 * x < heads;
      const __nv_bfloat16* row = q + (size_t)(r + 8 * x) * D;
      if constexpr (KV4) {
        float f[NG][8], big = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint4 raw = on ? *reinterpret_cast<const uint4*>(row + 32 * g + 8 * t) : make_uint4(0, 0, 0, 0);
          bf16x8_to_f32(raw, f[g]);
#pragma unroll
          for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(f[g][i]));
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // largest element in [2^14, 2^15); a zero row keeps its (irrelevant) factor
        const int e = (int)(__float_as_uint(big) >> 23) - 127;
        const float up = exp2_int((14 - e) / 2), up2 = exp2_int(14 - e - (14 - e) / 2);  // two exact steps: 2^(14 - e) itself may overflow
        norm[x] = exp2_int(min(e, 126) - 2);
        if (e < -124) norm[x] = 0x1p-126f * exp2_int(e + 124);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float total = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            f[g][i] = f[g][i] * up * up2;
            total += f[g][i];
          }
          total += __shfl_xor_sync(0xffffffffu, total, 1);
          total += __shfl_xor_sync(0xffffffffu, total, 2);
          sum[x][g] = total * 0x1p-24f;
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            a[2 * g + st][2 * x] = pack_f16x2(f[g][2 * st], f[g][4 + 2 * st]);
            a[2 * g + st][2 * x + 1] = pack_f16x2(f[g][2 * st + 1] * 0.0625f, f[g][5 + 2 * st] * 0.0625f);
          }
        }
      } else {
        norm[x] = 1.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          a[k][2 * x] = on ? *reinterpret_cast<const uint32_t*>(row + 16 * k + 2 * t) : 0u;
          a[k][2 * x + 1] = on ? *reinterpret_cast<const uint32_t*>(row + 16 * k + 8 + 2 * t) : 0u;
        }
      }
    }
  }
  __device__ __forceinline__ uint32_t a1(int k) const { return WIDE ? a[k][2 * (NR - 1)] : 0u; }
  __device__ __forceinline__ uint32_t a3(int k) const { return WIDE ? a[k][2 * (NR - 1) + 1] : 0u; }
};

// Shared-memory place (byte) of 16-byte granule gi of a K or V tile, swizzled so that the reads below meet
// every bank once.  4-bit: 128-byte lines of several rows, granule XOR twice the line's number; bf16: granule
// XOR the row's number within its row.
template <int D, bool KV4>
__device__ __forceinline__ int cache_granule(int gi) {
  if (KV4) {
    const int line = gi >> 3;
    return (line << 7) | (((gi & 7) ^ (2 * (line & (D == 128 ? 3 : 1)))) << 4);
  }
  constexpr int GPR = D / 8;
  const int row = gi / GPR;
  return row * (2 * D) + (((gi % GPR) ^ (row & 7)) << 4);
}

template <int D, bool KV4, bool WIDE>
__global__ void __launch_bounds__(CacheCfg<D, KV4, WIDE>::THREADS, CacheCfg<D, KV4, WIDE>::MIN_BLOCKS)
    sdpa_cache_split_kernel(const CacheDecodeParams p) {
  using C = CacheCfg<D, KV4, WIDE>;
  constexpr int NG = C::NG, NR = WIDE ? 2 : 1, NT = C::TILE / 8;  // NT: 8-key tiles of scores
  constexpr int CG = D / 8;                                        // 8-channel tiles of outputs
  const float NEG_INF = -__int_as_float(0x7f800000);
  const int hb = (p.group + C::ROWS - 1) / C::ROWS;
  const int s = blockIdx.x, kvh = blockIdx.y / hb, h0 = (blockIdx.y % hb) * C::ROWS, b = blockIdx.z;
  const int heads = min(C::ROWS, p.group - h0);
  const int len = cache_len(p.kv_lens, b, p.n_cap);
  const int k0 = s * p.chunk;
  if (k0 >= len) return;
  const int n = min(p.chunk, len - k0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
  const size_t row0 = ((size_t)b * p.H_kv + kvh) * p.n_cap + k0;
  const size_t head0 = (size_t)b * p.H_q + (size_t)kvh * p.group + h0;

  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t stage0 = sm100::smem_u32(smem) + warp * C::WARP_BYTES;
  const uint32_t scales0 = stage0 + C::STAGES * C::STAGE_BYTES;

  const uint8_t* src[2];
#pragma unroll
  for (int x = 0; x < 2; ++x)
    src[x] = (KV4 ? p.cache[x].codes : reinterpret_cast<const uint8_t*>(p.rows[x])) + row0 * C::ROW_BYTES;

  const int n_tiles = (n + C::TILE - 1) / C::TILE;
  auto fetch = [&](int tile, int stage) {
    if (tile < n_tiles) {
      const int left = n - tile * C::TILE;
      const size_t at = (size_t)tile * C::HALF_BYTES;
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < C::HALF_BYTES / 512; ++i) {
          const int gi = i * 32 + lane;
          const bool on = gi / (C::ROW_BYTES / 16) < left;  // rows past the length read as zeros
          cp_async16(stage0 + stage * C::STAGE_BYTES + x * C::HALF_BYTES + cache_granule<D, KV4>(gi),
                     src[x] + (on ? at + gi * 16 : 0), on);
        }
    }
    cp_async_commit();
  };
  // 4-bit: a lane holds the scales of one key of the coming tile, K's then V's.
  using Raw = typename std::conditional<D == 128, uint4, uint2>::type;
  Raw raw[2];
  auto fetch_scales = [&](int tile) {
    if constexpr (KV4) {
      const int j = tile * C::TILE + lane;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        Raw v = {};
        if (j < n) v = __ldg(reinterpret_cast<const Raw*>(p.cache[x].scales + (row0 + j) * NG));
        raw[x] = v;
      }
    }
  };

#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) fetch(warp + i * C::WARPS, i);
  fetch_scales(warp);

  CacheQuery<D, KV4, WIDE> q;
  q.load(p.Q + head0 * D, heads, lane);
  const float c2 = KV4 ? p.scale_log2 * 0x1p12f : p.scale_log2;  // 4-bit: 2^24 2^(e - 14) = 2^12 norm

  float m_ref[NR], l[NR], om[NR][KV4 ? NG : 1], o[CG][4];
#pragma unroll
  for (int x = 0; x < NR; ++x) {
    m_ref[x] = NEG_INF;
    l[x] = 0.f;
#pragma unroll
    for (int g = 0; g < (KV4 ? NG : 1); ++g) om[x][g] = 0.f;
  }
#pragma unroll
  for (int c = 0; c < CG; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) o[c][i] = 0.f;
  int f_exp = 1000;  // 4-bit: p s is multiplied by 2^f_exp (1000: not chosen yet)
  float f = 0.f;

  int stage = 0;
  for (int tile = warp; tile < n_tiles; tile += C::WARPS) {
    cp_async_wait<C::STAGES - 2>();
    if constexpr (KV4) {
      __syncwarp();  // the last tile's scales have been read
      // The scales as fp32 for the whole warp: [key pair][group][2] for each of K's s, K's m, V's s, V's m.
      const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&raw[0]);
      const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&raw[1]);
      uint32_t top = 0;  // the largest V scale
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t sb = w1[g] & 0xFFFFu;
        top = max(top, sb <= 0x7F80u ? sb : 0u);  // NaN scales do not count
      }
      const bool grow = f_exp == 1000 || bf16_bits_to_float(top) * f >= 0x1p11f;
      if (__any_sync(0xffffffffu, grow)) {
        const int e = (int)(__reduce_max_sync(0xffffffffu, top) >> 7) - 127;
        const int f_new = min(9 - e, 126);
        if (f_exp != 1000) {
          const float down = exp2_int(f_new - f_exp) * (f_new - f_exp < -126 ? 0.f : 1.f);
#pragma unroll
          for (int c = 0; c < CG; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[c][i] *= down;
        }
        f_exp = f_new;
        f = exp2_int(f_exp);
      }
      const bool odd = lane & 1;
      const uint32_t to = scales0 + (uint32_t)((lane >> 1) * NG * 8 + (odd ? NG * 4 : 0));
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t* w = x ? w1 : w0;
        // even lanes take the first half of the groups of both keys, odd lanes the second
        uint32_t mine[NG / 2], other[NG / 2];
#pragma unroll
        for (int g = 0; g < NG / 2; ++g) {
          const uint32_t give = odd ? w[g] : w[NG / 2 + g];
          mine[g] = odd ? w[NG / 2 + g] : w[g];
          other[g] = __shfl_xor_sync(0xffffffffu, give, 1);
        }
        float sv[NG], mv[NG];  // (group, key of the pair)
#pragma unroll
        for (int g = 0; g < NG / 2; ++g) {
          const uint32_t lo = odd ? other[g] : mine[g], hi = odd ? mine[g] : other[g];
          const float k = x ? f : 1.f;
          sv[2 * g] = __uint_as_float(lo << 16) * k;
          sv[2 * g + 1] = __uint_as_float(hi << 16) * k;
          mv[2 * g] = __uint_as_float(lo & 0xFFFF0000u);
          mv[2 * g + 1] = __uint_as_float(hi & 0xFFFF0000u);
        }
        const uint32_t at = to + x * 2 * (C::TILE * NG * 4);
        if constexpr (NG == 4) {
          sts128(at, sv[0], sv[1], sv[2], sv[3]);
          sts128(at + C::TILE * NG * 4, mv[0], mv[1], mv[2], mv[3]);
        } else {
          asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(at), "f"(sv[0]), "f"(sv[1]) : "memory");
          asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(at + C::TILE * NG * 4), "f"(mv[0]), "f"(mv[1]) : "memory");
        }
      }
    }
    __syncwarp();
    fetch(tile + (C::STAGES - 1) * C::WARPS, stage == 0 ? C::STAGES - 1 : stage - 1);
    if (tile + C::WARPS < n_tiles) fetch_scales(tile + C::WARPS);
    const uint32_t sK = stage0 + stage * C::STAGE_BYTES, sV = sK + C::HALF_BYTES;
    stage = stage == C::STAGES - 1 ? 0 : stage + 1;

    // ---------------------------------------------------------------- scores, base 2
    float sc[NT][2 * NR];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (KV4) {
        const int row = nt * 8 + r;
        uint32_t w[NG];  // pieces of groups (0, 1), (2, 3) of chunk 2 t, then of chunk 2 t + 1
        if constexpr (D == 128) {
          const uint4 v = lds<uint4>(sK + cache_granule<D, KV4>(row * 4 + t));
          w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
          const uint2 v = lds<uint2>(sK + cache_granule<D, KV4>(row * 2 + (t >> 1)) + (t & 1) * 8);
          w[0] = v.x, w[1] = v.y;
        }
        const uint32_t sat = scales0 + (uint32_t)((nt * 4 + t) * NG * 8);
        float2 sum[NR];
#pragma unroll
        for (int x = 0; x < NR; ++x) sum[x] = make_float2(0.f, 0.f);
#pragma unroll
        for (int g2 = 0; g2 < NG / 2; ++g2) {
          const uint4 ss = lds<uint4>(sat + g2 * 16), mm = lds<uint4>(sat + C::TILE * NG * 4 + g2 * 16);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int g = 2 * g2 + y;
            const uint32_t u = __byte_perm(w[g2], w[NG / 2 + g2], y ? 0x7632 : 0x5410), u8 = u >> 8;
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            mma16816<true>(c, q.a[2 * g][0], q.a1(2 * g), q.a[2 * g][1], q.a3(2 * g), u & 0x000F000Fu, u & 0x00F000F0u);
            mma16816<true>(c, q.a[2 * g + 1][0], q.a1(2 * g + 1), q.a[2 * g + 1][1], q.a3(2 * g + 1), u8 & 0x000F000Fu,
                           u8 & 0x00F000F0u);
            const float2 s2 = make_float2(__uint_as_float(y ? ss.z : ss.x), __uint_as_float(y ? ss.w : ss.y));
            const float2 m2 = make_float2(__uint_as_float(y ? mm.z : mm.x), __uint_as_float(y ? mm.w : mm.y));
#pragma unroll
            for (int x = 0; x < NR; ++x) {
              sum[x] = sm100::ffma2(s2, make_float2(c[2 * x], c[2 * x + 1]), sum[x]);
              sum[x] = sm100::ffma2(m2, make_float2(q.sum[x][g], q.sum[x][g]), sum[x]);
            }
          }
        }
#pragma unroll
        for (int x = 0; x < NR; ++x) {
          sc[nt][2 * x] = sum[x].x * c2 * q.norm[x];
          sc[nt][2 * x + 1] = sum[x].y * c2 * q.norm[x];
        }
      } else {
        float c[4] = {0.f, 0.f, 0.f, 0.f};
        const int row = nt * 8 + (lane & 7);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint32_t bfrag[4];
          ldmatrix4<false>(bfrag, sK + cache_granule<D, KV4>(row * (D / 8) + 4 * k + (lane >> 3)));
          mma16816<false>(c, q.a[2 * k][0], q.a1(2 * k), q.a[2 * k][1], q.a3(2 * k), bfrag[0], bfrag[1]);
          mma16816<false>(c, q.a[2 * k + 1][0], q.a1(2 * k + 1), q.a[2 * k + 1][1], q.a3(2 * k + 1), bfrag[2], bfrag[3]);
        }
#pragma unroll
        for (int i = 0; i < 2 * NR; ++i) sc[nt][i] = c[i] * c2;
      }
    }
    if (p.scores) {
#pragma unroll
      for (int x = 0; x < NR; ++x)
        if (r + 8 * x < heads) {
          float* to = p.scores + (head0 + r + 8 * x) * p.score_stride + k0 + tile * C::TILE + 2 * t;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            if (tile * C::TILE + nt * 8 + 2 * t < n)  // the stride leaves room for the pair
              *reinterpret_cast<float2*>(to + nt * 8) = make_float2(sc[nt][2 * x], sc[nt][2 * x + 1]);
        }
    }
    if ((tile + 1) * C::TILE > n) {  // the last tile: keys past the length
      const int left = n - tile * C::TILE;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2 * NR; ++i)
          if (nt * 8 + 2 * t + (i & 1) >= left) sc[nt][i] = NEG_INF;
    }

    // ---------------------------------------------------------------- online softmax
    float mt[NR];
    bool move = false;
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      mt[x] = NEG_INF;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mt[x] = sm100::max3f(mt[x], sc[nt][2 * x], sc[nt][2 * x + 1]);
      mt[x] = fmaxf(mt[x], __shfl_xor_sync(0xffffffffu, mt[x], 1));
      mt[x] = fmaxf(mt[x], __shfl_xor_sync(0xffffffffu, mt[x], 2));
      move |= mt[x] > m_ref[x] + 4.f;
    }
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int x = 0; x < NR; ++x) {
        const float mn = fmaxf(m_ref[x], mt[x]);
        const float alpha = m_ref[x] == NEG_INF ? 0.f : sm100::ex2_approx(m_ref[x] - mn);
        m_ref[x] = mn;
        l[x] *= alpha;
#pragma unroll
        for (int g = 0; g < (KV4 ? NG : 1); ++g) om[x][g] *= alpha;
#pragma unroll
        for (int c = 0; c < CG; ++c) {
          o[c][2 * x] *= alpha;
          o[c][2 * x + 1] *= alpha;
          if (!WIDE && !KV4) {  // rows 8 .. 15 hold the second parts of the same heads
            o[c][2] *= alpha;
            o[c][3] *= alpha;
          }
        }
      }
    }
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      const float m = m_ref[x] == NEG_INF ? 0.f : m_ref[x];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        sc[nt][2 * x] = sm100::ex2_approx(sc[nt][2 * x] - m);
        sc[nt][2 * x + 1] = sm100::ex2_approx(sc[nt][2 * x + 1] - m);
        l[x] += sc[nt][2 * x] + sc[nt][2 * x + 1];
      }
    }

    // ---------------------------------------------------------------- outputs, 16 keys a step
#pragma unroll
    for (int kk = 0; kk < NT / 2; ++kk) {
      if constexpr (KV4) {
        uint32_t w[2][2][NG / 2];  // [eight keys][key of the pair][pieces of two groups]
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = kk * 16 + y * 8 + 2 * t + e;
            if constexpr (D == 128) {
              const uint2 v = lds<uint2>(sV + cache_granule<D, KV4>(row * 4 + (r >> 1)) + (r & 1) * 8);
              w[y][e][0] = v.x, w[y][e][1] = v.y;
            } else {
              w[y][e][0] = lds<uint32_t>(sV + cache_granule<D, KV4>(row * 2 + (r >> 2)) + (r & 3) * 4);
            }
          }
        const uint32_t sat = scales0 + 2 * (C::TILE * NG * 4);
#pragma unroll
        for (int g2 = 0; g2 < NG / 2; ++g2) {
          uint4 ss[2], mm[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t at = sat + (uint32_t)((kk * 8 + y * 4 + t) * NG * 8 + g2 * 16);
            ss[y] = lds<uint4>(at);
            mm[y] = lds<uint4>(at + C::TILE * NG * 4);
          }
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int g = 2 * g2 + z;
            uint32_t a[2][2] = {{0u, 0u}, {0u, 0u}};  // [row half][eight keys]
#pragma unroll
            for (int x = 0; x < NR; ++x)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const float p0 = sc[2 * kk + y][2 * x], p1 = sc[2 * kk + y][2 * x + 1];
                a[x][y] = pack_f16x2(p0 * __uint_as_float(z ? ss[y].z : ss[y].x), p1 * __uint_as_float(z ? ss[y].w : ss[y].y));
                om[x][g] = fmaf(p0, __uint_as_float(z ? mm[y].z : mm[y].x), om[x][g]);
                om[x][g] = fmaf(p1, __uint_as_float(z ? mm[y].w : mm[y].y), om[x][g]);
              }
            const uint32_t u0 = __byte_perm(w[0][0][g2], w[0][1][g2], z ? 0x7632 : 0x5410);
            const uint32_t u1 = __byte_perm(w[1][0][g2], w[1][1][g2], z ? 0x7632 : 0x5410);
            const uint32_t v0 = u0 >> 8, v1 = u1 >> 8;
            mma16816<true>(o[4 * g], a[0][0], a[1][0], a[0][1], a[1][1], u0 & 0x000F000Fu, u1 & 0x000F000Fu);
            mma16816<true>(o[4 * g + 1], a[0][0], a[1][0], a[0][1], a[1][1], u0 & 0x00F000F0u, u1 & 0x00F000F0u);
            mma16816<true>(o[4 * g + 2], a[0][0], a[1][0], a[0][1], a[1][1], v0 & 0x000F000Fu, v1 & 0x000F000Fu);
            mma16816<true>(o[4 * g + 3], a[0][0], a[1][0], a[0][1], a[1][1], v0 & 0x00F000F0u, v1 & 0x00F000F0u);
          }
        }
      } else {
        uint32_t hi[NR][2], lo[NR][2];  // p as two bf16 parts
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float p0 = sc[2 * kk + y][2 * x], p1 = sc[2 * kk + y][2 * x + 1];
            hi[x][y] = sm100::pack_bf16x2(p0, p1);
            lo[x][y] = sm100::pack_bf16x2(p0 - __uint_as_float(hi[x][y] << 16), p1 - __uint_as_float(hi[x][y] & 0xFFFF0000u));
          }
#pragma unroll
        for (int c = 0; c < CG / 2; ++c) {
          uint32_t v[4];
          const int row = kk * 16 + (lane & 15);
          ldmatrix4<true>(v, sV + cache_granule<D, KV4>(row * (D / 8) + 2 * c + (lane >> 4)));
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            if constexpr (WIDE) {
              mma16816<false>(o[2 * c + y], hi[0][0], hi[NR - 1][0], hi[0][1], hi[NR - 1][1], v[2 * y], v[2 * y + 1]);
              mma16816<false>(o[2 * c + y], lo[0][0], lo[NR - 1][0], lo[0][1], lo[NR - 1][1], v[2 * y], v[2 * y + 1]);
            } else {
              mma16816<false>(o[2 * c + y], hi[0][0], lo[0][0], hi[0][1], lo[0][1], v[2 * y], v[2 * y + 1]);
            }
          }
        }
      }
    }
  }
  cp_async_wait<0>();

  // ------------------------------------------------------------------ the warps of the CTA together
#pragma unroll
  for (int x = 0; x < NR; ++x) {
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    if constexpr (KV4)
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        om[x][g] += __shfl_xor_sync(0xffffffffu, om[x][g], 1);
        om[x][g] += __shfl_xor_sync(0xffffffffu, om[x][g], 2);
      }
  }
  __syncthreads();  // every warp is done with its stages
  float* join = reinterpret_cast<float*>(smem);
  constexpr int JOIN = C::JOIN_BYTES / 4;
  {
    float* mine = join + warp * JOIN;
    // 4-bit: back from 2^f_exp and 2^-24, in two exact steps
    const int back = 24 - f_exp;
    const float b0 = exp2_int(back / 2), b1 = exp2_int(back - back / 2);
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      const int row = r + 8 * x;
      if (t == 0) {
        mine[C::ROWS * D + row] = m_ref[x];
        mine[C::ROWS * D + C::ROWS + row] = l[x];
      }
      float* to = mine + row * D;
#pragma unroll
      for (int c = 0; c < CG; ++c)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float v = o[c][2 * x + y];
          if constexpr (KV4) {
            const int g = c >> 2, i = c & 3;
            if (f_exp == 1000) v = 0.f;
            to[32 * g + 8 * t + 4 * y + i] = fmaf(v * b0 * (i & 1 ? 0.0625f : 1.f), b1, om[x][g]);
          } else {
            if (!WIDE) v += o[c][2 + y];
            to[8 * c + 2 * t + y] = v;
          }
        }
    }
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < heads * D; idx += C::THREADS) {
    const int row = idx / D, e = idx % D;
    float M = NEG_INF, L = 0.f, v = 0.f;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) M = fmaxf(M, join[w * JOIN + C::ROWS * D + row]);
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) {
      const float a = sm100::ex2_approx(join[w * JOIN + C::ROWS * D + row] - M);
      L = fmaf(a, join[w * JOIN + C::ROWS * D + C::ROWS + row], L);
      v = fmaf(a, join[w * JOIN + row * D + e], v);
    }
    const size_t part = (head0 + row) * p.n_split + s;
    p.part_o[part * D + e] = v / L;
    if (e == 0) p.part_lse[part] = M + log2f(L);
  }
}

// Joins the splits.  Grid: x < group: the output of query head x of the group; x >= group: the weights of
// 1024 keys; y: key/value head; z: sequence.
constexpr int CACHE_FINISH_THREADS = 256;
constexpr int CACHE_FINISH_KEYS = 1024;

template <int D>
__global__ void __launch_bounds__(CACHE_FINISH_THREADS) sdpa_cache_finish_kernel(const CacheDecodeParams p) {
  constexpr int LANES = D / 4, SETS = CACHE_FINISH_THREADS / LANES;  // threads per split's row, splits at a time
  __shared__ float s_lse[32];
  __shared__ float4 s_o[SETS][LANES];
  cudaGridDependencySynchronize();
  const float NEG_INF = -__int_as_float(0x7f800000);
  const int kvh = blockIdx.y, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = cache_len(p.kv_lens, b, p.n_cap);
  const int ns = (len + p.chunk - 1) / p.chunk;
  const size_t head0 = (size_t)b * p.H_q + (size_t)kvh * p.group;
  // base-2 log-sum-exp of a head, by one warp
  auto head_lse = [&](size_t head) {
    const float* lse = p.part_lse + head * p.n_split;
    float M = NEG_INF, L = 0.f;
    for (int s = lane; s < ns; s += 32) M = fmaxf(M, lse[s]);
#pragma unroll
    for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    const float m = M == NEG_INF ? 0.f : M;
    for (int s = lane; s < ns; s += 32) L += exp2f(lse[s] - m);
#pragma unroll
    for (int off = 16; off; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    return m + log2f(L);
  };
  if ((int)blockIdx.x < p.group) {
    const size_t head = head0 + blockIdx.x;
    if (warp == 0) {
      const float x = head_lse(head);
      if (lane == 0) s_lse[0] = x;
    }
    __syncthreads();
    const float l2 = s_lse[0];
    const int set = threadIdx.x / LANES, e = threadIdx.x % LANES;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = set; s < ns; s += SETS) {
      const size_t part = head * p.n_split + s;
      const float w = exp2f(p.part_lse[part] - l2);
      const float4 v = reinterpret_cast<const float4*>(p.part_o + part * D)[e];
      a.x = fmaf(w, v.x, a.x), a.y = fmaf(w, v.y, a.y), a.z = fmaf(w, v.z, a.z), a.w = fmaf(w, v.w, a.w);
    }
    s_o[set][e] = a;
    __syncthreads();
    if (threadIdx.x < LANES) {
#pragma unroll
      for (int i = 1; i < SETS; ++i) {
        const float4 v = s_o[i][e];
        a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
      }
      reinterpret_cast<uint2*>(p.O + head * D)[e] =
          make_uint2(sm100::pack_bf16x2(a.x, a.y), sm100::pack_bf16x2(a.z, a.w));
      if (p.LSE && e == 0) p.LSE[head] = ns ? l2 * 0.69314718055994531f : NEG_INF;
    }
    return;
  }
  const int j = ((int)blockIdx.x - p.group) * CACHE_FINISH_KEYS + 4 * threadIdx.x;
  if (((int)blockIdx.x - p.group) * CACHE_FINISH_KEYS >= len) return;
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  for (int h0 = 0; h0 < p.group; h0 += 32) {
    const int nh = min(32, p.group - h0);
    __syncthreads();
    for (int h = warp; h < nh; h += CACHE_FINISH_THREADS / 32) {
      const float x = head_lse(head0 + h0 + h);
      if (lane == 0) s_lse[h] = x;
    }
    __syncthreads();
    if (j < len)
      for (int h = 0; h < nh; ++h) {
        const float4 v = *reinterpret_cast<const float4*>(p.scores + (head0 + h0 + h) * p.score_stride + j);
        w[0] += exp2f(v.x - s_lse[h]), w[1] += exp2f(v.y - s_lse[h]);
        w[2] += exp2f(v.z - s_lse[h]), w[3] += exp2f(v.w - s_lse[h]);
      }
  }
  const size_t at = ((size_t)b * p.H_kv + kvh) * p.n_cap + j;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (j + i < len) p.acc_out[at + i] = (p.acc ? p.acc[at + i] : 0.f) + w[i];
}

}  // namespace sdpa
