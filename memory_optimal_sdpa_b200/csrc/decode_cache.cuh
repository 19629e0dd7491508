// decode_cache.cuh -- one query row per head against a bounded cache: bf16 or 4-bit rows, with the
// attention weights of every key added to an accumulator where asked for.
//
// The keys of all (sequence, key/value head, block of query heads) units, in blocks of 64 or 128, are one long
// line of work that is cut evenly among as many CTAs as fit on the GPU at once: lengths differ, and a
// wave that is not full costs as much as a full one (splits of 2048 keys 183 us, two, three, four lines' worth of CTAs 168,
// 170, 173 us against 165 us for the case below when this was chosen).  A CTA's cut is one or more segments, each of one unit; a segment gives
// a normalised partial output and a log-sum-exp (base 2, as a maximum and a sum) per query head.  Segment number unit + CTA is unique,
// as both only grow along the line.  With weights the scores (base 2, fp32) are written too: a key's weight
// needs the log-sum-exp over all of its unit's segments, and 4 bytes a score, written and read once, cost far less than
// reading the keys again.  sdpa_cache_finish_kernel joins the segments and adds sum_h 2^(score_h - m_h) / l_h per key.
//
// What bounds it: HBM, if the arithmetic fits under it.  A 4-bit row pair of d = 128 is 160 bytes, 6.4 clocks (at the 1.77 GHz
// of the profile below) of an SM's share of HBM, in which 256 codes have to become operands.  So the codes never leave registers:
// mma.sync takes its A operand from the registers they were unpacked in, where tcgen05 would need them
// written to shared memory as 16-bit numbers and read back (512 + 512 bytes, 8 clocks).  Measured on this
// part: m16n8k16 one per 2.1 clocks (one a key here), integer operations two warp instructions a clock, of which a key
// needs nine, six of them for the codes.  64 x 64 heads over 8, cache 16384 (713 MB): 161-169 us, 4.2-4.4 TB/s.  The split
// kernel alone, profiled: 152 us or 269000 clocks, 8.9 a key, in which it issues 19.7 instructions (2.35 a clock of the 4 there
// are, 2.2 with its start and end), so the instructions bound it (without them the same loads take 120 us), whether 8, 12 or 16
// warps share the SM (166 / 165 / 172 us when this was chosen).  bf16, 4 x 32 heads over 8, 32768, with
// weights (439 MB): 84 us, 5.2 TB/s, of which the finishing kernel 9 us.  More than 8 query heads to a key/value head (WIDE: two
// MMAs for each, 255 registers with 20 bytes spilled at d = 128, two CTAs an SM): 64 sequences of 8192 rows, d = 128, 8 key/value heads,
// 8 / 12 / 16 / 20 heads each 146 / 208 / 208 / 386 us (20: two units, which read the cache twice), at d = 64 134 us for 12 and 16;
// bf16 with weights, 16 such sequences, 112 / 120 / 126 / 212 us.
//
// Unpacking: (w & 0x000F000F) is, read as two fp16 numbers, c 2^-24 exactly (subnormal), and
// (w & 0x00F000F0) 16 c 2^-24: one integer operation gives two operands.  The powers of two are put back
// with the group scales.  For that Q enters as fp16, normalised by a power of two per head so that its
// largest element is near 2^14 (the 8 significant bits of bf16 fit in fp16's 11; elements 2^-27 times the
// largest and smaller lose bits, far below the rounding of the 32-bit sums unless a key is as much larger there).
//   scores   S[h, j] = sum_g s_jg (sum_{i in g} q_hi c_ji) + m_jg (sum_{i in g} q_hi)
//   output   O[h, i] = sum_j (p_hj s_jg) c_ji + sum_j p_hj m_jg          (g the group of channel i)
// p s is rounded to fp16, scaled by a power of two f that the scales of the tile set: 2^-3 <= s f < 2^11, so half a step is 2^-12 of
// it (a sixteenth of the rounding of O to bf16) for p from 2^-11 on, and below that 2^-22 of s at most.  The sums with m and everything
// else stay in fp32.  A tile whose scales leave that range moves f; one whose scales are too far apart for any f (an outlier
// among the rows) is added up in fp32, as the other rows would lose their bits to it: 64 x 64 heads over 8, 8192 rows of normal
// values 146 us; with a row 2^14 times as large among 8192 155 us, among 1024 185, among 128 452, in every tile 761 us.
// bf16 caches use the same kernel with bf16 products; there p is split in two bf16 parts (its rounding to one
// would cost as much again as that of O).
// Both products put the cache on the MMA's side of 16 rows (keys, then channels) and the heads on its side of 8, so
// eight heads fill it: S^T = K Q^T, O^T += V^T P^T.  The pairs p s of S^T are turned into the second product's
// operand by an 8 x 8 transpose of the warp (movmatrix).
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
  const __nv_bfloat16* kv[2];   // bf16 cache K, V
  Kv4Cache cache[2];            // or 4-bit cache K, V
  const int* kv_lens;
  float* part_o;    // [units + CTAs, ROWS, D]
  float2* part_stat;  // [units + CTAs, ROWS]: a reference m (-inf: no key counts) and the sum of 2^(score - m), base 2
  long long* seq_at;  // [B + 1]: blocks of work before each sequence, and all of them
  float* scores;    // [B, Hq, score_stride], base 2, or null
  const float* acc;
  float* acc_out;   // [B, Hkv, n_cap]
  __nv_bfloat16* O;
  float* LSE;
  int B, H_q, H_kv, group, n_cap;
  int head_blocks;   // units per (sequence, key/value head)
  int rows;          // query heads per unit
  int block;         // keys per block of work
  int n_cta;
  int score_stride;  // n_cap rounded up to 4
  float scale_log2;  // scale log2 e 2^-scale_exp
  int scale_exp;     // 2 for the largest scales, which log2 e takes out of range, -64 for the least, whose bits it would round away
};

// WIDE: 9 to 16 query heads per CTA, else up to 8.  Heads are on the MMA's side of 8, so WIDE takes two products for one.
template <int D, bool KV4, bool WIDE>
struct CacheCfg {
  static constexpr int WARPS = 4;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int ROWS = WIDE ? 16 : 8;         // query heads
  static constexpr int TILE = KV4 ? 32 : 16;         // keys per warp tile
  static constexpr int STAGES = 3;
  static constexpr int ROW_BYTES = KV4 ? D / 2 : 2 * D;
  static constexpr int HALF_BYTES = TILE * ROW_BYTES;  // K or V of a tile
  static constexpr int NG = D / 32;
  static constexpr int RAW_BYTES = KV4 ? TILE * NG * 4 : 0;  // the scales of a tile as they are stored, K's or V's
  static constexpr int STAGE_BYTES = 2 * (HALF_BYTES + RAW_BYTES);
  static constexpr int SCALE_BYTES = KV4 ? 3 * TILE * NG * 4 : 0;  // K's s, V's s and m as fp32
  static constexpr int WARP_BYTES = STAGES * STAGE_BYTES + SCALE_BYTES;
  static constexpr int JOIN_ROW = D + 4;                   // floats: the four columns of a quad meet other banks
  static constexpr int JOIN_BYTES = ROWS * JOIN_ROW * 4;   // a warp's outputs (over the stages)
  static constexpr int SMEM_BYTES = WARPS * (WARP_BYTES > JOIN_BYTES ? WARP_BYTES : JOIN_BYTES);
  static constexpr int MIN_BLOCKS = WIDE ? 2 : (KV4 ? 3 : 2);  // CTAs per SM
  static constexpr int BLOCK = WARPS * TILE;                    // keys per block of work
};

// The line of work: unit u = b upb + (key/value head, head block), of blocks(b) blocks each.  CTA c takes blocks
// [c T / n, (c + 1) T / n) of the T there are, with n = min(CTAs, T), so that none of the n is empty.
struct CacheLine {
  long long total;  // T
  int n;
  __device__ __forceinline__ static int blocks(const CacheDecodeParams& p, int b) {
    return (cache_len(p.kv_lens, b, p.n_cap) + p.block - 1) / p.block;
  }
  __device__ __forceinline__ CacheLine(const CacheDecodeParams& p, long long total_) : total(total_) {
    n = (int)min((long long)p.n_cta, total);
  }
  // By a whole warp.
  __device__ __forceinline__ CacheLine(const CacheDecodeParams& p, int lane) {
    int sum = 0;  // below 2^31: batch * heads * n_cap is
    for (int b = lane; b < p.B; b += 32) sum += blocks(p, b);
    total = (long long)__reduce_add_sync(0xffffffffu, sum) * p.H_kv * p.head_blocks;
    n = (int)min((long long)p.n_cta, total);
  }
  __device__ __forceinline__ long long begin(int c) const { return c * total / n; }
  // The CTA that has block x.
  __device__ __forceinline__ int cta_of(long long x) const { return (int)(((x + 1) * n + total - 1) / total) - 1; }
  // Runs over the sequences, 32 at a time, with a warp: f(b, blocks before b, blocks of b and before) -> stop.
  template <class F>
  __device__ __forceinline__ static void scan(const CacheDecodeParams& p, int lane, F f) {
    const long long upb = (long long)p.H_kv * p.head_blocks;
    long long run = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane, mine = b < p.B ? blocks(p, b) : 0;
      int sum = mine;  // inclusive over the lanes
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += y;
      }
      if (f(b, run + (sum - mine) * upb, run + sum * upb)) return;
      run += __shfl_sync(0xffffffffu, sum, 31) * upb;
    }
  }
  // The first sequence whose blocks end past x, and where they begin.
  __device__ __forceinline__ static long long find(const CacheDecodeParams& p, int lane, long long x, int& found) {
    long long at = 0;
    scan(p, lane, [&](int b, long long begin, long long end) {
      const uint32_t past = __ballot_sync(0xffffffffu, end > x);
      if (past == 0) return false;
      const int k = __ffs(past) - 1;
      found = __shfl_sync(0xffffffffu, b, k);
      at = __shfl_sync(0xffffffffu, begin, k);
      return true;
    });
    return at;
  }
  __device__ __forceinline__ static void write(const CacheDecodeParams& p, int lane) {
    scan(p, lane, [&](int b, long long begin, long long end) {
      if (b < p.B) p.seq_at[b] = begin;
      if (b == p.B - 1) p.seq_at[p.B] = end;
      return false;
    });
  }
};

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void sts_zero(uint32_t dst) {
  if constexpr (BYTES == 16)
    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(dst), "r"(0) : "memory");
  else
    asm volatile("st.shared.v2.u32 [%0], {%1,%1};" ::"r"(dst), "r"(0) : "memory");
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

// A B alone (C = 0), fp16.
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// A B alone, m16n8k8, tf32 operands.
__device__ __forceinline__ void mma1688_tf32_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                   uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t to_tf32(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
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

// The 8 x 8 matrix of 16-bit elements of which a thread holds row lane / 4, columns 2 (lane % 4) and + 1, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
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
template <int N>
__device__ __forceinline__ void sts_row(uint32_t addr, const float* x) {
  if constexpr (N == 4)
    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]) : "memory");
  else
    asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(addr), "f"(x[0]), "f"(x[1]) : "memory");
}
template <int N>
__device__ __forceinline__ void lds_row(uint32_t addr, float (&x)[N]) {
  if constexpr (N == 4) {
    const uint4 v = lds<uint4>(addr);
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  } else {
    const uint2 v = lds<uint2>(addr);
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
  }
}
// 2^e as a float, e clamped to the normal range.
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23); }

__device__ __forceinline__ int exponent_of(float x) { return (int)(__float_as_uint(x) >> 23 & 255) - 127; }

// ------------------------------------------------------------------------------------------ operands
// Q as the B operand (column: head 8 x + r).  4-bit: per group g and step st (channels i = 2 st, 2 st + 1 of the
// pieces), the pairs (32 g + 8 t + i, 32 g + 8 t + 4 + i), those of odd i divided by 16; see the file's head.
template <int D, bool KV4, bool WIDE>
struct CacheQuery {
  static constexpr int NG = D / 32, NR = WIDE ? 2 : 1;
  uint32_t b[NR][D / 16][2];
  // 4-bit: the group sums of the normalised q, times 2^-24, as two tf32 parts: the B operand (k = t, k = t + 4) of the
  // product with the minima.  d = 128: parts 0 and 1 of group t; d = 64: part t / 2 of group t mod 2, and 0.
  uint32_t sum[NR][2];
  int exp[NR];  // this head's scores are to be multiplied by 2^exp at the end

  // flip: the sign bits of a negative scale (two bf16 at a time).
  __device__ __forceinline__ void load(const __nv_bfloat16* q, int heads, uint32_t flip, int lane) {
    const int r = lane >> 2, t = lane & 3;
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      const bool on = r + 8 * x < heads;
      const __nv_bfloat16* row = q + (size_t)(r + 8 * x) * D;
      if constexpr (KV4) {
        float f[NG][8], big = 0.f;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          uint4 raw = on ? *reinterpret_cast<const uint4*>(row + 32 * g + 8 * t) : make_uint4(0, 0, 0, 0);
          raw.x ^= flip, raw.y ^= flip, raw.z ^= flip, raw.w ^= flip;
          bf16x8_to_f32(raw, f[g]);
#pragma unroll
          for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(f[g][i]));
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // largest element in [2^14, 2^15); a zero row keeps its (irrelevant) factor
        const int e = (int)(__float_as_uint(big) >> 23) - 127;
        const float up = exp2_int((14 - e) / 2), up2 = exp2_int(14 - e - (14 - e) / 2);  // two exact steps: 2^(14 - e) itself may overflow
        exp[x] = 24 + e - 14;  // the codes' 2^-24 undone too
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float total = 0.f;  // over the 32 channels
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            f[g][i] = f[g][i] * up * up2;
            total += f[g][i];
          }
          total += __shfl_xor_sync(0xffffffffu, total, 1);
          total += __shfl_xor_sync(0xffffffffu, total, 2);
          total *= 0x1p-24f;
          const uint32_t part0 = to_tf32(total), part1 = to_tf32(total - __uint_as_float(part0));
          if (NG == 4) {
            if (t == g) sum[x][0] = part0, sum[x][1] = part1;
          } else if ((t & 1) == g) {
            sum[x][0] = t < 2 ? part0 : part1, sum[x][1] = 0u;
          }
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            b[x][2 * g + st][0] = pack_f16x2(f[g][2 * st], f[g][4 + 2 * st]);
            b[x][2 * g + st][1] = pack_f16x2(f[g][2 * st + 1] * 0.0625f, f[g][5 + 2 * st] * 0.0625f);
          }
        }
      } else {
        exp[x] = 0;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          b[x][k][0] = on ? *reinterpret_cast<const uint32_t*>(row + 16 * k + 2 * t) ^ flip : 0u;
          b[x][k][1] = on ? *reinterpret_cast<const uint32_t*>(row + 16 * k + 8 + 2 * t) ^ flip : 0u;
        }
      }
    }
  }
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

// V's scales of a tile (a lane per key), where some are 0, NaN or outside what p s f may be in fp16: 2^-3 <= s f < 2^11.  Where
// they lie within 2^10 of each other f moves, and the sums o with it; otherwise (or where o would leave the 32-bit range)
// the result is true and the tile is added up in fp32.
template <int D, int NR>
__device__ __forceinline__ bool cache_move_scale(const float (&sv)[D / 32], float& f, float (&o)[D / 16][NR][4]) {
  uint32_t top = 0, least = 0x7F800000u;
#pragma unroll
  for (int g = 0; g < D / 32; ++g) {
    const uint32_t bits = __float_as_uint(fabsf(sv[g]));
    if (bits <= 0x7F800000u) top = max(top, bits);  // a NaN stays one in every product
    if (bits) least = min(least, bits);
  }
  const float hi = __uint_as_float(__reduce_max_sync(0xffffffffu, top)), lo = __uint_as_float(__reduce_min_sync(0xffffffffu, least));
  const bool near = lo * 0x1p10f > hi, none = f != f;
  const int want = min(7 - exponent_of(near ? hi : lo), 126), room = 100 - exponent_of(hi);  // room: p s f c in 32 bits
  auto fits = [&] { return hi * f < 0x1p11f && lo * f >= 0x1p-3f; };
  if (none) {  // no sums yet
    f = hi > 0.f ? exp2_int(min(want, room)) : 1.f;
    return hi > 0.f && !fits();
  }
  if (hi == 0.f || fits()) return false;
  const int old = exponent_of(f);
  float most = 0.f;
#pragma unroll
  for (int c = 0; c < D / 16; ++c)
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) most = fmaxf(most, fabsf(o[c][x][i]));
  const int e = min(__all_sync(0xffffffffu, near && exponent_of(most) + want - old < 100) ? want : old, room);
  const float m0 = exp2_int((e - old) / 2), m1 = exp2_int(e - old - (e - old) / 2);
#pragma unroll
  for (int c = 0; c < D / 16; ++c)
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[c][x][i] = o[c][x][i] * m0 * m1;
  f = exp2_int(e);
  return !fits();
}

// Adds a tile's p s c, p = 2^(sc c2 - m), to o in fp32, in the units of the products that it stands in for; about five times as
// slow as they.
template <int D, int NR>
__device__ __forceinline__ void cache_add_values(const float (&sc)[2][NR][4], const float (&c2)[NR][2], const float (&m)[NR][2],
                                                 float (&o)[D / 16][NR][4], uint32_t sV, uint32_t scales, int lane) {
  constexpr int NG = D / 32;
  const int r = lane >> 2, t = lane & 3;
#pragma unroll 1
  for (int row = 0; row < 32; ++row) {
    uint32_t w[NG / 2];
    if constexpr (D == 128) {
      const uint2 v = lds<uint2>(sV + cache_granule<D, true>(row * 4 + (r >> 1)) + (r & 1) * 8);
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = lds<uint32_t>(sV + cache_granule<D, true>(row * 2 + (r >> 2)) + (r & 3) * 4);
    }
    float s[NG];
    lds_row<NG>(scales + (uint32_t)(row * NG * 4), s);
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      float a[2];  // this key's p; its score is in the lane that has row's place in eight
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float lower = row & 8 ? sc[0][x][2 + y] : sc[0][x][y], upper = row & 8 ? sc[1][x][2 + y] : sc[1][x][y];
        const float s = __shfl_sync(0xffffffffu, row & 16 ? upper : lower, 4 * (row & 7) + t);
        a[y] = sm100::ex2_approx(fmaf(s, c2[x][y], m[x][y] == -__int_as_float(0x7f800000) ? 0.f : -m[x][y]));
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t c = w[g >> 1] >> (16 * (g & 1));  // four channels
        const float a0 = a[0] * s[g] * 0x1p-24f, a1 = a[1] * s[g] * 0x1p-24f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float c0 = (float)(c >> (8 * h) & 0x0Fu), c1 = (float)(c >> (8 * h) & 0xF0u);
          o[2 * g + h][x][0] = fmaf(a0, c0, o[2 * g + h][x][0]);
          o[2 * g + h][x][1] = fmaf(a1, c0, o[2 * g + h][x][1]);
          o[2 * g + h][x][2] = fmaf(a0, c1, o[2 * g + h][x][2]);
          o[2 * g + h][x][3] = fmaf(a1, c1, o[2 * g + h][x][3]);
        }
      }
    }
  }
}

template <int D, bool KV4, bool WIDE>
__global__ void __launch_bounds__(CacheCfg<D, KV4, WIDE>::THREADS, CacheCfg<D, KV4, WIDE>::MIN_BLOCKS)
    sdpa_cache_split_kernel(const CacheDecodeParams p) {
  using C = CacheCfg<D, KV4, WIDE>;
  constexpr int NG = C::NG, NR = WIDE ? 2 : 1, KT = C::TILE / 16;  // KT: 16-key tiles of scores
  constexpr int CT = D / 16;                                       // 16-channel tiles of outputs
  const float NEG_INF = -__int_as_float(0x7f800000);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t stage0 = sm100::smem_u32(smem) + warp * C::WARP_BYTES;
  const uint32_t scales0 = stage0 + C::STAGES * C::STAGE_BYTES;

  const CacheLine line(p, lane);
  const int cta = blockIdx.x, upb = p.H_kv * p.head_blocks;
  if (cta >= line.n) return;
  long long at = line.begin(cta);
  const long long end = line.begin(cta + 1);
  __shared__ float2 s_stat[C::WARPS][C::ROWS];  // m, l
  __shared__ float s_pre[C::THREADS][2 * NR];   // each thread's own: see `far`
  if (cta == 0 && warp == 0) CacheLine::write(p, lane);
  int b = 0;
  long long seq_at = CacheLine::find(p, lane, at, b);  // where sequence b begins
  int seq_blocks = CacheLine::blocks(p, b);

  for (bool first = true; at < end; first = false) {
  if (!first) __syncthreads();  // the last segment's results have been read
  while (at >= seq_at + (long long)upb * seq_blocks) {
    seq_at += (long long)upb * seq_blocks;
    seq_blocks = CacheLine::blocks(p, ++b);
  }
  const int unit = (int)((at - seq_at) / seq_blocks), block0 = (int)((at - seq_at) % seq_blocks);
  const int n_blocks = (int)min((long long)(seq_blocks - block0), end - at);
  at += n_blocks;
  const size_t part0 = ((size_t)b * upb + unit + cta) * C::ROWS;
  const int kvh = unit / p.head_blocks, h0 = (unit % p.head_blocks) * C::ROWS;
  const int heads = min(C::ROWS, p.group - h0);
  const int k0 = block0 * C::BLOCK;
  const int n = min(n_blocks * C::BLOCK, cache_len(p.kv_lens, b, p.n_cap) - k0);
  const size_t row0 = ((size_t)b * p.H_kv + kvh) * p.n_cap + k0;
  const size_t head0 = (size_t)b * p.H_q + (size_t)kvh * p.group + h0;

  const int n_tiles = (n + C::TILE - 1) / C::TILE;
  // This lane's places in the next tile to fetch.  32 granules further is whole lines further, so a lane's place in
  // every 512 bytes of 4-bit rows is the same.
  const uint8_t* src[2];
  const uint32_t* src_scales[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    src[x] = (KV4 ? p.cache[x].codes : reinterpret_cast<const uint8_t*>(p.kv[x])) +
             (row0 + warp * C::TILE) * C::ROW_BYTES + lane * 16;
    if (KV4) src_scales[x] = p.cache[x].scales + (row0 + warp * C::TILE + lane) * NG;
  }
  int left = n - warp * C::TILE;  // keys from there on
  const uint32_t lane_to = stage0 + cache_granule<D, KV4>(lane), lane_raw = stage0 + 2 * C::HALF_BYTES + lane * (NG * 4);
  auto fetch = [&](uint32_t put) {  // put: the stage, in bytes
    if (left > 0) {
      const bool full = left >= C::TILE;
      if constexpr (KV4) {  // scales: a lane per key; zeros past the length
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t to = lane_raw + put + x * C::RAW_BYTES;
          if (full || lane < left)
            cp_async<NG * 4>(to, src_scales[x]);
          else
            sts_zero<NG * 4>(to);
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < C::HALF_BYTES / 512; ++i) {
          const uint32_t to = (KV4 ? lane_to + i * 512 : stage0 + cache_granule<D, KV4>(i * 32 + lane)) + put + x * C::HALF_BYTES;
          // rows past the length: bf16 ones become zeros; of 4 bits any codes will do, as their scales are 0
          if (full || (i * 32 + lane) / (C::ROW_BYTES / 16) < left)
            cp_async<16>(to, src[x] + i * 512);
          else if (!KV4)
            sts_zero<16>(to);
        }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        src[x] += C::WARPS * C::HALF_BYTES;
        if (KV4) src_scales[x] += C::WARPS * C::TILE * NG;
      }
      left -= C::WARPS * C::TILE;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < C::STAGES - 1; ++i) fetch(i * C::STAGE_BYTES);

  CacheQuery<D, KV4, WIDE> q;
  q.load(p.Q + head0 * D, heads, p.scale_log2 < 0.f ? 0x80008000u : 0u, lane);
  // A thread's columns are the heads 8 x + 2 t + y (y = 0, 1).
  float c2[NR][2];
  uint32_t far = 0;  // a bit per column; four bits up: scores multiplied by s_pre
#pragma unroll
  for (int x = 0; x < NR; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      // |scale log2 e| 2^exp in two steps, which leave the range only where the result does.  Beyond 2^126 the scores are first
      // multiplied by 2^126 (`far`; at most 1 % slower for testing it).  Not 0 (scale 0), which would make NaN of the -inf
      // of a key past the length: with the smallest float, 2^-149, no score that is finite before comes to 2^-20.
      const float c = fabsf(p.scale_log2);
      const int e = __shfl_sync(0xffffffffu, q.exp[x], 8 * t + 4 * y) + p.scale_exp;
      c2[x][y] = c * exp2_int(e / 2) * exp2_int(e - e / 2);
      if (c2[x][y] > 0x1p126f) {
        far |= 1u << (2 * x + y);
        c2[x][y] = fminf(c * exp2_int((e - 126) / 2) * exp2_int(e - 126 - (e - 126) / 2), FLT_MAX);
      }
      c2[x][y] = fmaxf(c2[x][y], 0x1p-149f);
    }

  // Tiles whose scores need no second look: not the one that the length ends in, none where a column is far.
  int plain_tiles = __any_sync(0xffffffffu, far != 0) ? 0 : n / C::TILE;

  // Outputs, transposed: rows are channels (4-bit: tile 2 g + h holds channels 32 g + 4 r + 2 h and, in rows 8 .. 15, + 1;
  // bf16: 16 c + r and + 8), columns heads.  om: sums of p m.
  float m_ref[NR][2], l[NR][2], om[NR][2][KV4 ? NG : 1], o[CT][NR][4];
#pragma unroll
  for (int x = 0; x < NR; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      m_ref[x][y] = NEG_INF;
      l[x][y] = 0.f;
#pragma unroll
      for (int g = 0; g < (KV4 ? NG : 1); ++g) om[x][y][g] = 0.f;
    }
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[c][x][i] = 0.f;
  float f = __int_as_float(0x7FC00000);  // 4-bit: p s is multiplied by this power of two (NaN: not chosen yet)

  uint32_t get = 0;  // this tile's stage, in bytes
  for (int tile = warp; tile < n_tiles; tile += C::WARPS) {
    cp_async_wait<C::STAGES - 2>();
    bool uneven = false;  // 4-bit: V's scales of this tile are too far apart for fp16
    if constexpr (KV4) {
      __syncwarp();  // the last tile's scales have been read
      // The scales for the whole warp, [key][group] of K's s, V's s, V's m; K's m are taken from where they are.
      float w0f[NG], w1f[NG];  // this lane's key, as it copied it itself
      lds_row<NG>(lane_raw + get, w0f);
      lds_row<NG>(lane_raw + get + C::RAW_BYTES, w1f);
      uint32_t w0[NG], w1[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) w0[g] = __float_as_uint(w0f[g]), w1[g] = __float_as_uint(w1f[g]);
      float sv[NG];
      const uint32_t least = 0x3E000000u + 0x3F800000u - __float_as_uint(f);  // 2^-3 / f
      uint32_t beside = 0;  // how far up from there s is, in bits
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        sv[g] = __uint_as_float(w1[g] << 16);
        beside = max(beside, (w1[g] << 16) - least);
      }
      if (__any_sync(0xffffffffu, beside >= 0x07000000u || f != f)) uneven = cache_move_scale<D, NR>(sv, f, o);
      const uint32_t to = scales0 + (uint32_t)(lane * NG * 4);
      float k[NG], mv[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        k[g] = __uint_as_float(w0[g] << 16);
        sv[g] *= f;
        mv[g] = __uint_as_float(w1[g] & 0xFFFF0000u);
      }
      sts_row<NG>(to, k);
      sts_row<NG>(to + C::TILE * NG * 4, sv);
      sts_row<NG>(to + 2 * C::TILE * NG * 4, mv);
    }
    __syncwarp();
    fetch(get == 0 ? (C::STAGES - 1) * C::STAGE_BYTES : get - C::STAGE_BYTES);
    const uint32_t sK = stage0 + get, sV = sK + C::HALF_BYTES;
    get = get == (C::STAGES - 1) * C::STAGE_BYTES ? 0 : get + C::STAGE_BYTES;

    // ---------------------------------------------------------------- scores, to be multiplied by c2
    float sc[KT][NR][4];  // (key r, heads 2 t, 2 t + 1), (key r + 8, the same heads)
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      if constexpr (KV4) {
        uint32_t w[2][NG];  // keys r, r + 8: pieces of groups (0, 1), (2, 3) of chunk 2 t, then of chunk 2 t + 1
        float ks[2][NG];
        uint32_t km[2];     // the minima of group t: the A operand of the product with the group sums
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int row = kt * 16 + y * 8 + r;
          if constexpr (D == 128) {
            const uint4 v = lds<uint4>(sK + cache_granule<D, KV4>(row * 4 + t));
            w[y][0] = v.x, w[y][1] = v.y, w[y][2] = v.z, w[y][3] = v.w;
          } else {
            const uint2 v = lds<uint2>(sK + cache_granule<D, KV4>(row * 2 + (t >> 1)) + (t & 1) * 8);
            w[y][0] = v.x, w[y][1] = v.y;
          }
          lds_row<NG>(scales0 + (uint32_t)(row * NG * 4), ks[y]);
          km[y] = lds<uint32_t>(sK + 2 * C::HALF_BYTES + (uint32_t)((row * NG + (t & (NG - 1))) * 4)) & 0xFFFF0000u;
        }
#pragma unroll
        for (int x = 0; x < NR; ++x) mma1688_tf32_first(sc[kt][x], km[0], km[1], km[0], km[1], q.sum[x][0], q.sum[x][1]);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint32_t sel = g & 1 ? 0x7632 : 0x5410;
          const uint32_t u0 = __byte_perm(w[0][g >> 1], w[0][NG / 2 + (g >> 1)], sel), v0 = u0 >> 8;
          const uint32_t u1 = __byte_perm(w[1][g >> 1], w[1][NG / 2 + (g >> 1)], sel), v1 = u1 >> 8;
          const uint32_t a0[4] = {u0 & 0x000F000Fu, u1 & 0x000F000Fu, u0 & 0x00F000F0u, u1 & 0x00F000F0u};
          const uint32_t a1[4] = {v0 & 0x000F000Fu, v1 & 0x000F000Fu, v0 & 0x00F000F0u, v1 & 0x00F000F0u};
#pragma unroll
          for (int x = 0; x < NR; ++x) {
            float c[4];
            mma16816_first(c, a0[0], a0[1], a0[2], a0[3], q.b[x][2 * g][0], q.b[x][2 * g][1]);
            mma16816<true>(c, a1[0], a1[1], a1[2], a1[3], q.b[x][2 * g + 1][0], q.b[x][2 * g + 1][1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[kt][x][i] = fmaf(ks[i >> 1][g], c[i], sc[kt][x][i]);
          }
        }
      } else {
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[kt][x][i] = 0.f;
        const int row = kt * 16 + (lane & 15);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          uint32_t a[4];
          ldmatrix4<false>(a, sK + cache_granule<D, KV4>(row * (D / 8) + 2 * k + (lane >> 4)));
#pragma unroll
          for (int x = 0; x < NR; ++x) mma16816<false>(sc[kt][x], a[0], a[1], a[2], a[3], q.b[x][k][0], q.b[x][k][1]);
        }
      }
    }
    if (tile >= plain_tiles) {
      if (far) {
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              if (far >> (2 * x + (i & 1)) & 1) sc[kt][x][i] *= 0x1p126f;
              if (far >> (4 + 2 * x + (i & 1)) & 1) sc[kt][x][i] *= s_pre[threadIdx.x][2 * x + (i & 1)];
            }
      }
      const int left = n - tile * C::TILE;  // keys past the length
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (kt * 16 + (i >> 1) * 8 + r >= left) sc[kt][x][i] = NEG_INF;
    }
    if (p.scores) {
#pragma unroll
      for (int x = 0; x < NR; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int h = 8 * x + 2 * t + (i & 1);
          if (h < heads) {
            float* to = p.scores + (head0 + h) * p.score_stride + k0;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              const int j = tile * C::TILE + kt * 16 + (i >> 1) * 8 + r;
              if (j < n) to[j] = sc[kt][x][i] * c2[x][i & 1];
            }
          }
        }
    }
    // ---------------------------------------------------------------- online softmax
    float mt[NR][2];
    bool move = false;
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float m = fmaxf(sc[0][x][y], sc[0][x][2 + y]);
#pragma unroll
        for (int kt = 1; kt < KT; ++kt) m = sm100::max3f(m, sc[kt][x][y], sc[kt][x][2 + y]);
        mt[x][y] = m * c2[x][y];
        move |= mt[x][y] > m_ref[x][y] + 4.f;
      }
    if (KV4) move |= uneven;
    if (__any_sync(0xffffffffu, move)) {
#pragma unroll
      for (int x = 0; x < NR; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float m = fmaxf(m_ref[x][y], mt[x][y]);
#pragma unroll
          for (int off = 4; off <= 16; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
          const float alpha = m_ref[x][y] == NEG_INF ? 0.f : sm100::ex2_approx(m_ref[x][y] - m);
          m_ref[x][y] = m;
          l[x][y] *= alpha;
#pragma unroll
          for (int g = 0; g < (KV4 ? NG : 1); ++g) om[x][y][g] *= alpha;
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            o[c][x][y] *= alpha;
            o[c][x][2 + y] *= alpha;
          }
        }
      // sc c2 - m by a fused step would leave the rounding of m: half a unit of it, which beyond 2^20 is no longer small.  There
      // the products are rounded as m was, from here on.
      bool big = false;
#pragma unroll
      for (int x = 0; x < NR; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          if (fabsf(m_ref[x][y]) > 0x1p20f && m_ref[x][y] != NEG_INF && !(far >> (4 + 2 * x + y) & 1)) {
            big = true;
            far |= 16u << (2 * x + y);
            s_pre[threadIdx.x][2 * x + y] = c2[x][y];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              sc[kt][x][y] *= c2[x][y];
              sc[kt][x][2 + y] *= c2[x][y];
            }
            c2[x][y] = 1.f;
          }
      if (__any_sync(0xffffffffu, big)) plain_tiles = 0;
      if constexpr (KV4)
        if (uneven) {  // the tile's values now, and nothing of them below
          const uint32_t at = scales0 + C::TILE * NG * 4;
          cache_add_values<D, NR>(sc, c2, m_ref, o, sV, at, lane);
          __syncwarp();
          const float none[NG] = {};
          sts_row<NG>(at + (uint32_t)(lane * NG * 4), none);
          __syncwarp();
        }
    }
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float m = m_ref[x][i & 1] == NEG_INF ? 0.f : m_ref[x][i & 1];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          sc[kt][x][i] = sm100::ex2_approx(fmaf(sc[kt][x][i], c2[x][i & 1], -m));
          l[x][i & 1] += sc[kt][x][i];
        }
      }

    // ---------------------------------------------------------------- outputs, 16 keys a step
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      if constexpr (KV4) {
        uint32_t ps[NG][NR][2];  // p s, the B operand: [group][eight heads][eight keys]
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t at = scales0 + C::TILE * NG * 4 + (uint32_t)((kt * 16 + y * 8 + r) * NG * 4);
          float vs[NG], vm[NG];  // of key r + 8 y
          lds_row<NG>(at, vs);
          lds_row<NG>(at + C::TILE * NG * 4, vm);
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int x = 0; x < NR; ++x) {
              const float p0 = sc[kt][x][2 * y], p1 = sc[kt][x][2 * y + 1];
              ps[g][x][y] = transpose8x8(pack_f16x2(p0 * vs[g], p1 * vs[g]));
              om[x][0][g] = fmaf(p0, vm[g], om[x][0][g]);
              om[x][1][g] = fmaf(p1, vm[g], om[x][1][g]);
            }
        }
        uint32_t w[2][2][NG / 2];  // [eight keys][key of the pair][pieces of two groups]
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = kt * 16 + y * 8 + 2 * t + e;
            if constexpr (D == 128) {
              const uint2 v = lds<uint2>(sV + cache_granule<D, KV4>(row * 4 + (r >> 1)) + (r & 1) * 8);
              w[y][e][0] = v.x, w[y][e][1] = v.y;
            } else {
              w[y][e][0] = lds<uint32_t>(sV + cache_granule<D, KV4>(row * 2 + (r >> 2)) + (r & 3) * 4);
            }
          }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint32_t sel = g & 1 ? 0x7632 : 0x5410;
          const uint32_t u0 = __byte_perm(w[0][0][g >> 1], w[0][1][g >> 1], sel), v0 = u0 >> 8;
          const uint32_t u1 = __byte_perm(w[1][0][g >> 1], w[1][1][g >> 1], sel), v1 = u1 >> 8;
#pragma unroll
          for (int x = 0; x < NR; ++x) {
            mma16816<true>(o[2 * g][x], u0 & 0x000F000Fu, u0 & 0x00F000F0u, u1 & 0x000F000Fu, u1 & 0x00F000F0u, ps[g][x][0],
                           ps[g][x][1]);
            mma16816<true>(o[2 * g + 1][x], v0 & 0x000F000Fu, v0 & 0x00F000F0u, v1 & 0x000F000Fu, v1 & 0x00F000F0u,
                           ps[g][x][0], ps[g][x][1]);
          }
        }
      } else {
        uint32_t hi[NR][2], lo[NR][2];  // p as two bf16 parts
#pragma unroll
        for (int x = 0; x < NR; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float p0 = sc[kt][x][2 * y], p1 = sc[kt][x][2 * y + 1];
            const uint32_t h = sm100::pack_bf16x2(p0, p1);
            hi[x][y] = transpose8x8(h);
            lo[x][y] =
                transpose8x8(sm100::pack_bf16x2(p0 - __uint_as_float(h << 16), p1 - __uint_as_float(h & 0xFFFF0000u)));
          }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          uint32_t v[4];
          const int row = kt * 16 + (lane & 7) + ((lane >> 4) << 3);
          ldmatrix4<true>(v, sV + cache_granule<D, KV4>(row * (D / 8) + 2 * c + ((lane >> 3) & 1)));
#pragma unroll
          for (int x = 0; x < NR; ++x) {
            mma16816<false>(o[c][x], v[0], v[1], v[2], v[3], hi[x][0], hi[x][1]);
            mma16816<false>(o[c][x], v[0], v[1], v[2], v[3], lo[x][0], lo[x][1]);
          }
        }
      }
    }
  }
  cp_async_wait<0>();

  // ------------------------------------------------------------------ the warps of the CTA together
#pragma unroll
  for (int x = 0; x < NR; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
#pragma unroll
      for (int off = 4; off <= 16; off <<= 1) {
        l[x][y] += __shfl_xor_sync(0xffffffffu, l[x][y], off);
        if constexpr (KV4)
#pragma unroll
          for (int g = 0; g < NG; ++g) om[x][y][g] += __shfl_xor_sync(0xffffffffu, om[x][y][g], off);
      }
      if (r == 0) s_stat[warp][8 * x + 2 * t + y] = make_float2(m_ref[x][y], l[x][y]);
    }
  __syncthreads();  // and every warp is done with its stages
  float* join = reinterpret_cast<float*>(smem);
  constexpr int JOIN = C::JOIN_BYTES / 4;
  const bool whole = n_blocks == seq_blocks;  // the unit has no other segment
  {
    const int back = 24 - exponent_of(f);  // 4-bit: from f and 2^-24, in two exact steps
    const float b0 = exp2_int(back / 2), b1 = exp2_int(back - back / 2);
#pragma unroll
    for (int x = 0; x < NR; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int row = 8 * x + 2 * t + y;
        float M = NEG_INF, L = 0.f;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) M = fmaxf(M, s_stat[w][row].x);
        // no key scores more than -inf: 0 and -inf, as without a key (L is 0, or NaN where a score is)
        if (M == NEG_INF) M = 0.f;
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) L = fmaf(sm100::ex2_approx(s_stat[w][row].x - M), s_stat[w][row].y, L);
        const float mul = L == 0.f ? 0.f : sm100::ex2_approx(m_ref[x][y] - M) / L;  // of this warp's sums
        if (warp == 0 && r == 0 && row < heads) {
          p.part_stat[part0 + row] = make_float2(L == 0.f ? NEG_INF : M, L);
          if (whole && p.LSE) p.LSE[head0 + row] = (M + log2f(L)) * 0.69314718055994531f;
        }
        float* to = join + warp * JOIN + row * C::JOIN_ROW;
        if constexpr (KV4) {
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            float v[4] = {o[2 * g][x][y], o[2 * g][x][2 + y] * 0.0625f, o[2 * g + 1][x][y], o[2 * g + 1][x][2 + y] * 0.0625f};
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fmaf(v[i] * b0, b1, om[x][y][g]) * mul;
            *reinterpret_cast<float4*>(to + 32 * g + 4 * r) = make_float4(v[0], v[1], v[2], v[3]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            to[16 * c + r] = o[c][x][y] * mul;
            to[16 * c + 8 + r] = o[c][x][2 + y] * mul;
          }
        }
      }
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < heads * (D / 4); idx += C::THREADS) {
    const int row = idx / (D / 4), e = idx % (D / 4);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) {
      const float4 u = *reinterpret_cast<const float4*>(join + w * JOIN + row * C::JOIN_ROW + 4 * e);
      v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
    }
    if (whole)
      reinterpret_cast<uint2*>(p.O + (head0 + row) * D)[e] =
          make_uint2(sm100::pack_bf16x2(v.x, v.y), sm100::pack_bf16x2(v.z, v.w));
    else
      reinterpret_cast<float4*>(p.part_o + (part0 + row) * D)[e] = v;
  }
  }  // segments
}

// Joins the segments of units that have several.  Grid: x < head blocks: the outputs of a unit; x beyond: the weights of
// 4096 keys; y: key/value head; z: sequence.
constexpr int CACHE_FINISH_THREADS = 512;
constexpr int CACHE_FINISH_KEYS = 4096;

template <int D>
__global__ void __launch_bounds__(CACHE_FINISH_THREADS) sdpa_cache_finish_kernel(const CacheDecodeParams p) {
  constexpr int WARPS = CACHE_FINISH_THREADS / 32;
  __shared__ float s_o[WARPS][D];
  __shared__ float2 s_stat[WARPS];  // m, 1 / l
  cudaGridDependencySynchronize();
  const float NEG_INF = -__int_as_float(0x7f800000);
  const int kvh = blockIdx.y, b = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = cache_len(p.kv_lens, b, p.n_cap);
  const int key0 = ((int)blockIdx.x - p.head_blocks) * CACHE_FINISH_KEYS;
  if (key0 >= len) return;
  const size_t head0 = (size_t)b * p.H_q + (size_t)kvh * p.group;
  const int nb = (len + p.block - 1) / p.block;
  // The segments of unit (kvh, hb): numbers [first, first + n).
  struct Segments {
    size_t first;
    int n;
  };
  const long long seq_at = nb ? p.seq_at[b] : 0;
  const CacheLine line(p, nb ? p.seq_at[p.B] : 1);
  auto segments = [&](int hb) {
    const int unit = kvh * p.head_blocks + hb;
    const long long x = seq_at + (long long)unit * nb;
    const int c0 = line.cta_of(x), c1 = line.cta_of(x + nb - 1);
    return Segments{(size_t)b * p.H_kv * p.head_blocks + unit + c0, c1 - c0 + 1};
  };
  // A unit's row by one warp: the reference m and the sum l of 2^(score - m) over all segments (0: no key counts).  They stay
  // apart, as m + log2 l would lose l beside a large m.
  auto row_stat = [&](const Segments& g, int row) {
    const float2* stat = p.part_stat + g.first * p.rows + row;
    const float2 mine = lane < g.n ? stat[(size_t)lane * p.rows] : make_float2(NEG_INF, 0.f);
    float M = mine.x;
    for (int s = lane + 32; s < g.n; s += 32) M = fmaxf(M, stat[(size_t)s * p.rows].x);
#pragma unroll
    for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    if (M == NEG_INF) M = 0.f;
    float L = exp2f(mine.x - M) * mine.y;
    for (int s = lane + 32; s < g.n; s += 32) {
      const float2 x = stat[(size_t)s * p.rows];
      L = fmaf(exp2f(x.x - M), x.y, L);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    return make_float2(M, L);
  };
  if (key0 < 0) {
    const int hb = blockIdx.x, heads = min(p.rows, p.group - hb * p.rows);
    const size_t first_head = head0 + hb * p.rows;
    if (nb == 0) {  // no key: 0 and -inf
      for (int i = threadIdx.x; i < heads * D; i += CACHE_FINISH_THREADS) p.O[first_head * D + i] = __float2bfloat16_rn(0.f);
      if (p.LSE && threadIdx.x < heads) p.LSE[first_head + threadIdx.x] = NEG_INF;
      return;
    }
    const Segments g = segments(hb);
    if (g.n == 1) return;  // written where it was computed
    // WARPS / rows warps per query head, each with every so-manieth segment; D / 32 channels per lane
    constexpr int E = D / 32;
    const int row = warp % p.rows, set = warp / p.rows, sets = WARPS / p.rows;
    float acc[E] = {};
    if (row < heads) {
      const float2 stat = row_stat(g, row);
      const float inv = stat.y == 0.f ? 0.f : 1.f / stat.y;
#pragma unroll 4
      for (int s = set; s < g.n; s += sets) {
        const size_t part = (g.first + s) * p.rows + row;
        const float2 x = p.part_stat[part];
        const float w = exp2f(x.x - stat.x) * x.y * inv;
        const float* v = p.part_o + part * D + lane * E;
        if constexpr (E == 4) {
          const float4 u = *reinterpret_cast<const float4*>(v);
          acc[0] = fmaf(w, u.x, acc[0]), acc[1] = fmaf(w, u.y, acc[1]), acc[2] = fmaf(w, u.z, acc[2]), acc[3] = fmaf(w, u.w, acc[3]);
        } else {
          const float2 u = *reinterpret_cast<const float2*>(v);
          acc[0] = fmaf(w, u.x, acc[0]), acc[1] = fmaf(w, u.y, acc[1]);
        }
      }
      if (p.LSE && set == 0 && lane == 0) p.LSE[first_head + row] = (stat.x + log2f(stat.y)) * 0.69314718055994531f;
    }
#pragma unroll
    for (int i = 0; i < E; ++i) s_o[warp][lane * E + i] = acc[i];
    __syncthreads();
    for (int i = threadIdx.x; i < heads * D; i += CACHE_FINISH_THREADS) {
      float v = 0.f;
      for (int w = i / D; w < WARPS; w += p.rows) v += s_o[w][i % D];
      p.O[first_head * D + i] = __float2bfloat16_rn(v);
    }
    return;
  }
  // Eight keys a thread, four and four.
  float w[2][4] = {};
  for (int h0 = 0; h0 < p.group; h0 += WARPS) {
    const int nh = min(WARPS, p.group - h0);
    if (h0) __syncthreads();
    if (warp < nh) {
      const float2 x = row_stat(segments((h0 + warp) / p.rows), (h0 + warp) % p.rows);
      if (lane == 0) s_stat[warp] = make_float2(x.x, x.y == 0.f ? 0.f : 1.f / x.y);
    }
    __syncthreads();
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int j = key0 + y * (CACHE_FINISH_KEYS / 2) + 4 * threadIdx.x;
      if (j < len) {
        const float* from = p.scores + (head0 + h0) * p.score_stride + j;
#pragma unroll 4
        for (int h = 0; h < nh; ++h) {
          const float4 v = __ldcs(reinterpret_cast<const float4*>(from + (size_t)h * p.score_stride));
          const float2 l = s_stat[h];
          w[y][0] = fmaf(exp2f(v.x - l.x), l.y, w[y][0]);
          w[y][1] = fmaf(exp2f(v.y - l.x), l.y, w[y][1]);
          w[y][2] = fmaf(exp2f(v.z - l.x), l.y, w[y][2]);
          w[y][3] = fmaf(exp2f(v.w - l.x), l.y, w[y][3]);
        }
      }
    }
  }
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int j = key0 + y * (CACHE_FINISH_KEYS / 2) + 4 * threadIdx.x;
    const size_t at = ((size_t)b * p.H_kv + kvh) * p.n_cap + j;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j + i < len) p.acc_out[at + i] = (p.acc ? p.acc[at + i] : 0.f) + w[y][i];
  }
}

}  // namespace sdpa
