// kv4.cuh -- writing rows into the 4-bit key/value cache and reading them back.
//
// A row's d channels form NG = d / 32 groups; group g has a scale s and a minimum m (bf16) and a 4-bit
// code per channel, x ~ s c + m.  Byte 2 (r NG + g) + e holds channels 32 g + 4 r + 2 e (low four bits)
// and + 1: a row is 8 chunks (r) of NG 16-bit pieces (g) of four channels.
//
// Both directions are streams (append: 2 d bytes in and d / 2 + d / 8 out per row, plus 2 d for the values
// read back; load: the reverse), so a thread moves 16 bytes of bf16 with one access: eight channels
// 32 g + 8 t .. + 7 (t = 0 .. 3), which are the pieces r = 2 t and 2 t + 1 of group g.  The four threads
// of a group find its extremes by shuffles.  Load runs at HBM's rate; append is bound by its instructions (about 180 per eight
// channels of 32 threads, at 2.7 per clock), then HBM: 4.85 TB/s for 250 MB.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "decode.cuh"
#include "sm100.cuh"

namespace sdpa {

struct Kv4Cache {
  uint8_t* codes;   // [B, H, n_cap, D / 2]
  uint32_t* scales; // [B, H, n_cap, NG] (s in bits 0 .. 15, m in bits 16 .. 31)
};

// Unsigned division by a number fixed at launch, for dividends below 2^31 (multiply high, then shift).
struct FastDiv {
  uint32_t d, mul, shift;
  static FastDiv of(uint32_t d) {
    FastDiv f = {d, 0, 0};
    while ((1ull << f.shift) < d) ++f.shift;  // 2^(shift - 1) < d <= 2^shift
    f.mul = (uint32_t)(((1ull << (31 + f.shift)) + d - 1) / d);  // ceil: exact for dividends below 2^31
    return f;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return (uint32_t)(((unsigned long long)n * mul) >> (31 + shift));
  }
};

struct Kv4RowsParams {
  Kv4Cache cache[2];          // K, V
  __nv_bfloat16* rows[2];     // [B, H, n_rows, D]
  __nv_bfloat16* read[2];     // append: the values read back, or null
  const int* kv_lens;         // [B]
  const int* n_new;           // append: [B] or null
  int B, H, n_rows, n_cap;
  FastDiv by_rows, by_heads;
};

__device__ __forceinline__ float bf16_bits_to_float(uint32_t bits) { return __uint_as_float(bits << 16); }

// The smallest bf16 number (its bits) not below (hi - lo) / 15, hi >= lo finite, for hi - lo < 2^128: the
// difference is kept exactly as the pair dh + dl (two-sum), the estimate is at most two steps low, and
// 15 s - dh - dl has the right sign because 15 s is exact and the fused step rounds once.
__device__ __forceinline__ uint32_t kv4_scale_bits(float lo, float hi) {
  const float dh = hi - lo;
  const float z = dh - hi;
  const float dl = (hi - (dh - z)) - (lo + z);
  uint32_t s = __float_as_uint(dh * (1.f / 15.f)) >> 16;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (fmaf(15.f, bf16_bits_to_float(s), -dh) < dl) ++s;
  return s;
}

// (x - lo) / s rounded to a whole number, halves to even, by the exact quotient, where its estimate is too near a half
// to tell; code: the estimate rounded.  x - lo = a + e exactly (two-sum), d = a - code s is exact (fused, and no
// more bits than a), and so is |d| - s / 2 next to a half; then e decides, and the code's parity where all is equal.
__device__ __forceinline__ float kv4_code_exact(float x, float lo, float s, float code) {
  const float a = x - lo;
  const float z = a - x;
  const float e = (x - (a - z)) - (lo + z);
  const float d = fmaf(-code, s, a);
  const float one = copysignf(1.f, d);
  const float over = fmaf(-0.5f, s, fabsf(d)), rest = -one * e;  // past the half by over - rest
  return over > rest || (over == rest && ((int)code & 1)) ? code + one : code;
}

// Smaller and larger of two pairs of bf16, NaN if either is.
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Lane-wise product of two pairs.
__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  float2 r;
  asm("{ .reg .b64 x, y, z; mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mul.rn.f32x2 z, x, y; mov.b64 {%0, %1}, z; }"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// The codes (as floats, and packed) of eight channels x of a group with minimum lo and scale s, inv its reciprocal.
__device__ __forceinline__ uint32_t kv4_codes(const float (&x)[8], float lo, float s, float inv, float (&code)[8]) {
  float t[8], far = 0.f;
  constexpr float ROUND = 12582912.f;  // 1.5 2^23: adding it rounds to a whole number, halves to even
  const float2 low = make_float2(-lo, -lo), up = make_float2(ROUND, ROUND), back = make_float2(-ROUND, -ROUND);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {  // in pairs: half the instructions
    const float2 q = fmul2(sm100::fadd2(make_float2(x[i], x[i + 1]), low), make_float2(inv, inv));  // within 1e-5 of the quotients
    const float2 c = sm100::fadd2(sm100::fadd2(q, up), back);
    const float2 off = sm100::ffma2(c, make_float2(-1.f, -1.f), q);
    t[i] = q.x, t[i + 1] = q.y, code[i] = c.x, code[i + 1] = c.y;
    far = sm100::max3f(far, fabsf(off.x), fabsf(off.y));
  }
  if (far > 0.49998f) {  // one of them is near a half
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (fabsf(t[i] - code[i]) > 0.49998f) code[i] = kv4_code_exact(x[i], lo, s, code[i]);
  }
  // 16-bit pieces as whole numbers in fp32, read off the sum with 2^23
  const float p0 = fmaf(code[3], 4096.f, fmaf(code[2], 256.f, fmaf(code[1], 16.f, code[0] + 8388608.f)));
  const float p1 = fmaf(code[7], 4096.f, fmaf(code[6], 256.f, fmaf(code[5], 16.f, code[4] + 8388608.f)));
  return __byte_perm(__float_as_uint(p0), __float_as_uint(p1), 0x5410);
}
__device__ __forceinline__ float kv4_reciprocal(float s) {
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  return inv;
}

// The smallest (low half) and minus the largest of this thread's eight channels.
__device__ __forceinline__ uint32_t kv4_extremes(const uint4 raw) {
  const uint32_t mn = min_bf16x2(min_bf16x2(raw.x, raw.y), min_bf16x2(raw.z, raw.w));
  const uint32_t mx = max_bf16x2(max_bf16x2(raw.x, raw.y), max_bf16x2(raw.z, raw.w));
  const uint32_t both = min_bf16x2(__byte_perm(mn, mx, 0x5410), __byte_perm(mn, mx, 0x7632));
  return (both & 0xFFFFu) | ((max_bf16x2(mx, mx >> 16) << 16) ^ 0x80000000u);
}

// The codes of this thread's eight channels (as floats and packed), and the group's scale (bits 0 .. 15) and minimum.
// The four threads of a group are lanes differing in bits 0 and 1.  both: kv4_extremes.
__device__ __forceinline__ uint32_t kv4_quantise(const uint4 raw, uint32_t both, uint32_t& scale, float (&code)[8]) {
  both = min_bf16x2(both, __shfl_xor_sync(0xffffffffu, both, 1));
  both = min_bf16x2(both, __shfl_xor_sync(0xffffffffu, both, 2));
  float lo = __uint_as_float(both << 16), hi = -__uint_as_float(both & 0xFFFF0000u);
#pragma unroll
  for (int i = 0; i < 8; ++i) code[i] = 0.f;
  if (!(lo >= -FLT_MAX && hi <= FLT_MAX)) {  // a NaN or an infinity
    scale = 0x7FC07FC0u;
    return 0u;
  }
  // Differences of values near the largest float would overflow: work 2^-16 smaller there.
  const float big = fmaxf(fabsf(lo), fabsf(hi));
  const float down = big > 0x1p120f ? 0x1p-16f : 1.f;
  const float s_down = bf16_bits_to_float(kv4_scale_bits(lo * down, hi * down));
  const uint32_t scale_bits = __float_as_uint(s_down * (big > 0x1p120f ? 0x1p16f : 1.f)) >> 16;
  scale = scale_bits | (both << 16);
  if (s_down == 0.f) return 0u;
  // and the reciprocal of a tiny scale would: work 2^64 larger there (both factors are exact)
  const float f = big < 0x1p-60f ? 0x1p64f : down;
  const float s = bf16_bits_to_float(scale_bits) * f;
  float x[8];
  bf16x8_to_f32(raw, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= f;
  return kv4_codes(x, lo * f, s, kv4_reciprocal(s), code);
}

// The scales of four rows at once where no group of the warp is out of the ordinary (a NaN, an infinity, all values
// equal, numbers that the above moves to another range): each of a group's four threads works one row's out, and all get
// them by shuffles.  Returns whether that holds.
__device__ __forceinline__ bool kv4_scales(const uint32_t (&both)[4], int lane, uint32_t (&scale)[4], float (&inv)[4]) {
  const bool b0 = lane & 1, b1 = lane & 2;
  uint32_t k0 = b1 ? both[2] : both[0], k1 = b1 ? both[3] : both[1];
  k0 = min_bf16x2(k0, __shfl_xor_sync(0xffffffffu, b1 ? both[0] : both[2], 2));
  k1 = min_bf16x2(k1, __shfl_xor_sync(0xffffffffu, b1 ? both[1] : both[3], 2));
  const uint32_t mine = min_bf16x2(b0 ? k1 : k0, __shfl_xor_sync(0xffffffffu, b0 ? k0 : k1, 1));
  const float lo = __uint_as_float(mine << 16), hi = -__uint_as_float(mine & 0xFFFF0000u);
  const float big = fmaxf(fabsf(lo), fabsf(hi));
  const bool plain = lo < hi && big <= 0x1p120f && big >= 0x1p-60f;  // false for NaN
  if (!__all_sync(0xffffffffu, plain)) return false;
  const uint32_t bits = kv4_scale_bits(lo, hi);
  const float r = kv4_reciprocal(bf16_bits_to_float(bits));
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    scale[u] = __shfl_sync(0xffffffffu, bits | (mine << 16), u, 4);
    inv[u] = __shfl_sync(0xffffffffu, r, u, 4);
  }
  return true;
}

// A thread's eight codes are the 16-bit pieces r = 2 t (low half) and 2 t + 1 (high half) of its group; the
// 4 NG bytes from byte 4 NG t on hold piece 2 t of every group, then piece 2 t + 1 of every group.
// Between the threads with the same t (lanes 4 g + t, g < NG): to word g of those bytes, and back.
template <int NG>
__device__ __forceinline__ uint32_t kv4_to_words(uint32_t codes, int lane) {
  const int g = (lane >> 2) & (NG - 1), base = lane & ~((NG - 1) << 2);
  const int g0 = (2 * g) & (NG - 1);               // word g: pieces of groups g0 and g0 + 1 ...
  const uint32_t a = __shfl_sync(0xffffffffu, codes, base | (g0 << 2));
  const uint32_t b = __shfl_sync(0xffffffffu, codes, base | ((g0 + 1) << 2));
  return __byte_perm(a, b, g >= NG / 2 ? 0x7632 : 0x5410);  // ... the second half of the words: pieces 2 t + 1
}
template <int NG>
__device__ __forceinline__ uint32_t kv4_from_words(uint32_t word, int lane) {
  const int g = (lane >> 2) & (NG - 1), base = lane & ~((NG - 1) << 2);
  const uint32_t a = __shfl_sync(0xffffffffu, word, base | ((g >> 1) << 2));
  const uint32_t b = __shfl_sync(0xffffffffu, word, base | ((NG / 2 + (g >> 1)) << 2));
  return __byte_perm(a, b, (g & 1) ? 0x7632 : 0x5410);
}

// s c + m for eight codes, rounded to bf16 (s c is exact in fp32).
__device__ __forceinline__ uint4 kv4_values(const float (&code)[8], uint32_t scale) {
  const float s = __uint_as_float(scale << 16), m = __uint_as_float(scale & 0xFFFF0000u);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = sm100::ffma2(make_float2(code[2 * i], code[2 * i + 1]), make_float2(s, s), make_float2(m, m));
    w[i] = sm100::pack_bf16x2(x.x, x.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Eight packed codes as floats: two at a time as fp16 1024 + c, which is exact.
__device__ __forceinline__ void kv4_unpack(uint32_t codes, float (&code)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // channels i and 4 + i
    const uint32_t h = ((codes >> (4 * i)) & 0x000F000Fu) | 0x64006400u;
    const float2 v = __half22float2(__hsub2(*reinterpret_cast<const __half2*>(&h), __float2half2_rn(1024.f)));
    code[i] = v.x;
    code[4 + i] = v.y;
  }
}

// Blocks of 128 threads at 64 registers (append spills 52 bytes at that limit).  4 x 8 heads, d = 128: append of 5001-8192 rows 51.7 us, load of 9001-16384 rows 45.3 us;
// 256 threads at 78 registers 57.2 and 47.0 us, at 64 registers 51.8 and 46.9 us, 128 threads at 72 and 56 registers 53.0
// and 51.1 us (append), 64 threads 51.5 and 46.3 us.
constexpr int KV4_THREADS = 128;
constexpr int KV4_BLOCKS = 8;  // per SM
constexpr int KV4_UNROLL = 4;  // rows a thread has in flight

// Length of sequence b clamped to [0, n_cap]; anything else is recorded.
__device__ __forceinline__ int cache_len(const int* kv_lens, int b, int n_cap) {
  const int len = kv_lens[b];
  if (len >= 0 && len <= n_cap) return len;
  record_error(7 /* SDPA_ERR_DEVICE_BAD_LENGTH */);
  return len < 0 ? 0 : n_cap;
}

// What a thread moves: KV4_UNROLL rows' parts, each at its own place.
template <int NG, bool LOAD, class Place>
__device__ __forceinline__ void kv4_move(const Place& place, bool want_read, int lane, bool first_of_group) {
  if (LOAD) {
    uint32_t word[KV4_UNROLL], scale[KV4_UNROLL];
#pragma unroll
    for (int u = 0; u < KV4_UNROLL; ++u) {
      word[u] = place.on(u) ? *place.codes(u) : 0u;
      scale[u] = place.on(u) ? *place.scales(u) : 0u;
    }
#pragma unroll
    for (int u = 0; u < KV4_UNROLL; ++u) {
      float code[8];
      kv4_unpack(kv4_from_words<NG>(word[u], lane), code);
      if (place.on(u)) *place.row(u) = kv4_values(code, scale[u]);
    }
  } else {
    uint4 raw[KV4_UNROLL];
#pragma unroll
    for (int u = 0; u < KV4_UNROLL; ++u) raw[u] = place.on(u) ? ld_nc_v4(place.row(u)) : make_uint4(0x3F800000u, 0, 0, 0);  // an ordinary row
    static_assert(KV4_UNROLL == 4, "a row for each of a group's four threads");
    uint32_t both[KV4_UNROLL], scales[KV4_UNROLL];
    float inv[KV4_UNROLL];
#pragma unroll
    for (int u = 0; u < KV4_UNROLL; ++u) both[u] = kv4_extremes(raw[u]);
    auto put = [&](int u, uint32_t codes, uint32_t scale, const float (&code)[8]) {
      const uint32_t word = kv4_to_words<NG>(codes, lane);
      if (place.on(u)) {
        *place.codes(u) = word;
        if (first_of_group) *place.scales(u) = scale;
        if (want_read) *place.read(u) = kv4_values(code, scale);
      }
    };
    float code[8];
    if (kv4_scales(both, lane, scales, inv)) {
#pragma unroll
      for (int u = 0; u < KV4_UNROLL; ++u) {
        float x[8];
        bf16x8_to_f32(raw[u], x);
        put(u, kv4_codes(x, __uint_as_float(scales[u] & 0xFFFF0000u), bf16_bits_to_float(scales[u] & 0xFFFFu), inv[u], code),
            scales[u], code);
      }
    } else {
#pragma unroll
      for (int u = 0; u < KV4_UNROLL; ++u) {
        uint32_t scale;
        const uint32_t codes = kv4_quantise(raw[u], both[u], scale, code);
        put(u, codes, scale, code);
      }
    }
  }
}

// LOAD false: append.  Grid: x blocks over the B H n_rows row slots, y: K, V.  A block whose rows are all of one
// sequence and head (every block of a long prompt) knows its places as one base and fixed offsets, and leaves at once where no
// row is to be moved; the others (single tokens) find each row's place by itself.
template <int D, bool LOAD>
__global__ void __launch_bounds__(KV4_THREADS, KV4_BLOCKS) sdpa_kv4_rows_kernel(const Kv4RowsParams p) {
  constexpr int NG = D / 32, TPR = D / 8;  // threads per row
  constexpr int RPB = KV4_THREADS / TPR;   // rows per block and pass
  const int lane = threadIdx.x & 31;
  const int part = threadIdx.x % TPR, g = part >> 2, t = part & 3, mine = threadIdx.x / TPR;
  const bool second = blockIdx.y != 0;
  uint8_t* codes = (second ? p.cache[1].codes : p.cache[0].codes) + 4 * (t * NG + g);
  uint32_t* scales = (second ? p.cache[1].scales : p.cache[0].scales) + g;
  __nv_bfloat16* rows = (second ? p.rows[1] : p.rows[0]) + 8 * part;
  __nv_bfloat16* read = second ? p.read[1] : p.read[0];
  const bool want_read = read != nullptr;
  if (want_read) read += 8 * part;
  const uint32_t total = (uint32_t)p.B * p.H * p.n_rows, first = blockIdx.x * (uint32_t)(RPB * KV4_UNROLL);
  // Rows of sequence b that are moved, and the cache row of the first.
  auto limits = [&](uint32_t b, int& limit, int& to) {
    const int len = cache_len(p.kv_lens, b, p.n_cap);
    to = LOAD ? 0 : len;
    limit = len;
    if (!LOAD) {
      const int n = p.n_new ? p.n_new[b] : p.n_rows;
      if (n < 0 || n > p.n_rows || n > p.n_cap - len) record_error(7 /* SDPA_ERR_DEVICE_BAD_LENGTH */);
      limit = min(n, p.n_cap - len);
    }
    limit = min(limit, p.n_rows);
  };
  const uint32_t bh0 = p.by_rows.div(first), row0 = first - bh0 * p.n_rows;
  if (row0 + RPB * KV4_UNROLL <= (uint32_t)p.n_rows) {
    struct Place {
      uint8_t *c, *s, *x, *r;
      int left;  // rows from this thread's first one to the limit
      __device__ __forceinline__ bool on(int u) const { return u * RPB < left; }
      __device__ __forceinline__ uint32_t* codes(int u) const { return (uint32_t*)(c + u * (RPB * (D / 2))); }
      __device__ __forceinline__ uint32_t* scales(int u) const { return (uint32_t*)(s + u * (RPB * NG * 4)); }
      __device__ __forceinline__ uint4* row(int u) const { return (uint4*)(x + u * (RPB * D * 2)); }
      __device__ __forceinline__ uint4* read(int u) const { return (uint4*)(r + u * (RPB * D * 2)); }
    };
    int limit, to;
    limits(p.by_heads.div(bh0), limit, to);
    if ((int)row0 >= limit) return;
    const int row = (int)row0 + mine;
    const size_t cache_row = (size_t)bh0 * p.n_cap + to + row, at = (size_t)(first + mine) * D;
    const Place place = {codes + cache_row * (D / 2), (uint8_t*)(scales + cache_row * NG), (uint8_t*)(rows + at),
                         (uint8_t*)(want_read ? read + at : nullptr), limit - row};
    kv4_move<NG, LOAD>(place, want_read, lane, t == 0);
  } else {
    struct Place {
      uint32_t *c[KV4_UNROLL], *s[KV4_UNROLL];
      uint4 *x[KV4_UNROLL], *r[KV4_UNROLL];
      bool o[KV4_UNROLL];
      __device__ __forceinline__ bool on(int u) const { return o[u]; }
      __device__ __forceinline__ uint32_t* codes(int u) const { return c[u]; }
      __device__ __forceinline__ uint32_t* scales(int u) const { return s[u]; }
      __device__ __forceinline__ uint4* row(int u) const { return x[u]; }
      __device__ __forceinline__ uint4* read(int u) const { return r[u]; }
    } place;
#pragma unroll
    for (int u = 0; u < KV4_UNROLL; ++u) {
      const uint32_t slot = first + mine + u * RPB;
      place.o[u] = false;
      if (slot < total) {
        const uint32_t bh = p.by_rows.div(slot), row = slot - bh * p.n_rows;
        int limit, to;
        limits(p.by_heads.div(bh), limit, to);
        place.o[u] = (int)row < limit;
        const size_t cache_row = (size_t)bh * p.n_cap + to + row, at = (size_t)slot * D;
        place.c[u] = (uint32_t*)(codes + cache_row * (D / 2));
        place.s[u] = scales + cache_row * NG;
        place.x[u] = (uint4*)(rows + at);
        if (want_read) place.r[u] = (uint4*)(read + at);
      }
    }
    kv4_move<NG, LOAD>(place, want_read, lane, t == 0);
  }
}

}  // namespace sdpa
