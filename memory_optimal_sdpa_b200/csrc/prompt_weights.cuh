// prompt_weights.cuh -- the attention weights of a prompt, summed over its queries, on the sm_100a tensor cores.
//
//     w_j = sum over the heads h of a group and the queries i that see key j of 2^(c q_hi . k_j - L_hi)
//
// (c = scale log2 e, L the base-2 log-sum-exp): the scores of a prefill once more, but with the sums along the
// other axis and nothing else kept.  So the keys are the rows of the product, S^T = K Q^T: a thread of the softmax
// warps owns a key (a TMEM lane), walks over the queries (columns) and keeps the key's sum in registers.  No
// running maximum, no exchange between threads, no atomics; the order of the sums is fixed.
//
// A unit of work is 128 MT keys of one (sequence, key/value head); its queries stream past in tiles of 128, head
// after head.  MT = 2 halves the waits of the producer and the MMA issuer and the L2 traffic of the queries, but a unit is
// the least that an SM can be given: MT = 1 where the heaviest unit of 256 keys, which sees all queries, is more than 15 % above an
// SM's share.  Measured, MT = 2 against 1, us (causal, calls back to back): 32 heads over 8, d = 128, n = 4096 175 and 94, 6000 256
// and 198, 7000 296 and 260, 8192 (14 % above) 340 and 344, 9472 423 and 442, 32768 5111 and 5388; the last 64 queries of
// 2 x 32 heads over 8, 16001 keys 39 and 47, the last 512 162 and 166; of 4 x 16 heads, d = 64, 16001 keys 45 and 55, of 1 x 32 heads over 8,
// 2000 keys 14.3 and 12.3.  What bounds it: for many queries the exponentials (16
// per clock and SM on the MUFU unit, so 1024 clocks for 128 x 128 scores, against 512 for the MMA at d = 128; 239 us for the
// former case, whose heaviest unit is also 12 % above an SM's share).  For few queries the hand-offs of a
// unit and its exponentials in a chain (about 3000 clocks for 256 keys and 64 queries), not HBM (21 us for the latter case).
//
// Warps: 0 TMA producer, 1 MMA issuer and TMEM owner, 2 and 3 log-sum-exps into shared memory, then softmax groups of
// four warps.  S^T stages: 512 / (128 MT) in TMEM, so the MMA runs ahead across units.  Query tile i of a CTA goes to the
// groups of turn i mod TURNS (one group for each 128 keys), so that a stage always meets the same groups and they
// wait for each of its phases in order: a parity cannot be mistaken for a later one.  At the end of a unit the group that had its last
// tile collects the other turns' sums through shared memory (monotonic counters, two slots) and stores.  640 threads leave 96 registers
// each, at which MT = 2 spills 20 bytes.
#pragma once

#include "kv4.cuh"
#include "prefill_bf16.cuh"

namespace sdpa {

struct PromptWeightsParams {
  const float* LSE;        // [B, Hq, n_q], natural
  const float* acc;        // [B, Hkv, n_acc] or null
  float* acc_out;
  int heads_q, heads_kv, group, n_q, n_kv, n_acc, causal;
  int bkv, n_kt;           // B Hkv; key units per (sequence, key/value head)
  float scale_log2;        // scale log2 e, or a quarter of it
  int quarter;             // log2 e takes the largest scales out of range: their products are multiplied by 4 first
};

template <int D, int MT>
struct PromptCfg {
  static constexpr int TILE_BYTES = 128 * D * 2;
  static constexpr int BLOCK_BYTES = 128 * 64 * 2;  // one 64-channel swizzle block
  static constexpr int KSLOT = D == 128 ? (MT == 2 ? 2 : 3) : (MT == 2 ? 4 : 6);
  static constexpr int QSLOT = D == 128 ? (MT == 2 ? 2 : 3) : (MT == 2 ? 4 : 6);
  static constexpr int NSTAGE = 512 / (128 * MT);
  static constexpr int K_OFF = 0;
  static constexpr int Q_OFF = KSLOT * MT * TILE_BYTES;
  static constexpr int GROUPS = 4;  // of softmax warps (two: 394 us against 355 us for 32 heads, n = 8192, causal)
  static constexpr int TURNS = GROUPS / MT;
  static_assert(NSTAGE % TURNS == 0, "a stage belongs to one turn");
  static constexpr int LSE_OFF = Q_OFF + QSLOT * TILE_BYTES;  // [NSTAGE][128]
  static constexpr int CNT_OFF = LSE_OFF + NSTAGE * 128 * 4;  // [2][TURNS][TURNS][MT * 4]: sums sent, sums collected
  static constexpr int CNT = TURNS * TURNS * MT * 4;
  static constexpr int SUM_OFF = CNT_OFF + 2 * CNT * 4;        // [2][TURNS][TURNS][MT * 128]
  static constexpr int BAR_OFF = SUM_OFF + 2 * TURNS * TURNS * MT * 128 * 4;
  // k_full, k_empty, q_full, q_empty, s_full, s_free, drain
  static constexpr int NBAR = 2 * KSLOT + 2 * QSLOT + 2 * NSTAGE * MT + 1;
  static constexpr int SMEM_BYTES = BAR_OFF + NBAR * 8 + 16 + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory of an SM");
  static constexpr int THREADS = 128 + 128 * GROUPS;
};

// The sum of 2^(s c2 - L) over 16 columns, added to `sum` (two partial sums).  MASKED: columns below `first` and from `end`
// on count 0, whatever their scores are (a row of zeros that stands for no query gives NaN with an infinite key).
// All exponentials on the MUFU unit: every 8th pair by a degree-5 polynomial on the FMA pipe measured 1.5 % faster for
// many queries and slower for few, every 4th and 2nd 0 and 10 % slower for many.
template <bool MASKED>
__device__ __forceinline__ float2 prompt_chunk(const uint32_t (&s)[16], float c2, const float4* L, int first, int end,
                                               float2 sum) {
  using namespace sm100;
  float2 a0 = make_float2(0.f, 0.f), a1 = a0;
  const float2 cc = make_float2(c2, c2);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 l = L[i];  // minus the log-sum-exps
    const float2 x0 = ffma2(make_float2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), cc, make_float2(l.x, l.y));
    const float2 x1 = ffma2(make_float2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), cc, make_float2(l.z, l.w));
    float2 e0 = make_float2(ex2_approx(x0.x), ex2_approx(x0.y)), e1 = make_float2(ex2_approx(x1.x), ex2_approx(x1.y));
    if (MASKED) {
      if (4 * i < first || 4 * i >= end) e0.x = 0.f;
      if (4 * i + 1 < first || 4 * i + 1 >= end) e0.y = 0.f;
      if (4 * i + 2 < first || 4 * i + 2 >= end) e1.x = 0.f;
      if (4 * i + 3 < first || 4 * i + 3 >= end) e1.y = 0.f;
    }
    a0 = fadd2(a0, e0);
    a1 = fadd2(a1, e1);
  }
  return fadd2(sum, fadd2(a0, a1));
}

template <int D, int MT>
__global__ void __launch_bounds__(PromptCfg<D, MT>::THREADS, 1)
    sdpa_prompt_weights_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                               const PromptWeightsParams p) {
  using C = PromptCfg<D, MT>;
  using namespace sm100;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sK = smem + C::K_OFF;
  uint8_t* sQ = smem + C::Q_OFF;
  float* sL = (float*)(smem + C::LSE_OFF);
  uint32_t* sent = (uint32_t*)(smem + C::CNT_OFF);  // [from turn][to turn][key warp]
  uint32_t* collected = sent + C::CNT;
  float* sums = (float*)(smem + C::SUM_OFF);
  uint64_t* k_full = (uint64_t*)(smem + C::BAR_OFF);
  uint64_t* k_empty = k_full + C::KSLOT;
  uint64_t* q_full = k_empty + C::KSLOT;
  uint64_t* q_empty = q_full + C::QSLOT;
  uint64_t* s_full = q_empty + C::QSLOT;
  uint64_t* s_free = s_full + C::NSTAGE * MT;  // [stage][128 keys]
  uint64_t* drain = s_free + C::NSTAGE * MT;
  uint32_t* tmem_slot = (uint32_t*)(drain + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::KSLOT; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::QSLOT; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < C::NSTAGE * MT; ++i) {
      mbar_init(&s_full[i], 2);  // the product and the log-sum-exps
      mbar_init(&s_free[i], 4);  // the warps of the group that reads it
    }
    mbar_init(drain, 1);
    for (int i = 0; i < 2 * C::CNT; ++i) sent[i] = 0;
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  bool timed_out = false;
  const bool tmem_bad = tmem_alloc_bad(tmem);  // debug builds only

  // Units: key unit by key unit, the (sequence, key/value head) slices side by side; under a causal mask the first
  // keys have the most queries, so the heaviest come first, and successive rounds are dealt in alternating directions.
  // (Round k of CTA b, of G: unit k G + b, or (k + 1) G - 1 - b where k is odd.  A walk steps from one to the next without
  // a division: with one query tile a unit, the roles' own arithmetic is what a unit costs.)
  const int n_units = p.bkv * p.n_kt, off = p.n_kv - p.n_q, n_qt = (p.n_q + 127) / 128;
  const int step_even = 2 * ((int)gridDim.x - 1 - (int)blockIdx.x) + 1, step_odd = 2 * (int)blockIdx.x + 1;
  const int even_q = step_even / p.bkv, even_r = step_even % p.bkv, odd_q = step_odd / p.bkv, odd_r = step_odd % p.bkv;
  struct Unit {
    int u, k;       // number, round
    int kt, bkv;    // u / p.bkv, u % p.bkv
    int key0, qt0;  // first key; query tiles [qt0, n_qt) of every head of the group
  };
  auto place = [&](Unit& g) {
    g.key0 = g.kt * (128 * MT);
    const int first = p.causal ? g.key0 - off : 0;  // the first query that sees the unit's first key
    g.qt0 = first > 0 ? first / 128 : 0;
    return g.u < n_units;
  };
  auto begin = [&](Unit& g) {
    g.u = (int)blockIdx.x;
    g.k = 0;
    g.kt = g.u / p.bkv;
    g.bkv = g.u % p.bkv;
    return place(g);
  };
  auto advance = [&](Unit& g) {
    const bool odd = g.k & 1;
    g.u += odd ? step_odd : step_even;
    g.kt += odd ? odd_q : even_q;
    g.bkv += odd ? odd_r : even_r;
    if (g.bkv >= p.bkv) {
      g.bkv -= p.bkv;
      ++g.kt;
    }
    ++g.k;
    return place(g);
  };
  auto q_head = [&](int bkv, int h) { return bkv * p.group + h; };  // row of [B Hq]

  if (tmem_bad) {
  } else if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      int nk = 0, nq = 0;  // units and query tiles loaded
      bool ok = true;
      Unit g;
      for (bool more = begin(g); ok && more; more = advance(g)) {
        if (g.qt0 >= n_qt) continue;
        const int ks = nk % C::KSLOT;
        if (!(ok = mbar_wait_bounded(&k_empty[ks], ((uint32_t)(nk / C::KSLOT) & 1u) ^ 1u, abort_flag, &timed_out))) break;
        mbar_arrive_expect_tx(&k_full[ks], MT * C::TILE_BYTES);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sK + (ks * MT + m) * C::TILE_BYTES + c * C::BLOCK_BYTES, &tmK, &k_full[ks], 64 * c, g.key0 + 128 * m,
                        g.bkv);
        ++nk;
        for (int h = 0; ok && h < p.group; ++h)
          for (int qt = g.qt0; qt < n_qt; ++qt) {
            const int qs = nq % C::QSLOT;
            if (!(ok = mbar_wait_bounded(&q_empty[qs], ((uint32_t)(nq / C::QSLOT) & 1u) ^ 1u, abort_flag, &timed_out))) break;
            mbar_arrive_expect_tx(&q_full[qs], C::TILE_BYTES);
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(sQ + qs * C::TILE_BYTES + c * C::BLOCK_BYTES, &tmQ, &q_full[qs], 64 * c, 128 * qt, q_head(g.bkv, h));
            ++nq;
          }
      }
      if (*abort_flag) {  // let the copies in flight land before the CTA exits
        for (int i = nk > C::KSLOT ? nk - C::KSLOT : 0; i < nk; ++i)
          mbar_wait_drain(&k_full[i % C::KSLOT], (uint32_t)(i / C::KSLOT) & 1u);
        for (int i = nq > C::QSLOT ? nq - C::QSLOT : 0; i < nq; ++i)
          mbar_wait_drain(&q_full[i % C::QSLOT], (uint32_t)(i / C::QSLOT) & 1u);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t id = idesc_bf16_f32(128, 128, false, false);
      const uint64_t dK = smem_desc_sw128(smem_u32(sK), 16, 1024), dQ = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      int nk = 0, nq = 0;
      bool ok = true;
      Unit g;
      for (bool more = begin(g); ok && more; more = advance(g)) {
        if (g.qt0 >= n_qt) continue;
        const int ks = nk % C::KSLOT;
        if (!(ok = mbar_wait_bounded(&k_full[ks], (uint32_t)(nk / C::KSLOT) & 1u, abort_flag, &timed_out))) break;
        const int tiles = p.group * (n_qt - g.qt0);
        for (int i = 0; i < tiles; ++i, ++nq) {
          const int qs = nq % C::QSLOT, st = nq % C::NSTAGE;
          if (!(ok = mbar_wait_bounded(&q_full[qs], (uint32_t)(nq / C::QSLOT) & 1u, abort_flag, &timed_out))) break;
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            if (!(ok = ok && mbar_wait_bounded(&s_free[st * MT + m], ((uint32_t)(nq / C::NSTAGE) & 1u) ^ 1u, abort_flag,
                                               &timed_out)))
              break;
            tc_fence_after_sync();  // the stage's last reads come before this product
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t o = ((kk >> 2) * C::BLOCK_BYTES) + (kk & 3) * 32;
              mma_ss(tmem + (uint32_t)((st * MT + m) * 128), dK + (uint64_t)(((ks * MT + m) * C::TILE_BYTES + o) >> 4),
                     dQ + (uint64_t)((qs * C::TILE_BYTES + o) >> 4), id, kk > 0 ? 1u : 0u);
            }
            tc_commit(&s_full[st * MT + m]);
          }
          if (!ok) break;
          tc_commit(&q_empty[qs]);
        }
        if (!ok) break;
        tc_commit(&k_empty[ks]);
        ++nk;
      }
      tc_commit(drain);
      mbar_wait_drain(drain, 0);
    }
  } else if (warp <= 3) {
    // ------------------------------------------------------------------ log-sum-exps, negated, base 2
    // Two warps take turns; each has its next tile's values on the way while it waits for a stage.
    struct Walk {  // over the query tiles of this CTA
      int h, qt;
      Unit g;
    };
    auto settle = [&](Walk& x, bool more) {  // on to a unit with tiles; false: none is left
      while (more && x.g.qt0 >= n_qt) more = advance(x.g);
      x.h = 0;
      x.qt = x.g.qt0;
      return more;
    };
    auto next = [&](Walk& x) {
      if (++x.qt < n_qt) return true;
      if (++x.h < p.group) {
        x.qt = x.g.qt0;
        return true;
      }
      return settle(x, advance(x.g));
    };
    auto fetch = [&](const Walk& x, float (&v)[4]) {
      const float* L = p.LSE + (size_t)q_head(x.g.bkv, x.h) * p.n_q;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 128 * x.qt + 32 * i + lane;
        v[i] = row < p.n_q ? __ldg(L + row) : -__int_as_float(0x7f800000);
      }
      // A new unit: its keys' weights on the way to L2, for the groups to add to (loaded at the unit's start instead they took
      // a register too many and their latency: 47.4 us against 43.9 for the last 64 queries above).
      if (p.acc && x.h == 0 && x.qt == x.g.qt0 && lane < 4 * MT && x.g.key0 + 32 * lane < p.n_kv)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.acc + (size_t)x.g.bkv * p.n_acc + x.g.key0 + 32 * lane));
    };
    Walk x;
    bool more = begin(x.g);
    more = settle(x, more);
    if (more && warp == 3) more = next(x);
    float v[4];
    if (more) fetch(x, v);
    for (int nq = warp - 2; more; nq += 2) {
      float next_v[4] = {};
      more = next(x) && next(x);
      if (more) fetch(x, next_v);
      const int st = nq % C::NSTAGE;
      bool free = true;
#pragma unroll
      for (int m = 0; m < MT; ++m)
        free = free && mbar_wait_bounded(&s_free[st * MT + m], ((uint32_t)(nq / C::NSTAGE) & 1u) ^ 1u, abort_flag, &timed_out);
      if (!__all_sync(0xffffffffu, free)) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y = -1.4426950408889634f * v[i];
        // a query that sees no key (LSE -inf) or does not exist adds nothing
        sL[st * 128 + 32 * i + lane] = y == __int_as_float(0x7f800000) ? -y : y;
      }
      __syncwarp();
      if (lane < MT) mbar_arrive(&s_full[st * MT + lane]);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = next_v[i];  // after the arrival: it waits for them
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------ softmax groups
    const int grp = (warp - 4) >> 2, q4 = warp & 3;
    const int m = grp % MT, turn = grp / MT, kw = 4 * m + q4;  // kw: which 32 keys of the unit
    const uint32_t lane_base = (uint32_t)(32 * q4) << 16;
    const float c2 = p.scale_log2;
    int nq = 0;             // query tiles of the units so far
    uint32_t n_sent[C::TURNS] = {}, n_got[C::TURNS] = {};  // sums sent to and collected from each turn
    bool ok = true;
    Unit g;
    for (bool more = begin(g); ok && more; more = advance(g)) {
      const int tiles_head = n_qt - g.qt0 > 0 ? n_qt - g.qt0 : 0, tiles = p.group * tiles_head;
      const int key = g.key0 + 32 * kw + lane;
      const int warp_last = g.key0 + 32 * kw + 31;  // the warp's last key: masks the most
      const size_t at = (size_t)g.bkv * p.n_acc + key;
      float w = 0.f;
      const int skip = (turn - nq % C::TURNS + C::TURNS) % C::TURNS;  // this turn's first tile of the unit
      int qt = g.qt0 + (tiles_head ? skip % tiles_head : 0);
      for (int i = skip; i < tiles; i += C::TURNS) {
        const int st = (nq + i) % C::NSTAGE;
        ok = __all_sync(0xffffffffu,
                        mbar_wait_bounded(&s_full[st * MT + m], (uint32_t)((nq + i) / C::NSTAGE) & 1u, abort_flag, &timed_out));
        if (!ok) break;
        tc_fence_after_sync();
        const int row0 = 128 * qt;
        const int cols = p.n_q - row0 < 128 ? p.n_q - row0 : 128;
        const uint32_t ta = tmem + (uint32_t)((st * MT + m) * 128) + lane_base;
        const float4* L = reinterpret_cast<const float4*>(sL + st * 128);
        // query row0 + c sees the key iff c >= key - off - row0
        const int first = p.causal ? key - off - row0 : 0;
        const bool masked = p.causal && warp_last - off - row0 > 0;
        float2 part = make_float2(0.f, 0.f);
        uint32_t s[2][16];
        tmem_ld_32x32b_x16(ta, s[0]);
        const int plain = masked || p.quarter ? 0 : cols;  // columns that are just added up
        if (plain == 128) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            tmem_wait_ld();
            reg_fence(s[c & 1]);
            if (c < 7) tmem_ld_32x32b_x16(ta + (uint32_t)(16 * (c + 1)), s[(c + 1) & 1]);
            part = prompt_chunk<false>(s[c & 1], c2, L + 4 * c, 0, 16, part);
          }
        } else {
#pragma unroll 1
          for (int c = 0; 16 * c < cols; c += 2)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              tmem_wait_ld();
              reg_fence(s[y]);
              if (c + y < 7) tmem_ld_32x32b_x16(ta + (uint32_t)(16 * (c + y + 1)), s[y ^ 1]);
              if (16 * (c + y + 1) <= plain) {
                part = prompt_chunk<false>(s[y], c2, L + 4 * (c + y), 0, 16, part);
                continue;
              }
              if (p.quarter)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[y][i] = __float_as_uint(4.f * __uint_as_float(s[y][i]));
              part = prompt_chunk<true>(s[y], c2, L + 4 * (c + y), first - 16 * (c + y), cols - 16 * (c + y), part);
            }
          tmem_wait_ld();  // the load ahead of the last columns
        }
        w += part.x + part.y;
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[st * MT + m]);
        qt += C::TURNS;
        while (qt >= n_qt) qt -= tiles_head;  // on to the next head
      }
      if (!ok) break;
      const int last_turn = tiles > 0 ? (nq + tiles - 1) % C::TURNS : 0;
      // Between any two turns the sums go in order, through two slots and two monotonic counters of their own.
      auto channel = [&](int from, int to) { return (from * C::TURNS + to) * (4 * MT) + kw; };
      if (turn != last_turn) {
        if (skip < tiles) {
          uint32_t n = 0;
#pragma unroll
          for (int t = 0; t < C::TURNS; ++t)
            if (t == last_turn) n = n_sent[t]++;
          const int ch = channel(turn, last_turn);
          // the slot's last sum has been collected
          ok = __all_sync(0xffffffffu, count_wait_bounded(&collected[ch], n < 2 ? 0 : n - 1, abort_flag, &timed_out));
          if (!ok) break;
          sums[((n & 1) * (C::TURNS * C::TURNS * 4 * MT) + ch) * 32 + lane] = w;
          __syncwarp();
          if (lane == 0) red_release_add(&sent[ch], 1);
        }
      } else {
#pragma unroll
        for (int t = 0; t < C::TURNS; ++t) {
          if (t == last_turn || (t - nq % C::TURNS + C::TURNS) % C::TURNS >= tiles) continue;  // no sum from there
          const uint32_t n = n_got[t]++;
          const int ch = channel(t, turn);
          ok = ok && __all_sync(0xffffffffu, count_wait_bounded(&sent[ch], n + 1, abort_flag, &timed_out));
          if (!ok) break;
          w += sums[((n & 1) * (C::TURNS * C::TURNS * 4 * MT) + ch) * 32 + lane];
          __syncwarp();
          if (lane == 0) red_release_add(&collected[ch], 1);
        }
      }
      nq += tiles;
      if (!ok || turn != last_turn) continue;
      if (key < p.n_kv) p.acc_out[at] = (p.acc ? p.acc[at] : 0.f) + w;
    }
  }

  if (timed_out) record_error(6 /* SDPA_ERR_DEVICE_TIMEOUT */);
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace sdpa
