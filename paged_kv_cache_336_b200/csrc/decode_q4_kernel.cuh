// Decode attention over the 4-bit cache for sm_100a (templates; instantiated in
// decode_q4_inst.cu).
//
// What is computed is pa_decode_split's result, windows and sinks included,
// on the values mn + s * code that the 4-bit pools stand for. With i the
// 64-dim group of a dim, Q_i = sum over the group of q and c the codes:
//   logit_t = scale * sum_i (s_ti * sum_d q_d c_td + mn_ti * Q_i)
//   out_d   = sum_t p_t s_ti (c_td - 8) + sum_t p_t (mn_ti + 8 s_ti),
// so both products run on the codes themselves, exact small integers, and
// scales and minima enter once per (token, group). The codes of V are taken
// relative to 8, so that what is summed over a long context stays near zero.
//
// How.
// * Work is cut as in paged_decode_sinks_kernel: one list of 16-token units per
//   KV head (per 8 query heads of it where a group has more), every consumer
//   warp of a persistent grid an equal run of its list, pieces merged by
//   lse_merge_kernel. A unit is one sub-tile of K and of V, 9 head_dim bytes
//   each and contiguous: one bulk copy each.
// * Four producer warps keep the consumers' rings full (eight lanes per
//   consumer, one unit each), because a warp that fills its own ring spends
//   74 of its 330 instructions a unit on that; registers are split by
//   setmaxnreg, 160 a consumer thread and 32 a producer one with 12 consumers.
// * mma.sync with the 16 tokens of a unit as the rows and 8 query heads as the
//   columns, both times: S = K Q^T, O^T = V^T P^T. A group of 8 heads then wastes
//   no row (with heads as rows half would be padding). Fragments come straight
//   from the code words: which dims (or tokens) stand at which k index is free
//   as long as both operands agree, so the words are stored in the order the
//   lanes want them, and no ldmatrix or shuffle is needed. Row r of S is token
//   r / 2 (r even) or 7 - r / 2 (odd), + 8 for r >= 8: the rows that lanes read
//   together then lie in different banks.
// * S: codes as bytes (a mask of the word and of the word >> 4) against q as
//   rint(2^k q), 16 bits in two bytes, k bringing the head's largest |q| into
//   [2^14, 2^15): u8 x s8 and u8 x u8 products of depth 32 with exact 32-bit
//   sums. Against bf16 operands (128 + c by a mask-or) that is 3 integer
//   instructions for 8 codes instead of 7. e4m3 products, whose bytes 0..15 are
//   c / 512 exactly, measured slower: without native hardware behind mma.sync
//   they cost conversions and two f16 products each.
// * O: codes less 8 as f16 (CodeBits) against p s in f16, transposed between
//   its two layouts by movmatrix. f16 needs the weights' range bounded: see
//   Q4Warp::up. In exchange O accumulates in place, where a mask-or'ed bf16
//   code (128 + c) would leave a cancellation of 128 to a few.
// * A step (64 tokens at head_dim 128, 128 at 64, 48 at 256) shares one running
//   maximum; the accumulators are rescaled only when it (or a group's up) moves.
//   Steps that are not whole go unit by unit through the masked build.
// Rounding: q to 16 bits of its head's range (at most 2^-15 of the largest),
// p s to f16 (2^-11), the output to bf16; sums, logits, minima in fp32 or exact.
// Bound: 8 x 131072 tokens (64 heads over 8, head_dim 128) take 249 us in a burst,
// 1.21 GB at 4.85 TB/s, 0.74 of the measured copy rate, and 278 us once the GPU has
// reached its 1000 W limit (1.86 GHz), after some 100 ms of such calls. 332 warp
// instructions a unit, producers included; integer pipe 53% busy, issue slots 61%.
// (With one power of two for all groups, which overflowed or lost bits, 325
// instructions and 246 us; copies alone then took 203 us and the math alone 214.)
#pragma once

#include <climits>

#include "decode_sinks_kernel.cuh"
#include "q4_common.cuh"

namespace pagedkv {

// W consumer warps and four producer warps; a step takes up to US units (a
// producer has eight lanes per consumer); each consumer's ring has NS slots of US
// sub-tiles, filled in the order K, V, K, V, ... of its steps.
template <int BS_, int D_, int W_, int US_, int NS_>
struct Q4Cfg {
  static constexpr int BS = BS_, D = D_, W = W_, US = US_, NS = NS_;
  static constexpr int UPB = BS / 16;
  using Geo = Q4Geo<D>;
  static constexpr int kThreads = 32 * (W + 4);
  static constexpr int kSlotBytes = US * Geo::kSubBytes;
  static constexpr int kRingBytes = W * NS * kSlotBytes;
  // ring | full, empty barriers [W][NS] | units present per slot [W][NS]
  static constexpr int kFixedSmem = 128 + kRingBytes + W * NS * (8 + 8 + 4);
  // Registers a thread at launch, and after the split (what the producers
  // give up is what the consumers take).
  static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
  static constexpr int kProducerRegs = W == 12 ? 32 : 40;
  static constexpr int kConsumerRegs = (kLaunchRegs * (W + 4) - kProducerRegs * 4) / W / 8 * 8;
  static_assert(W % 4 == 0 && W <= 12 && US <= 8 && NS >= 2 && NS <= 8, "whole warpgroups; ring layout");
  static_assert(kConsumerRegs * W + kProducerRegs * 4 <= kLaunchRegs * (W + 4), "registers of the split");
  static_assert(kRingBytes % 16 == 0 && kFixedSmem + (2 * 4096 + 1) * 4 <= 226 * 1024, "shared memory budget exceeded");
};

// Bulk copy global -> shared, completion on `bar`; addresses and size are
// multiples of 16 bytes at every call site.
__device__ __forceinline__ void bulk_load(void* smem_dst, const void* src, uint32_t bytes, uint64_t* bar,
                                          uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_addr(smem_dst)),
      "l"(src), "r"(bytes), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

// D += A(16x16) * B(16x8), f16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 8x8 transpose of 16-bit elements across the warp (mma fragment layout).
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// D = A * B (first) or D += A * B for bytes, A (16 x 32) unsigned, B (32 x 8)
// signed or unsigned, 32-bit sums.
#define PA_MMA_BYTES(types)                                                                          \
  if (first)                                                                                         \
    asm volatile("mma.sync.aligned.m16n8k32.row.col." types                                          \
                 " {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"              \
                 : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])                                    \
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "r"(0));            \
  else                                                                                               \
    asm volatile("mma.sync.aligned.m16n8k32.row.col." types                                          \
                 " {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"                  \
                 : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])                                    \
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1))
template <bool kSigned>
__device__ __forceinline__ void mma_bytes(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool first) {
  if constexpr (kSigned) {
    PA_MMA_BYTES("s32.u8.s8.s32");
  } else {
    PA_MMA_BYTES("s32.u8.u8.s32");
  }
}
#undef PA_MMA_BYTES

// Greater of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The codes of a word less 8, as f16: out[j] holds those of dims j (low half) and
// j + 4. A mask-or puts a code into the mantissa of 1024, from where it stands
// (1024 + c, or 1024 + 16 c for the second nibble of a byte), and one packed
// add or multiply-add makes c - 8 of it, exactly: 5 integer and 4 packed
// instructions for 8 codes, on different pipes (the conversion of Y. J. Kim et al.,
// "Who Says Elephants Can't Run: Bringing Large Scale MoE Models into Cloud Scale
// Production", 2022). The mask-or's constants come from registers (an instruction
// takes one immediate at most).
struct CodeBits {
  uint32_t lo4, hi4, k1024;
  __device__ __forceinline__ CodeBits() {
    asm volatile("mov.b32 %0, 0x000f000f;" : "=r"(lo4));
    asm volatile("mov.b32 %0, 0x00f000f0;" : "=r"(hi4));
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(k1024));
  }
  __device__ __forceinline__ void unpack(uint32_t w, uint32_t (&out)[4]) const {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t x, y;
      asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(x) : "r"(w >> (8 * b)), "r"(lo4), "r"(k1024));  // (a & b) | c
      asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(y) : "r"(w >> (8 * b)), "r"(hi4), "r"(k1024));
      asm("add.rn.f16x2 %0, %1, %2;" : "=r"(out[2 * b]) : "r"(x), "r"(0xe408e408u));                   // - 1032
      asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(out[2 * b + 1]) : "r"(y), "r"(0x2c002c00u), "r"(0xd480d480u));  // / 16 - 72
    }
  }
};

// N consecutive 32-bit words at a shared-memory address, N * 4 bytes aligned.
template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
    static_assert(N == 1, "1, 2 or 4 words");
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  }
}

// One warp's running state for 8 query heads; lane = 4 g + t holds heads 2t
// and 2t + 1 of S and O, head g of the query operand.
template <class Cfg>
struct Q4Warp {
  using Geo = typename Cfg::Geo;
  static constexpr int D = Cfg::D;
  static constexpr int US = Cfg::US;
  static constexpr int GR = Geo::kGroups;

  // Query operand: rint(2^k q), 16 bits, as high bytes (signed) and low bytes
  // (unsigned) per octet of 8 dims that the lane holds (even dims, odd dims).
  uint32_t qb[GR][2][2][2];
  float qs[GR][2];        // 2^k Q_i of heads 2t, 2t + 1
  float f[2];             // |scale| log2(e) 2^-k of heads 2t, 2t + 1
  float o[GR][4][4];      // up[i] times O^T: dims 64 i + 8 g + 2 j (+ 1 for e >= 2), head 2t + (e & 1)
  float mid[GR][2];       // sum p (mn + 8 s) over this lane's tokens
  // Softmax weights are p = 2^(y - m), m the running maximum of the logits y (log2
  // domain). A weight times a value scale enters O's products as f16, so group i's
  // scales are taken times up[i] = 2^(14 - e), with 2^e the largest power of two
  // among those met: products below 2^15, 11 bits down to 2^-28 of the largest
  // weight times the group's largest scale and 2^-39 of that apart below.
  // A power for each group, and none in mid, because groups may differ by any
  // factor, and minima by any factor from scales.
  float m[2], l[2];       // l: this lane's part of the sum
  float up[GR];
  // This lane's places in a sub-tile. K: its row (rows g and g + 8 of S are
  // tokens tok and tok + 8); V: tokens t and 7 - t (+ 8); both: parameters.
  CodeBits bits;
  int tok;
  uint32_t k_at, v_at[2], par_at;

  __device__ __forceinline__ void places(int lane) {
    const int g = lane >> 2, t = lane & 3;
    tok = (g & 1) ? 7 - (g >> 1) : (g >> 1);
    k_at = tok * Geo::kRowBytes + (D == 256 ? (tok & 1) * 64 + t * 16 : t * (8 * GR));
    par_at = Geo::kCodeBytes + tok * Geo::kParamRow;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int tk = r ? 7 - t : t;
      v_at[r] = tk * Geo::kRowBytes + ((g ^ Geo::v_turn(tk)) * (D / 16));
    }
  }

  __device__ __forceinline__ void begin(const __nv_bfloat16* row, bool valid, float scale_log2, int lane) {
    const int t = lane & 3;
    uint4 x[GR][2];
    float largest = 0.f;
#pragma unroll
    for (int i = 0; i < GR; ++i) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        x[i][w] = make_uint4(0u, 0u, 0u, 0u);
        if (valid) x[i][w] = *reinterpret_cast<const uint4*>(row + 64 * i + 16 * t + 8 * w);
        const uint32_t v[4] = {x[i][w].x, x[i][w].y, x[i][w].z, x[i][w].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) largest = max_nan(largest, max_nan(fabsf(bf16_lo(v[j])), fabsf(bf16_hi(v[j]))));
      }
    }
    largest = max_nan(largest, __shfl_xor_sync(0xffffffffu, largest, 1));
    largest = max_nan(largest, __shfl_xor_sync(0xffffffffu, largest, 2));
    // k brings the row's largest |q| into [2^14, 2^15); q of a negative scale is negated
    const int e = max(static_cast<int>(__float_as_uint(largest) >> 23), 16);
    const float pow_k = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);  // 2^k, k = 141 - e
    const float down = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);  // 2^-k
    float fac = fabsf(scale_log2) * down;
    if (!(largest < INFINITY)) fac = __uint_as_float(0x7fc00000u);
    const float sgn = scale_log2 < 0.f ? -pow_k : pow_k;
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint32_t v[4] = {x[i][w].x, x[i][w].y, x[i][w].z, x[i][w].w};
#pragma unroll
        for (int odd = 0; odd < 2; ++odd) {
          uint32_t hi = 0, lo = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float q = (odd ? bf16_hi(v[j]) : bf16_lo(v[j])) * sgn;
            sum += q;
            const uint32_t n = static_cast<uint32_t>(__float2int_rn(q));
            hi |= ((n >> 8) & 0xffu) << (8 * j);
            lo |= (n & 0xffu) << (8 * j);
          }
          qb[i][w][0][odd] = hi;
          qb[i][w][1][odd] = lo;
        }
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      qs[i][0] = __shfl_sync(0xffffffffu, sum, 8 * t);
      qs[i][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4);
      mid[i][0] = mid[i][1] = 0.f;
      up[i] = 0x1p126f;  // (a scale of 2^-111 or more asks for less)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
    }
    f[0] = __shfl_sync(0xffffffffu, fac, 8 * t);
    f[1] = __shfl_sync(0xffffffffu, fac, 8 * t + 4);
    m[0] = m[1] = kNoTokens;
    l[0] = l[1] = 0.f;
  }

  // A step is logits() and then attend(), over NU units whose sub-tiles lie one
  // after the other at shared addresses k_tile and v_tile. kEdge (NU = 1): of
  // the unit's rows tok and tok + 8 those with out[] set are not visible and
  // may hold anything, NaN parameters included.
  template <int NU, bool kEdge>
  __device__ __forceinline__ void logits(uint32_t k_tile, float (&x)[NU][4], const bool (&out)[2]) const {
    static_assert(!kEdge || NU == 1, "an edge step takes one unit");
    const uint32_t k_row = k_tile + k_at, k_par = k_tile + par_at;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      uint32_t w[2][2 * GR], par[2][GR];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t at = k_row + u * Geo::kSubBytes + 8 * r * Geo::kRowBytes;
        if constexpr (D == 256) {  // two halves of 64 bytes, swapped in odd rows
          uint32_t p0[4], p1[4];
          lds_words(at, p0);
          lds_words(at ^ 64u, p1);
#pragma unroll
          for (int c = 0; c < 4; ++c) w[r][c] = p0[c], w[r][4 + c] = p1[c];
        } else {
          lds_words(at, w[r]);
        }
        lds_words(k_par + u * Geo::kSubBytes + 8 * r * Geo::kParamRow, par[r]);
      }
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        int sh[4], sl[4];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t wa = w[0][2 * i + c], wb = w[1][2 * i + c];
          constexpr uint32_t kNib = 0x0f0f0f0fu;
          const uint32_t a[4] = {wa & kNib, wb & kNib, (wa >> 4) & kNib, (wb >> 4) & kNib};
          mma_bytes<true>(sh, a, qb[i][c][0][0], qb[i][c][0][1], c == 0);
          mma_bytes<false>(sl, a, qb[i][c][1][0], qb[i][c][1][1], c == 0);
        }
        float s[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = __int2float_rn(256 * sh[e] + sl[e]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float sc = bf16_lo(par[r][i]), mn = bf16_hi(par[r][i]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float base = i == 0 ? mn * qs[i][h] : fmaf(mn, qs[i][h], x[u][2 * r + h]);
            x[u][2 * r + h] = fmaf(s[2 * r + h], sc, base);
          }
        }
      }
      if (kEdge) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[u][e] = out[e >> 1] ? -INFINITY : x[u][e] * f[e & 1];
      }
    }
  }

  template <int NU, bool kEdge>
  __device__ __forceinline__ void attend(uint32_t v_tile, float (&x)[NU][4], const bool (&out)[2]) {
    const uint32_t v_par = v_tile + par_at;
    // ---- a value scale that up[] would take to 2^15 or more asks for less. (A NaN
    // hides the group's other scales: its values are NaN anyway.) ---------------------
    uint32_t smax[GR] = {};
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t par[GR];
        lds_words(v_par + u * Geo::kSubBytes + 8 * r * Geo::kParamRow, par);
#pragma unroll
        for (int i = 0; i < GR; ++i) smax[i] = __vmaxu2(smax[i], out[r] ? 0u : par[i]);
      }
    bool large = false;
#pragma unroll
    for (int i = 0; i < GR; ++i) large |= bf16_lo(smax[i]) * up[i] >= 0x1p15f;
    if (__any_sync(0xffffffffu, large)) lower_up<NU>(v_par, out);
    // ---- running softmax over the step's tokens ------------------------------------
    float ref[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = fmaxf(x[0][h], x[0][2 + h]);
#pragma unroll
      for (int u = 1; u < NU; ++u) mx = fmaxf(mx, fmaxf(x[u][h], x[u][2 + h]));
#pragma unroll
      for (int off = 4; off <= 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      ref[h] = fmaxf(m[h], kEdge ? mx : mx * f[h]);
    }
    if (__any_sync(0xffffffffu, ref[0] != m[0] || ref[1] != m[1])) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float alpha = fast_exp2(m[h] - ref[h]);
        m[h] = ref[h];
        l[h] *= alpha;
#pragma unroll
        for (int i = 0; i < GR; ++i) {
          mid[i][h] *= alpha;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[i][j][h] *= alpha;
            o[i][j][2 + h] *= alpha;
          }
        }
      }
    }
    uint32_t pb[NU][GR][2];  // P^T s, f16
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[e] = fast_exp2(kEdge ? x[u][e] - m[e & 1] : fmaf(x[u][e], f[e & 1], -m[e & 1]));
        l[e & 1] += p[e];
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t par[GR];
        lds_words(v_par + u * Geo::kSubBytes + 8 * r * Geo::kParamRow, par);
#pragma unroll
        for (int i = 0; i < GR; ++i) {
          if (out[r]) par[i] = 0u;
          const float sc = bf16_lo(par[i]);
          const float mi = fmaf(8.f, sc, bf16_hi(par[i])), su = sc * up[i];
          pb[u][i][r] = movmatrix(pack_f16x2(p[2 * r] * su, p[2 * r + 1] * su));
          mid[i][0] = fmaf(p[2 * r], mi, mid[i][0]);
          mid[i][1] = fmaf(p[2 * r + 1], mi, mid[i][1]);
        }
      }
    }
    // ---- O^T += V^T P^T --------------------------------------------------------------
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      uint32_t w[4][GR];  // tokens t, 7 - t, 8 + t, 15 - t: k indices 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
      for (int r = 0; r < 4; ++r)
        lds_words(v_tile + v_at[r & 1] + u * Geo::kSubBytes + (r >> 1) * 8 * Geo::kRowBytes, w[r]);
#pragma unroll
      for (int i = 0; i < GR; ++i) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // dims 8 g + 4 half + 0 .. 3
          const uint32_t sel = half ? 0x7632u : 0x5410u;
          uint32_t ca[4], cb[4];
          bits.unpack(__byte_perm(w[0][i], w[1][i], sel), ca);
          bits.unpack(__byte_perm(w[2][i], w[3][i], sel), cb);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t a[4] = {ca[2 * j], ca[2 * j + 1], cb[2 * j], cb[2 * j + 1]};
            mma_f16_16816(o[i][2 * half + j], a, pb[u][i][0], pb[u][i][1]);
          }
        }
      }
    }
  }

  // up[i] falls to 2^(14 - e), with e the largest exponent of the step's finite
  // scales of group i, and the group's sums with it.
  template <int NU>
  __device__ __forceinline__ void lower_up(uint32_t v_par, const bool (&out)[2]) {
    uint32_t big[GR] = {};  // biased exponents
#pragma unroll 1
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t par[GR];
        lds_words(v_par + u * Geo::kSubBytes + 8 * r * Geo::kParamRow, par);
#pragma unroll
        for (int i = 0; i < GR; ++i) {
          const uint32_t e = (par[i] >> 7) & 0xffu;
          if (!out[r] && e < 255u) big[i] = max(big[i], e);
        }
      }
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      const int old = static_cast<int>(__float_as_uint(up[i]) >> 23);  // 14 .. 253
      const int now = min(old, 268 - static_cast<int>(max(__reduce_max_sync(0xffffffffu, big[i]), 15u)));
      up[i] = __uint_as_float(static_cast<uint32_t>(now) << 23);
      const float by = __uint_as_float(static_cast<uint32_t>(max(127 + now - old, 0)) << 23);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][j][e] *= by;
    }
  }

  // Completes the sums over lanes and takes up[] back; then head 2t + h's dims
  // 64 i + 8 g + 0..7 are value(i, h, 0..7).
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      const float down = __uint_as_float((254u << 23) - __float_as_uint(up[i]));  // 1 / up[i]
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][j][e] *= down;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int off = 4; off <= 16; off <<= 1) {
        l[h] += __shfl_xor_sync(0xffffffffu, l[h], off);
#pragma unroll
        for (int i = 0; i < GR; ++i) mid[i][h] += __shfl_xor_sync(0xffffffffu, mid[i][h], off);
      }
    }
  }
  __device__ __forceinline__ float value(int i, int h, int d) const { return o[i][d >> 1][2 * (d & 1) + h] + mid[i][h]; }

  __device__ __forceinline__ void store_final(__nv_bfloat16* out, int h, int g) const {
    const float inv = l[h] > 0.f ? 1.f / l[h] : 0.f;
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int d = 0; d < 4; ++d) w[d] = pack_bf16x2(value(i, h, 2 * d) * inv, value(i, h, 2 * d + 1) * inv);
      *reinterpret_cast<uint4*>(out + 64 * i + 8 * g) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ void store_partial(const DecodeArgs& a, int64_t pr, int h, int g) const {
    if (g == 0) {
      a.part_m[pr] = m[h];
      a.part_l[pr] = l[h];
    }
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      float4* dst = reinterpret_cast<float4*>(a.part_acc + pr * D + 64 * i + 8 * g);
      dst[0] = make_float4(value(i, h, 0), value(i, h, 1), value(i, h, 2), value(i, h, 3));
      dst[1] = make_float4(value(i, h, 4), value(i, h, 5), value(i, h, 6), value(i, h, 7));
    }
  }
};

// What a sequence costs a warp besides its units (query rows, the result, the
// steps at its ends), in units. Measured on 256 sequences of 16 to 8192 tokens:
// 105 us for 0, 97.3 for 2, 95.1 for 4, 98.7 for 8.
constexpr int kQ4Pad = 4;

// What a warp has to do: units [g0, g1) of list (h, qt); with seq_cut, as piece
// `piece` of sequence `seq` (num_seqs and up: nothing).
struct Q4Run {
  int g0, g1, gi, h, qt, C, seq, piece;
};

template <class Cfg>
__device__ __forceinline__ Q4Run q4_run(const SinksArgs& a, const UnitLists& lists, const int* prefix, int q_tiles,
                                        int warp) {
  const int num_lists = a.num_kv_heads * q_tiles;
  Q4Run r{};
  if (a.seq_cut > 0) {  // each sequence by itself
    const int item = static_cast<int>(blockIdx.x) * (Cfg::W / a.seq_cut) + warp / a.seq_cut, list = item % num_lists;
    r.h = list / q_tiles;
    r.qt = list % q_tiles;
    r.seq = item / num_lists;
    r.piece = warp % a.seq_cut;
    if (r.seq >= a.num_seqs) return r;
    const int end = prefix[r.seq + 1] - kQ4Pad;
    r.C = (end - prefix[r.seq] + a.seq_cut - 1) / a.seq_cut;
    r.g0 = min(prefix[r.seq] + r.piece * r.C, end);
    r.g1 = min(r.g0 + r.C, end);
    return r;
  }
  const int wg = static_cast<int>(blockIdx.x) * Cfg::W + warp;
  const int groups = static_cast<int>(gridDim.x) * Cfg::W / num_lists;
  r.h = (wg % num_lists) / q_tiles;  // KV head
  r.qt = wg % q_tiles;               // run of its query heads
  r.gi = wg / num_lists;
  r.C = max((lists.total + groups - 1) / groups, (lists.longest + a.max_pieces - 2) / (a.max_pieces - 1));
  const int64_t total = lists.total, begin = static_cast<int64_t>(r.gi) * r.C;
  r.g0 = static_cast<int>(min(begin, total));
  r.g1 = r.gi < groups ? static_cast<int>(min(begin + r.C, total)) : r.g0;
  return r;
}

__device__ __forceinline__ int q4_locate(const int* prefix, int num_seqs, int g) {  // last s with prefix[s] <= g
  int lo = 0, hi = num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= g) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Producer warp `which` of four fills the rings of consumers which, which + 4,
// ...: eight lanes each, lane u of them its unit u. Block ids are read a step
// ahead.
template <class Cfg>
__device__ __forceinline__ void q4_produce(const uint8_t* k_pool, const uint8_t* v_pool, const SinksArgs& a, int q_tiles,
                                           const UnitLists& lists, const int* prefix, const int* first_unit,
                                           uint8_t* ring, uint64_t* full, uint64_t* empty, uint32_t* present,
                                           int which) {
  using Geo = typename Cfg::Geo;
  constexpr int US = Cfg::US, NS = Cfg::NS, UPB = Cfg::UPB;
  const int lane = threadIdx.x & 31, u = lane & 7;
  const int c = which + 4 * (lane >> 3);
  Q4Run run = q4_run<Cfg>(a, lists, prefix, q_tiles, min(c, Cfg::W - 1));
  if (c >= Cfg::W) run.g1 = run.g0;
  const int g1 = run.g1, h = run.h;
  ring += (min(c, Cfg::W - 1) * NS) * Cfg::kSlotBytes + u * Geo::kSubBytes;
  full += min(c, Cfg::W - 1) * NS;
  empty += min(c, Cfg::W - 1) * NS;
  present += min(c, Cfg::W - 1) * NS;
  const uint64_t policy = l2_policy(a.l2_hint);

  // The next step: units [g - n, g) of sequence s, this lane's table entry.
  int g = run.g0, s = 0, end = 0, n = 0, id = -1, half = 0;
  auto look_up = [&]() {
    n = 0;
    id = -1;
    if (g >= g1) return;
    if (g >= end) {  // (the first time, and at a sequence's end)
      if (end == 0) {
        s = q4_locate(prefix, a.num_seqs, g);
        if (g >= prefix[s + 1] - kQ4Pad) g = prefix[++s];
      } else {
        g = prefix[++s];
      }
      if (g >= g1) return;
      end = min(prefix[s + 1] - kQ4Pad, g1);
    }
    n = min(US, end - g);
    const int fu = first_unit[s];
    if (u < n && fu >= 0) {
      const int un = g - prefix[s] + u, ns = sink_units(a, fu);
      const int v = un < ns ? un : (fu & ~kSinkFlag) + un - ns;
      id = a.block_tables[static_cast<int64_t>(s) * a.max_blocks_per_seq + v / UPB];
      if (id < 0) id = INT_MAX;  // no block; -1 means nothing to read
      half = v % UPB;
    }
    g += n;
  };
  int64_t src = -1;  // byte offset of this lane's tile in the step being filled, -1: none
  auto settle = [&]() {
    src = -1;
    if (id >= 0) {
      if (id < a.num_blocks)
        src = static_cast<int64_t>((id * a.num_kv_heads + h) * UPB + half) * Geo::kSubBytes;
      else
        report(a.dev_err, PA_DEVERR_BLOCK_ID);
    }
  };
  look_up();
  bool active = n != 0, value = false;
  if (active) {
    settle();
    look_up();
  }
  int slot = 0;
  uint32_t parity = 1, polls = 0, filled = 0;  // a fresh barrier's phase of parity 1 counts as complete
  uint64_t t0 = 0;
  while (__any_sync(0xffffffffu, active)) {
    const bool free_slot = active && mbar_try_wait(&empty[slot], parity);
    const bool go = __shfl_sync(0xffffffffu, free_slot, lane & 24);
    const uint32_t got = (__ballot_sync(0xffffffffu, src >= 0) >> (lane & 24)) & 0xffu;
    if (go && u == 0) {
      if (!value) present[slot] = got;
      if (got) mbar_arrive_expect_tx(&full[slot], Geo::kSubBytes * __popc(got));
      else mbar_arrive(&full[slot]);  // completes the phase with no data
    }
    __syncwarp();
    if (go) {
      if (src >= 0) {
        fence_proxy_async_smem();
        bulk_load(ring + slot * Cfg::kSlotBytes, (value ? v_pool : k_pool) + src, Geo::kSubBytes, &full[slot], policy);
      }
      ++filled;
      if (++slot == NS) {
        slot = 0;
        parity ^= 1u;
      }
      value = !value;
      if (!value) {  // both halves asked for: on to the next step
        active = n != 0;
        settle();
        look_up();
      }
    }
    if (__any_sync(0xffffffffu, go)) {
      polls = 0;
      t0 = 0;
    } else if ((++polls & 1023u) == 0u) {  // consumers that do not come: give up after the limit
      const uint64_t now = __shfl_sync(0xffffffffu, global_timer_ns(), 0);  // one answer for the warp
      if (t0 == 0) t0 = now;
      else if (now - t0 > kWaitLimitNs || polls >= kWaitMaxPolls) {
        if (lane == 0) report(a.dev_err, PA_DEVERR_TIMEOUT);
        break;
      }
    }
  }
  // No copy is in flight when the last warp leaves.
  for (uint32_t i = 0; i < NS && i < filled; ++i) {
    if (slot-- == 0) {
      slot = NS - 1;
      parity ^= 1u;
    }
    mbar_wait_bounded(&full[slot], parity ^ 1u, a.dev_err);
  }
}

// Walks a consumer's run; with seq_cut above 1 it leaves the run's state in `st`.
template <class Cfg>
__device__ __forceinline__ void q4_walk(const SinksArgs& a, const Q4Run& run, Q4Warp<Cfg>& st, const int* prefix,
                                        const int* first_unit, const uint8_t* ring, uint64_t* full, uint64_t* empty,
                                        const uint32_t* present) {
  using Geo = typename Cfg::Geo;
  constexpr int US = Cfg::US, NS = Cfg::NS, D = Cfg::D;
  constexpr uint32_t kUnitMask = (1u << US) - 1u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g0 = run.g0, g1 = run.g1, h = run.h, C = run.C;
  if (g0 >= g1) return;
  const uint32_t my_ring = smem_addr(ring) + warp * NS * Cfg::kSlotBytes;
  full += warp * NS;
  empty += warp * NS;
  present += warp * NS;

  const int g = lane >> 2, t = lane & 3;
  const int heads = min(8, a.group - 8 * run.qt);
  const int head0 = h * a.group + 8 * run.qt;
  int s = q4_locate(prefix, a.num_seqs, g0), cg = g0;
  if (cg >= prefix[s + 1] - kQ4Pad) cg = prefix[++s];
  if (cg >= g1) return;
  int seg0 = prefix[s], seg1 = prefix[s + 1] - kQ4Pad;  // the sequence's units in the list
  int ctx = 0, ftok = 0, ub = 0, ns = 0;
  int full0 = 0, full1 = 0;                      // units of the list whose 16 tokens are all visible
  auto begin_segment = [&]() {
    ctx = clamp_ctx(a.context_lens[s], a.max_blocks_per_seq * Cfg::BS);
    ftok = first_token(a, ctx);
    ub = first_unit[s];
    ns = ub < 0 ? 0 : sink_units(a, ub);
    if (ub >= 0) ub &= ~kSinkFlag;
    if (!sinks_apart(a, ftok)) ftok = 0;
    full0 = seg0 + ns + (ftok + 15) / 16 - ub;
    full1 = ub < 0 ? 0 : seg0 + ns + ctx / 16 - ub;
    const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(a.q) +
                               (static_cast<int64_t>(s) * a.num_q_heads + head0 + g) * D;
    if (seg1 + kQ4Pad < g1 && t == 0 && g < heads) {      // the next sequence's query rows: into L2 now
      const char* nq = reinterpret_cast<const char*>(row + static_cast<int64_t>(a.num_q_heads) * D);
      for (int b = 0; b < D * 2; b += 128) prefetch_l2(nq + b);
    }
    st.begin(row, g < heads, a.scale_log2, lane);
    if (a.seq_cut == 0 && seg0 >= g0 && run.qt == 0 && lane == 0)  // the first piece's warp records how many there are
      a.seg_pieces[static_cast<int64_t>(s) * a.num_kv_heads + h] = (seg1 - 1) / C - seg0 / C + 1;
  };
  auto end_segment = [&]() {
    st.finish();
    const bool whole = seg0 >= g0 && seg1 <= g1;
    const int64_t row0 = static_cast<int64_t>(s) * a.num_q_heads + head0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (2 * t + e >= heads) continue;
      const int64_t row = row0 + 2 * t + e;
      if (whole) st.store_final(static_cast<__nv_bfloat16*>(a.out) + row * D, e, g);
      else st.store_partial(a, row * a.max_partitions + run.gi - seg0 / C, e, g);
    }
  };

  int slot = 0;
  uint32_t parity = 0;
  // Waits for the ring's next slot; false after a timeout.
  auto take = [&]() {
    const bool okw = mbar_wait_bounded(&full[slot], parity, a.dev_err);
    return __all_sync(0xffffffffu, okw) != 0;
  };
  auto give = [&]() {  // the slot's reads are done: it may be filled again
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[slot]);
    if (++slot == NS) {
      slot = 0;
      parity ^= 1u;
    }
  };
  begin_segment();
  for (;;) {
    if (cg == min(seg1, g1)) {
      if (a.seq_cut > 1) return;
      end_segment();
      cg = prefix[++s];
      if (cg >= g1) return;
      seg0 = cg;
      seg1 = prefix[s + 1] - kQ4Pad;
      begin_segment();
    }
    const int n = min(US, min(seg1, g1) - cg);
    if (!take()) return;
    const uint32_t got = present[slot];
    const uint32_t kt = my_ring + slot * Cfg::kSlotBytes;
    if (got == kUnitMask && cg >= full0 && cg + US <= full1) {
      const bool all[2] = {false, false};
      float x[US][4];
      st.template logits<US, false>(kt, x, all);
      give();
      if (!take()) return;
      st.template attend<US, false>(my_ring + slot * Cfg::kSlotBytes, x, all);
      give();
    } else {                                     // unit by unit; K's slot is held until V is done with
      const int vslot = slot + 1 == NS ? 0 : slot + 1;
      const bool okw = mbar_wait_bounded(&full[vslot], vslot == 0 ? parity ^ 1u : parity, a.dev_err);
      if (!__all_sync(0xffffffffu, okw)) return;
      const uint32_t vt = my_ring + vslot * Cfg::kSlotBytes;
      const int un = cg - seg0;                  // index in the sequence's units
#pragma unroll 1
      for (int u = 0; u < n; ++u) {
        if (!(got >> u & 1)) continue;
        const bool sink = un + u < ns;
        const int u0 = (sink ? un + u : ub + un + u - ns) * 16;  // first token
        const int lo = sink ? 0 : ftok - u0, hi = (sink ? a.num_sinks : ctx) - u0;
        const bool out[2] = {st.tok < lo || st.tok >= hi, st.tok + 8 < lo || st.tok + 8 >= hi};
        float x[1][4];
        st.template logits<1, true>(kt + u * Geo::kSubBytes, x, out);
        st.template attend<1, true>(vt + u * Geo::kSubBytes, x, out);
      }
      give();
      give();
    }
    cg += n;
  }
}

template <class Cfg>
__device__ __forceinline__ void q4_consume(const SinksArgs& a, int q_tiles, const UnitLists& lists, const int* prefix,
                                           const int* first_unit, uint8_t* ring, uint64_t* full, uint64_t* empty,
                                           const uint32_t* present) {
  constexpr int D = Cfg::D, W = Cfg::W;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Q4Run run = q4_run<Cfg>(a, lists, prefix, q_tiles, warp);
  Q4Warp<Cfg> st;
  st.places(lane);
  st.m[0] = st.m[1] = kNoTokens;
  q4_walk<Cfg>(a, run, st, prefix, first_unit, ring, full, empty, present);
  if (a.seq_cut <= 1) return;
  // ---- pieces of one sequence, merged in shared memory: every consumer comes
  // here, with or without units. A warp's state takes the place of its ring,
  // whose last copies it has used. ------------------------------------------------
  constexpr int kState = 8 * (D + 2);  // values [8 heads][D], m [8], l [8]
  static_assert(kState * 4 <= Cfg::NS * Cfg::kSlotBytes, "a warp's state fits its ring");
  auto state = [&](int w) { return reinterpret_cast<float*>(ring + w * Cfg::NS * Cfg::kSlotBytes); };
  const int g = lane >> 2, t = lane & 3;
  float* mine = state(warp);
  const bool some = run.g0 < run.g1;
  if (some) st.finish();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (some) {
#pragma unroll
      for (int i = 0; i < Cfg::Geo::kGroups; ++i) {
        float4* dst = reinterpret_cast<float4*>(mine + (2 * t + e) * D + 64 * i + 8 * g);
        dst[0] = make_float4(st.value(i, e, 0), st.value(i, e, 1), st.value(i, e, 2), st.value(i, e, 3));
        dst[1] = make_float4(st.value(i, e, 4), st.value(i, e, 5), st.value(i, e, 6), st.value(i, e, 7));
      }
    }
    if (g == 0) {
      mine[8 * D + 2 * t + e] = st.m[e];
      mine[8 * D + 8 + 2 * t + e] = some ? st.l[e] : -1.f;  // (a sum is at least 0, or NaN)
    }
  }
  named_bar_sync(1, 32 * W);
  if (run.seq >= a.num_seqs) return;
  const int heads = min(8, a.group - 8 * run.qt), w0 = warp - run.piece;
  for (int hd = run.piece; hd < heads; hd += a.seq_cut) {
    // A piece whose logits are all NaN has the maximum of one without a token
    // (fmaxf passes over NaN), but sums of NaN, which any weight keeps.
    float top = kNoTokens;
    for (int p = 0; p < a.seq_cut; ++p) top = fmaxf(top, state(w0 + p)[8 * D + hd]);
    float sum = 0.f, acc[D / 32];
#pragma unroll
    for (int j = 0; j < D / 32; ++j) acc[j] = 0.f;
    for (int p = 0; p < a.seq_cut; ++p) {
      const float* from = state(w0 + p);
      if (from[8 * D + 8 + hd] < 0.f) continue;  // no unit: its values may be anything
      const float wt = fast_exp2(from[8 * D + hd] - top);
      sum = fmaf(from[8 * D + 8 + hd], wt, sum);
#pragma unroll
      for (int j = 0; j < D / 32; ++j) acc[j] = fmaf(from[hd * D + 2 * lane + 64 * (j / 2) + (j & 1)], wt, acc[j]);
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const int64_t row = static_cast<int64_t>(run.seq) * a.num_q_heads + run.h * a.group + 8 * run.qt + hd;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + row * D);
#pragma unroll
    for (int j = 0; j < D / 64; ++j) out[lane + 32 * j] = pack_bf16x2(acc[2 * j] * inv, acc[2 * j + 1] * inv);
  }
}

// q_tiles: runs of 8 query heads per KV head, ceil(group / 8).
template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, 1)
    paged_decode_q4_kernel(const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool, int q_tiles,
                           const SinksArgs a) {
  constexpr int W = Cfg::W, NS = Cfg::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + Cfg::kRingBytes);
  uint64_t* empty = full + W * NS;
  uint32_t* present = reinterpret_cast<uint32_t*>(empty + W * NS);
  int* prefix = reinterpret_cast<int*>(present + W * NS);  // [B + 1] units before sequence s
  int* first_unit = prefix + a.num_seqs + 1;               // [B]

  grid_dependents_launch();  // the merge grid may be scheduled; it waits for this grid before it reads
  if (threadIdx.x < 2 * W * NS) mbar_init(&full[threadIdx.x], 1);
  fence_barrier_init();
  const UnitLists lists = build_unit_lists<W + 4, kQ4Pad>(a, Cfg::BS, prefix, first_unit);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
  if (warp < W) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kConsumerRegs));
    q4_consume<Cfg>(a, q_tiles, lists, prefix, first_unit, ring, full, empty, present);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kProducerRegs));
    q4_produce<Cfg>(k_pool, v_pool, a, q_tiles, lists, prefix, first_unit, ring, full, empty, present, warp - W);
  }
}

}  // namespace pagedkv
