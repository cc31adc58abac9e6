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
// * Work is cut as in paged_decode_stream_kernel: one list of 16-token units
//   per KV head (per 8 query heads of it where a group has more), every warp
//   of a persistent grid an equal run of its list, pieces merged by
//   lse_merge_kernel. A unit is one sub-tile of K and of V, 9 head_dim bytes
//   each and contiguous: two bulk copies into the warp's ring.
// * mma.sync m16n8k16 with the 16 tokens of a unit as the rows and 8 query
//   heads as the columns, both times: S = K Q^T, O^T = V^T P^T. A group of 8
//   heads then wastes no row (with heads as rows half would be padding).
//   Fragments come straight from the code words: which dims (or tokens) stand
//   at which k index is free as long as both operands agree, so the words
//   are stored in the order the lanes want them, and no ldmatrix or shuffle
//   is needed. Row r of S is token r / 2 (r even), 7 - r / 2 (odd), + 8 for
//   r >= 8: the rows that lanes read together then lie in different banks.
// * A code becomes bf16 128 + c by one mask-or of two codes in place: (w >> 4j)
//   & 0x000f000f | 0x43004300. The 128 is taken out by the accumulators'
//   start: -128 Q_i for S, and -136 sum p s (a product with a constant row,
//   so that it is the same rounded numbers) for O. Accumulators of O start
//   afresh each step and are added to the running O in fp32, which bounds
//   what that cancellation can cost.
// * P is scaled by s, rounded to bf16 (as P is in the 16-bit kernel), and
//   transposed between its two layouts by movmatrix.
// Bound: HBM by bytes (4.5 bits a value), with the integer pipe close behind:
// about 0.9 mask, shift and permute instructions a value.
#pragma once

#include "decode_sinks_kernel.cuh"
#include "q4_common.cuh"

namespace pagedkv {

// W warps; a stage holds US units (one softmax step); NS stages per warp.
template <int BS_, int D_, int W_, int US_, int NS_>
struct Q4Cfg {
  static constexpr int BS = BS_, D = D_, W = W_, US = US_, NS = NS_;
  static constexpr int UPB = BS / 16;
  using Geo = Q4Geo<D>;
  static constexpr int kThreads = 32 * W;
  static constexpr int kStageBytes = US * 2 * Geo::kSubBytes;  // K units, then V units
  static constexpr int kRingBytes = W * NS * kStageBytes;
  static constexpr int kFixedSmem = 128 + kRingBytes + W * NS * 8;
  static_assert(kRingBytes % 16 == 0 && US <= 4 && US * NS <= 32, "stage layout");
  static_assert(kFixedSmem + (2 * 4096 + 1) * 4 <= 226 * 1024, "shared memory budget exceeded");
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

// D = A * B + C with D and C apart.
__device__ __forceinline__ void mma_bf16_init(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                              const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// 8x8 transpose of 16-bit elements across the warp (mma fragment layout).
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Codes j (low half) and j + 4 (high half) of a word as bf16 128 + code.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int j) { return ((w >> (4 * j)) & 0x000f000fu) | 0x43004300u; }

// N consecutive 32-bit words of shared memory, N * 4 bytes aligned.
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
    static_assert(N == 1, "1, 2 or 4 words");
    w[0] = *reinterpret_cast<const uint32_t*>(p);
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

  uint32_t qb[GR][4][2];  // query operand
  float nq[GR][2];        // -128 Q_i of heads 2t, 2t + 1
  float o[GR][4][4];      // O^T: dims 64 i + 8 g + 2 j (+ 1 for e >= 2), head 2t + (e & 1)
  float mid[GR][2];       // sum p (mn + 8 s) over this lane's tokens
  float m[2], l[2];       // running max (log2 domain), this lane's part of the sum
  float scale_log2;

  __device__ __forceinline__ void begin(const __nv_bfloat16* row, bool valid, float scale, int lane) {
    const int t = lane & 3;
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (valid) x = *reinterpret_cast<const uint4*>(row + 64 * i + 16 * t + 8 * w);
        qb[i][2 * w][0] = __byte_perm(x.x, x.z, 0x5410);      // dims 0, 4
        qb[i][2 * w][1] = __byte_perm(x.x, x.z, 0x7632);      // dims 1, 5
        qb[i][2 * w + 1][0] = __byte_perm(x.y, x.w, 0x5410);  // dims 2, 6
        qb[i][2 * w + 1][1] = __byte_perm(x.y, x.w, 0x7632);  // dims 3, 7
        sum += ((bf16_lo(x.x) + bf16_hi(x.x)) + (bf16_lo(x.y) + bf16_hi(x.y))) +
               ((bf16_lo(x.z) + bf16_hi(x.z)) + (bf16_lo(x.w) + bf16_hi(x.w)));
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      nq[i][0] = -128.f * __shfl_sync(0xffffffffu, sum, 8 * t);
      nq[i][1] = -128.f * __shfl_sync(0xffffffffu, sum, 8 * t + 4);
      mid[i][0] = mid[i][1] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
    }
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    scale_log2 = scale;
  }

  // One step: the units u with bit u of `use` set (at least one). Token r of
  // unit u takes part if lo[u] <= r < hi[u]; with kEdge false all do. Rows
  // outside may hold anything, NaN parameters included.
  template <bool kEdge>
  __device__ __forceinline__ void step(const uint8_t* stage, uint32_t use, const int (&lo)[US], const int (&hi)[US],
                                       int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int tok = (g & 1) ? 7 - (g >> 1) : (g >> 1);  // rows g and g + 8 of S: tokens tok, tok + 8
    float x[US][4];
    // ---- S = K Q^T -----------------------------------------------------------------
#pragma unroll
    for (int u = 0; u < US; ++u) {
      if (kEdge && !(use >> u & 1)) {
        x[u][0] = x[u][1] = x[u][2] = x[u][3] = -INFINITY;
        continue;
      }
      const uint8_t* kt = stage + u * Geo::kSubBytes;
      uint32_t w[2][2 * GR], par[2][GR];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint8_t* row = kt + (tok + 8 * r) * Geo::kRowBytes;
        if constexpr (D == 256) {
          uint32_t p0[4], p1[4];
          lds_words(row + ((tok & 1) * 64) + t * 16, p0);
          lds_words(row + ((tok & 1) ^ 1) * 64 + t * 16, p1);
#pragma unroll
          for (int c = 0; c < 4; ++c) w[r][c] = p0[c], w[r][4 + c] = p1[c];
        } else {
          lds_words(row + t * (8 * GR), w[r]);
        }
        lds_words(kt + Geo::kCodeBytes + (tok + 8 * r) * Geo::kParamRow, par[r]);
      }
      x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0.f;
#pragma unroll
      for (int i = 0; i < GR; ++i) {
        float s[4];
        const float start[4] = {nq[i][0], nq[i][1], nq[i][0], nq[i][1]};
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint32_t wa = w[0][2 * i + (ks >> 1)], wb = w[1][2 * i + (ks >> 1)];
          const int j = 2 * (ks & 1);
          const uint32_t a[4] = {code_pair(wa, j), code_pair(wb, j), code_pair(wa, j + 1), code_pair(wb, j + 1)};
          if (ks == 0) mma_bf16_init(s, a, qb[i][ks][0], qb[i][ks][1], start);
          else mma_bf16_16816(s, a, qb[i][ks][0], qb[i][ks][1]);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float sc = bf16_lo(par[r][i]), mn = bf16_hi(par[r][i]) * -0.0078125f;  // mn Q = (-mn / 128) nq
          x[u][2 * r] = fmaf(s[2 * r], sc, fmaf(mn, nq[i][0], x[u][2 * r]));
          x[u][2 * r + 1] = fmaf(s[2 * r + 1], sc, fmaf(mn, nq[i][1], x[u][2 * r + 1]));
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[u][e] *= scale_log2;
        if (kEdge) {
          const int r = tok + 8 * (e >> 1);
          if (r < lo[u] || r >= hi[u]) x[u][e] = -INFINITY;
        }
      }
    }
    // ---- running softmax over the step's tokens ------------------------------------
    float alpha[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = fmaxf(x[0][h], x[0][2 + h]);
#pragma unroll
      for (int u = 1; u < US; ++u) mx = fmaxf(mx, fmaxf(x[u][h], x[u][2 + h]));
#pragma unroll
      for (int off = 4; off <= 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float mn = fmaxf(m[h], mx);
      alpha[h] = fast_exp2(m[h] - mn);
      m[h] = mn;
      l[h] *= alpha[h];
#pragma unroll
      for (int i = 0; i < GR; ++i) mid[i][h] *= alpha[h];
    }
    // ---- O^T += V^T P^T --------------------------------------------------------------
    uint32_t pb[US][GR][2];
#pragma unroll
    for (int u = 0; u < US; ++u) {
      if (kEdge && !(use >> u & 1)) continue;
      const uint8_t* vt = stage + (US + u) * Geo::kSubBytes;
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[e] = fast_exp2(x[u][e] - m[e & 1]);
        l[e & 1] += p[e];
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t par[GR];
        lds_words(vt + Geo::kCodeBytes + (tok + 8 * r) * Geo::kParamRow, par);
        const bool out = kEdge && (tok + 8 * r < lo[u] || tok + 8 * r >= hi[u]);
#pragma unroll
        for (int i = 0; i < GR; ++i) {
          if (out) par[i] = 0u;
          const float sc = bf16_lo(par[i]);
          const float mi = fmaf(8.f, sc, bf16_hi(par[i]));
          pb[u][i][r] = movmatrix(pack_bf16x2(p[2 * r] * sc, p[2 * r + 1] * sc));
          mid[i][0] = fmaf(p[2 * r], mi, mid[i][0]);
          mid[i][1] = fmaf(p[2 * r + 1], mi, mid[i][1]);
        }
      }
    }
    constexpr uint32_t kNeg136 = 0xc308c308u;
    const uint32_t neg[4] = {kNeg136, kNeg136, kNeg136, kNeg136};
    float start[GR][4];
#pragma unroll
    for (int i = 0; i < GR; ++i) {
      start[i][0] = start[i][1] = start[i][2] = start[i][3] = 0.f;
#pragma unroll
      for (int u = 0; u < US; ++u)
        if (!kEdge || (use >> u & 1)) mma_bf16_16816(start[i], neg, pb[u][i][0], pb[u][i][1]);
    }
    float acc[GR][4][4];
#pragma unroll
    for (int i = 0; i < GR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = start[i][e];
#pragma unroll
    for (int u = 0; u < US; ++u) {
      if (kEdge && !(use >> u & 1)) continue;
      const uint8_t* vt = stage + (US + u) * Geo::kSubBytes;
      uint32_t w[4][GR];  // tokens t, 7 - t, 8 + t, 15 - t: k indices 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int tk = (r & 1) ? 7 - t + 8 * (r >> 1) : t + 8 * (r >> 1);
        lds_words(vt + tk * Geo::kRowBytes + ((g ^ Geo::v_turn(tk)) * (D / 16)), w[r]);
      }
#pragma unroll
      for (int i = 0; i < GR; ++i) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t sel = half ? 0x7632u : 0x5410u;
          const uint32_t wa = __byte_perm(w[0][i], w[1][i], sel), wb = __byte_perm(w[2][i], w[3][i], sel);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t a[4] = {code_pair(wa, 2 * j), code_pair(wa, 2 * j + 1), code_pair(wb, 2 * j),
                                   code_pair(wb, 2 * j + 1)};
            mma_bf16_16816(acc[i][2 * half + j], a, pb[u][i][0], pb[u][i][1]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < GR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][j][e] = fmaf(o[i][j][e], alpha[e & 1], acc[i][j][e]);
  }

  // Completes the sums over lanes; then head 2t + h's dims 64 i + 8 g + 0..7 are
  // value(i, h, 0..7).
  __device__ __forceinline__ void finish() {
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

// q_tiles: runs of 8 query heads per KV head, ceil(group / 8).
template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads, 1)
    paged_decode_q4_kernel(const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool, int q_tiles,
                           const SinksArgs a) {
  using Geo = typename Cfg::Geo;
  constexpr int W = Cfg::W, NS = Cfg::NS, US = Cfg::US, BS = Cfg::BS, UPB = Cfg::UPB, D = Cfg::D;
  constexpr uint32_t kUnitMask = (1u << US) - 1u;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kRingBytes);
  int* prefix = reinterpret_cast<int*>(bars + W * NS);  // [B + 1] units before sequence s
  int* first_unit = prefix + a.num_seqs + 1;            // [B]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = a.num_seqs;
  const int max_tokens = a.max_blocks_per_seq * BS;
  grid_dependents_launch();  // the merge grid may be scheduled; it waits for this grid before it reads
  if (tid == 0) {
    for (int i = 0; i < W * NS; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
  }
  const UnitLists lists = build_unit_lists<W>(a, BS, prefix, first_unit);

  // ---- this warp's list and run of units -----------------------------------------------
  const int num_lists = a.num_kv_heads * q_tiles;
  const int wg = static_cast<int>(blockIdx.x) * W + warp;
  const int groups = static_cast<int>(gridDim.x) * W / num_lists;
  const int h = (wg % num_lists) / q_tiles, qt = wg % q_tiles;  // KV head, run of its query heads
  const int gi = wg / num_lists;
  const int C = max((lists.total + groups - 1) / groups, (lists.longest + a.max_pieces - 2) / (a.max_pieces - 1));
  const int64_t g_begin = static_cast<int64_t>(gi) * C;
  const int g0 = static_cast<int>(min(g_begin, static_cast<int64_t>(lists.total)));
  const int g1 = static_cast<int>(min(g_begin + C, static_cast<int64_t>(lists.total)));
  if (gi >= groups || g1 <= g0) return;

  auto locate = [&](int g) {  // last s with prefix[s] <= g
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= g) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  // Sub-tile of unit g of the list (>= 0), -1: nothing to read, -2: block id outside the pool.
  auto unit_row = [&](int g) -> int {
    if (g >= g1) return -1;
    const int s = locate(g);
    const int fu = first_unit[s];
    if (fu < 0) return -1;
    const int un = g - prefix[s], ns = sink_units(a, fu);
    const int u = un < ns ? un : (fu & ~kSinkFlag) + un - ns;
    const int phys = a.block_tables[static_cast<int64_t>(s) * a.max_blocks_per_seq + u / UPB];
    if (phys < 0 || phys >= a.num_blocks) return -2;
    return (phys * a.num_kv_heads + h) * UPB + u % UPB;
  };

  const uint64_t policy = l2_policy(a.l2_hint);
  uint8_t* ring = smem + warp * NS * Cfg::kStageBytes;
  uint64_t* my_bars = bars + warp * NS;

  // ---- producer: steps of up to US units of one sequence ----------------------------------
  int win = g0;                                  // rows of units win + lane, win + 32 + lane
  int row_cur = unit_row(g0 + lane), row_nxt = unit_row(g0 + 32 + lane);
  int pg = g0, ps = locate(g0);                  // next unit to ask for, its sequence
  int p_end = min(prefix[ps + 1], g1);           // end of that sequence's units in this run
  uint32_t present = 0;                          // US bits per stage: the unit was asked for
  int issued = 0;
  auto issue = [&]() {
    const int n = min(US, p_end - pg);
    const int stage = issued % NS;
    const int i = lane & 15;                     // lanes 0..n-1 bring K units, 16..16+n-1 V units
    const int at = pg + min(i, n - 1) - win;
    const int r0 = __shfl_sync(0xffffffffu, row_cur, at & 31), r1 = __shfl_sync(0xffffffffu, row_nxt, at & 31);
    const int row = at < 32 ? r0 : r1;
    const uint32_t got = __ballot_sync(0xffffffffu, lane < n && row >= 0);
    present = (present & ~(kUnitMask << (US * stage))) | (got << (US * stage));
    uint64_t* bar = &my_bars[stage];
    fence_proxy_async_smem();                    // the stage's reads precede its next copies
    if (lane == 0) {
      if (got) mbar_arrive_expect_tx(bar, 2 * Geo::kSubBytes * __popc(got));
      else mbar_arrive(bar);                     // completes the phase with no data
    }
    if (lane < n && row == -2) report(a.dev_err, PA_DEVERR_BLOCK_ID);
    __syncwarp();
    if (i < n && row >= 0) {
      const bool v = lane >= 16;
      bulk_load(ring + stage * Cfg::kStageBytes + ((v ? US : 0) + i) * Geo::kSubBytes,
                (v ? v_pool : k_pool) + static_cast<int64_t>(row) * Geo::kSubBytes, Geo::kSubBytes, bar, policy);
    }
    ++issued;
    pg += n;
    if (pg - win >= 32) {
      win += 32;
      row_cur = row_nxt;
      row_nxt = unit_row(win + 32 + lane);
    }
    if (pg == p_end && pg < g1) {
      ++ps;
      p_end = min(prefix[ps + 1], g1);
    }
  };
  for (int i = 0; i < NS && pg < g1; ++i) issue();

  // ---- consumer ------------------------------------------------------------------------------
  Q4Warp<Cfg> st;
  const int g = lane >> 2, t = lane & 3;
  const int heads = min(8, a.group - 8 * qt);    // of this run
  const int head0 = h * a.group + 8 * qt;
  int s = locate(g0);
  int seg0 = prefix[s], seg1 = prefix[s + 1];    // the sequence's units in the list
  int ctx = 0, ftok = 0, ub = 0, ns = 0;
  auto begin_segment = [&]() {
    ctx = clamp_ctx(a.context_lens[s], max_tokens);
    ftok = first_token(a, ctx);
    ub = first_unit[s];
    ns = ub < 0 ? 0 : sink_units(a, ub);
    if (ub >= 0) ub &= ~kSinkFlag;
    if (!sinks_apart(a, ftok)) ftok = 0;
    const __nv_bfloat16* row = static_cast<const __nv_bfloat16*>(a.q) +
                               (static_cast<int64_t>(s) * a.num_q_heads + head0 + g) * D;
    if (seg1 < g1 && t == 0 && g < heads) {      // the next sequence's query rows: into L2 now
      const char* nq = reinterpret_cast<const char*>(row + static_cast<int64_t>(a.num_q_heads) * D);
      for (int b = 0; b < D * 2; b += 128) prefetch_l2(nq + b);
    }
    st.begin(row, g < heads, a.scale_log2, lane);
    if (seg0 >= g0 && qt == 0 && lane == 0)      // the first piece's warp records how many there are
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
      else st.store_partial(a, row * a.max_partitions + gi - seg0 / C, e, g);
    }
  };

  begin_segment();
  int done = 0, cg = g0;
  bool timed_out = false;
  while (cg < g1) {
    if (cg == seg1) {
      end_segment();
      ++s;
      seg0 = seg1;
      seg1 = prefix[s + 1];
      begin_segment();
    }
    const int n = min(US, min(seg1, g1) - cg);
    const int stage = done % NS;
    const bool okw = mbar_wait_bounded(&my_bars[stage], (done / NS) & 1, a.dev_err);
    if (!__all_sync(0xffffffffu, okw)) {
      timed_out = true;
      break;
    }
    const uint32_t got = (present >> (US * stage)) & kUnitMask;
    const uint8_t* data = ring + stage * Cfg::kStageBytes;
    const int un = cg - seg0;                    // index in the sequence's units
    const int u0 = (ub + un - ns) * 16;          // first token, past the sinks
    int lo[US], hi[US];
    if (got == kUnitMask && un >= ns && u0 >= ftok && u0 + 16 * US <= ctx) {
      st.template step<false>(data, got, lo, hi, lane);
    } else {
      uint32_t use = 0;
#pragma unroll
      for (int u = 0; u < US; ++u) {
        const bool sink = un + u < ns;
        lo[u] = sink ? 0 : ftok - (u0 + 16 * u);
        hi[u] = min(16, sink ? a.num_sinks - 16 * (un + u) : ctx - (u0 + 16 * u));
        if ((got >> u & 1) && lo[u] < hi[u] && lo[u] < 16 && hi[u] > 0) use |= 1u << u;
      }
      if (use) st.template step<true>(data, use, lo, hi, lane);
    }
    __syncwarp();
    cg += n;
    ++done;
    if (pg < g1) issue();
  }
  if (timed_out) {
    // Give copies still in flight a bounded chance to land before leaving.
    for (int j = done; j < issued; ++j) mbar_wait_bounded(&my_bars[j % NS], (j / NS) & 1, a.dev_err);
  } else {
    end_segment();
  }
}

}  // namespace pagedkv
