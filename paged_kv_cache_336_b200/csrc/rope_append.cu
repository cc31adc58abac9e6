// Rotary positions fused with the cache write, and the 4-bit cache's append
// and read-back (pa_rope_append, pa_rope_append_q4, pa_kv_append_q4,
// pa_kv_gather_q4, pa_rope_frequencies; see include/pagedkv.h).
//
// Rotation of pair i of a token at position p, angle f = p * inv_freq[i]:
//   a' = c a - s b,  b' = c b + s a,  c = mscale cos f, s = mscale sin f
// in fp32, rounded once to the element type. f is reduced in double: an fp32
// product is off by up to 2^-25 f radians, a whole 0.004 at position 131072.
// Writing u = f / pi (one double multiply), u - 2 rint(u / 2) in [-1, 1] is
// exact in double and loses 2^-25 of a half turn when rounded to fp32, where
// sincospif takes over.
//
// 4-bit groups: 64 dims of one (token, KV head), mn = min x,
// s = bf16((max x - mn) / 15), code = rint((x - mn) / s) in 0..15,
// value = mn + s code. x is bf16, so mn is exact. The quotient has to be the
// correctly rounded one: x, mn and s lie on coarse grids, exact ties
// (k + 1/2) are common, and a product with 1/s breaks them by its rounding.
// With r = 1/s correctly rounded, q = x r and q + r (x - q s) by two fused
// multiply-adds is the correctly rounded quotient (P. Markstein, IBM J. Res.
// Dev. 34, 1990), a third of the cost of a division per element.
//
// How. One item is two 16-byte vectors of one head of one token: in the half
// layout vector j and its partner rotary_dim / 2 further on, otherwise two
// neighbours; every item of a head is then the same work, and a head is
// head_dim / (2 x vector) neighbouring threads. A CTA takes a tile of tokens,
// puts its cos and sin in shared memory (one pair a thread, so that all heads
// of a token share them) and walks the tile's items, each thread loading
// kUnroll items before it uses any. Bound: HBM (each element read and written
// once): 16384 tokens of 32 + 8 + 8 heads of 128 in bf16 take 68.4 us in graph
// replays, 0.90 of the measured copy rate (73.6 as calls whose inputs change, 0.84);
// for a decode step, launch latency (one token 2.8 us, a call 14).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "device_common.cuh"
#include "pa_internal.h"
#include "q4_common.cuh"

namespace pagedkv {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kUnroll = 2;

struct RopeArgs {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const int32_t* positions;
  const float* inv_freq;
  const int64_t* slots;
  void* q_out;
  void* k_pool;
  void* v_pool;
  uint32_t* dev_err;
  int num_tokens, num_q_heads, num_kv_heads, rotary_dim, block_size;
  float mscale;
  // set by the launch
  int block_shift, tile_tokens;
  int64_t num_slots;
};

struct __align__(16) Vec16 {
  uint32_t w[4];
};

__device__ __forceinline__ Vec16 load16(const void* p) {
  const uint4 x = *reinterpret_cast<const uint4*>(p);
  return Vec16{{x.x, x.y, x.z, x.w}};
}
__device__ __forceinline__ void store16(void* p, const Vec16& x) {
  *reinterpret_cast<uint4*>(p) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
}

template <typename T>
struct VecOf;
template <>
struct VecOf<float> {
  static constexpr int N = 4;
  __device__ __forceinline__ static void widen(const Vec16& x, float (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(x.w[i]);
  }
  __device__ __forceinline__ static Vec16 narrow(const float (&f)[4]) {
    return Vec16{{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])}};
  }
};
template <>
struct VecOf<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ __forceinline__ static void widen(const Vec16& x, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(x.w[i]);
      f[2 * i + 1] = bf16_hi(x.w[i]);
    }
  }
  __device__ __forceinline__ static Vec16 narrow(const float (&f)[8]) {
    return Vec16{{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                  pack_bf16x2(f[6], f[7])}};
  }
};

// Rotates one item's two vectors. cs: (cos, sin) of the token's pairs. Half
// layout: pair n of the item is (x0[n], x1[n]), number `pair0 + n`;
// interleaved: (x0[0], x0[1]), ..., (x1[0], x1[1]), ...
template <typename T, bool kInterleaved>
__device__ __forceinline__ void rotate(Vec16& a, Vec16& b, const float2* cs, int pair0) {
  constexpr int N = VecOf<T>::N;
  float x[2][N], y[2][N];
  VecOf<T>::widen(a, x[0]);
  VecOf<T>::widen(b, x[1]);
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const float2 c = cs[pair0 + n];
    const int v0 = kInterleaved ? 2 * n / N : 0, i0 = kInterleaved ? 2 * n % N : n;
    const int v1 = kInterleaved ? v0 : 1, i1 = kInterleaved ? i0 + 1 : n;
    y[v0][i0] = x[v0][i0] * c.x - x[v1][i1] * c.y;
    y[v1][i1] = x[v1][i1] * c.x + x[v0][i0] * c.y;
  }
  a = VecOf<T>::narrow(y[0]);
  b = VecOf<T>::narrow(y[1]);
}

// ---- 4-bit groups ------------------------------------------------------------------------
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

// (min x) in the low half, (min -x) in the high half, over eight elements.
__device__ __forceinline__ uint32_t spread8(const Vec16& x) {
  const uint32_t lo = min_bf16x2(min_bf16x2(x.w[0], x.w[1]), min_bf16x2(x.w[2], x.w[3]));
  const uint32_t hi = max_bf16x2(max_bf16x2(x.w[0], x.w[1]), max_bf16x2(x.w[2], x.w[3]));
  const uint32_t mn = min_bf16x2(lo, lo >> 16), mx = max_bf16x2(hi, hi >> 16);
  return (mn & 0xffffu) | ((mx << 16) ^ 0x80000000u);
}

struct Quant {
  uint32_t param;  // scale (low half), minimum (high half), bf16 bits
  float s, mn, r;  // scale, minimum, 1 / scale (0: divide)
};

// A group's scale and minimum from its spread. A NaN or infinity in the group
// makes both NaN (every value of the group then reads NaN). The range is
// taken as max/2 - min/2 over 7.5, which cannot overflow and is the same
// number otherwise.
__device__ __forceinline__ Quant group_params(uint32_t spread) {
  const float mn = bf16_lo(spread), mx = -bf16_hi(spread);
  Quant g;
  const float half = 0.5f * mx - 0.5f * mn;
  // the correctly rounded quotient again; residuals of small ranges may underflow
  constexpr float kInv = 1.f / 7.5f;
  const float q0 = half * kInv;
  float s = half >= 0x1p-100f ? fmaf(fmaf(-q0, 7.5f, half), kInv, q0) : __fdiv_rn(half, 7.5f);
  float m = mn;
  if (!(fabsf(mn) < INFINITY) || !(fabsf(mx) < INFINITY)) s = m = __uint_as_float(0x7fc00000u);
  const uint32_t packed = pack_bf16x2(s, m);
  g.param = packed;
  g.s = bf16_lo(packed);
  g.mn = bf16_hi(packed);
  // outside this range 1 / s, x - mn or the residuals leave the normal range
  g.r = (g.s >= 0x1p-100f && g.s <= 0x1p100f) ? __frcp_rn(g.s) : 0.f;
  return g;
}

// Codes of eight elements, dim 0 in the lowest nibble. Adding 1.5 * 2^23 leaves
// rint(q) in the low mantissa bits; shifted sums of those words hold the codes
// and a constant.
__device__ __forceinline__ uint32_t codes8(const Vec16& x, const Quant& g) {
  float f[8];
  VecOf<__nv_bfloat16>::widen(x, f);
  uint32_t word = 0;
  if (g.r > 0.f) {
    constexpr uint32_t kBias = 0x4b400000u * 0x11111111u;  // mod 2^32
    word = 0u - kBias;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = f[i] - g.mn;
      float q = d * g.r;
      q = fmaf(fmaf(-q, g.s, d), g.r, q);  // the correctly rounded d / s, at most 15 (1 + 2^-8): no clamp
      word += __float_as_uint(q + 12582912.f) << (4 * i);
    }
  } else if (g.s > 0.f) {  // a scale near the ends of the range: halves, and a division
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = __fdiv_rn(0.5f * f[i] - 0.5f * g.mn, 0.5f * g.s);
      word |= static_cast<uint32_t>(rintf(fminf(q, 15.f))) << (4 * i);
    }
  }  // s == 0 (all equal, or a spread below half the smallest scale) or NaN: codes 0
  return word;
}

// Where a slot's code row and its parameters stand in a pool.
template <int D>
struct Q4Place {
  int64_t row, params;
  int tok;
  __device__ __forceinline__ Q4Place(int64_t slot, int64_t h, int num_kv_heads, int block_shift) {
    using Geo = Q4Geo<D>;
    const int64_t blk = slot >> block_shift;
    const int off = static_cast<int>(slot) & ((1 << block_shift) - 1);
    tok = off & 15;
    const int64_t sub = (((blk * num_kv_heads + h) << (block_shift - 4)) + (off >> 4)) * Geo::kSubBytes;
    row = sub + tok * Geo::kRowBytes;
    params = sub + Geo::kCodeBytes + tok * Geo::kParamRow;
  }
};

// Writes an item (vectors c0 and c1 of 8 dims) of token `slot`, KV head h, to
// a 4-bit pool; called by all lanes of the head's threads together (lanes
// whose token is not written pass slot < 0 and only take part in the
// shuffles). kSplit: c0 and c1 may lie in different 64-dim groups (a rotated
// half layout), and each group's spread is folded over all of the head's D / 16
// lanes, a lane adding what its vectors hold of the group; otherwise an item
// is 16 neighbouring dims and four neighbouring lanes hold a group.
template <int D, bool kValue, bool kSplit>
__device__ __forceinline__ void store_q4(uint8_t* pool, const Vec16& a, const Vec16& b, int c0, int c1,
                                         int item, int64_t slot, int h, const RopeArgs& p) {
  using Geo = Q4Geo<D>;
  constexpr uint32_t kNone = 0x7f807f80u;  // (+inf, +inf): neutral for min
  const uint32_t sa = spread8(a), sb = spread8(b);
  Quant ga, gb;
  uint32_t mine = 0;  // the parameters that this lane writes, of group `item` or item / 4
  if constexpr (kSplit) {
    uint32_t spread_a = 0, spread_b = 0, spread_i = 0;
#pragma unroll
    for (int g = 0; g < Geo::kGroups; ++g) {
      uint32_t s = kNone;
      if (c0 >> 3 == g) s = sa;
      if (c1 >> 3 == g) s = min_bf16x2(s, sb);
#pragma unroll
      for (int off = D / 32; off >= 1; off >>= 1) s = min_bf16x2(s, __shfl_xor_sync(0xffffffffu, s, off));
      if (c0 >> 3 == g) spread_a = s;
      if (c1 >> 3 == g) spread_b = s;
      if (item == g) spread_i = s;
    }
    ga = group_params(spread_a);
    gb = group_params(spread_b);
    // the lane that writes group `item`'s parameters may hold neither of its vectors
    if (item < Geo::kGroups)
      mine = spread_i == spread_a ? ga.param : spread_i == spread_b ? gb.param : group_params(spread_i).param;
  } else {
    uint32_t s = min_bf16x2(sa, sb);
    s = min_bf16x2(s, __shfl_xor_sync(0xffffffffu, s, 1));
    s = min_bf16x2(s, __shfl_xor_sync(0xffffffffu, s, 2));
    ga = gb = group_params(s);
    mine = ga.param;
  }
  if (slot < 0) return;
  const Q4Place<D> at(slot, h, p.num_kv_heads, p.block_shift);
  *reinterpret_cast<uint32_t*>(pool + at.row + Geo::template word<kValue>(at.tok, c0)) = codes8(a, ga);
  *reinterpret_cast<uint32_t*>(pool + at.row + Geo::template word<kValue>(at.tok, c1)) = codes8(b, gb);
  const int group = kSplit ? item : (item & 3) == 0 ? item >> 2 : Geo::kGroups;
  if (group < Geo::kGroups)
    *reinterpret_cast<uint32_t*>(pool + at.params + group * 4) = mine;
}

// grid.x walks tiles of tile_tokens tokens, grid.y slices of a tile's items.
template <typename T, int D, bool kInterleaved, bool kQ4>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeArgs p) {
  constexpr int N = VecOf<T>::N;
  constexpr int kItems = D / (2 * N);  // items (threads) of one head
  extern __shared__ float2 cs[];       // [tile_tokens][rotary_dim / 2]
  const int tid = threadIdx.x;
  const int half = p.rotary_dim / 2;
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  const int rot_items = p.rotary_dim / (2 * N);  // the head's first items hold its rotated dims

  for (int tile = blockIdx.x; tile * static_cast<int64_t>(p.tile_tokens) < p.num_tokens; tile += gridDim.x) {
    const int64_t tok0 = tile * static_cast<int64_t>(p.tile_tokens);
    const int nt = static_cast<int>(min(static_cast<int64_t>(p.tile_tokens), p.num_tokens - tok0));
    for (int i = tid; i < nt * half; i += kRopeThreads) {
      const int t = i / half;
      const double u = static_cast<double>(p.positions[tok0 + t]) *
                       (static_cast<double>(p.inv_freq[i - t * half]) * 0.31830988618379067154);
      float s, c;
      sincospif(static_cast<float>(u - 2.0 * rint(0.5 * u)), &s, &c);
      cs[i] = make_float2(c * p.mscale, s * p.mscale);
    }
    __syncthreads();

    const int total = nt * heads * kItems;
    const int step = gridDim.y * kRopeThreads;
    // all threads run the same number of rounds: the 4-bit path shuffles
    for (int base = blockIdx.y * kRopeThreads; base < total; base += step * kUnroll) {
      Vec16 a[kUnroll], b[kUnroll];
      int hd[kUnroll], tk[kUnroll], c0[kUnroll], c1[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int i = base + u * step + tid;
        const int item = i % kItems, th = i / kItems;
        tk[u] = th / heads;
        hd[u] = th - tk[u] * heads;
        const bool rotated = item < rot_items && hd[u] < p.num_q_heads + p.num_kv_heads;
        c0[u] = !kInterleaved && rotated ? item : 2 * item;
        c1[u] = !kInterleaved && rotated ? item + rot_items : 2 * item + 1;
        if (i >= total) {
          hd[u] = -1;
          a[u] = b[u] = Vec16{{0u, 0u, 0u, 0u}};
          continue;
        }
        const int64_t t = tok0 + tk[u];
        const T* src;
        if (hd[u] < p.num_q_heads)
          src = static_cast<const T*>(p.q) + t * p.q_stride + static_cast<int64_t>(hd[u]) * D;
        else if (hd[u] < p.num_q_heads + p.num_kv_heads)
          src = static_cast<const T*>(p.k) + t * p.k_stride + static_cast<int64_t>(hd[u] - p.num_q_heads) * D;
        else
          src = static_cast<const T*>(p.v) + t * p.v_stride +
                static_cast<int64_t>(hd[u] - p.num_q_heads - p.num_kv_heads) * D;
        a[u] = load16(src + c0[u] * N);
        b[u] = load16(src + c1[u] * N);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int item = (base + u * step + tid) % kItems;
        const bool is_q = hd[u] >= 0 && hd[u] < p.num_q_heads;
        const bool is_v = hd[u] >= p.num_q_heads + p.num_kv_heads;
        if (hd[u] >= 0 && !is_v && item < rot_items)
          rotate<T, kInterleaved>(a[u], b[u], cs + tk[u] * half, item * N);
        const int64_t t = tok0 + tk[u];
        if (is_q) {
          T* dst = static_cast<T*>(p.q_out) + (t * p.num_q_heads + hd[u]) * D;
          store16(dst + c0[u] * N, a[u]);
          store16(dst + c1[u] * N, b[u]);
        }
        int64_t slot = -1;
        if (hd[u] >= p.num_q_heads) {
          slot = p.slots[t];
          if (slot >= p.num_slots) {
            if (item == 0) report(p.dev_err, PA_DEVERR_SLOT);
            slot = -1;
          }
        }
        const int h = is_v ? hd[u] - p.num_q_heads - p.num_kv_heads : hd[u] - p.num_q_heads;
        if constexpr (kQ4) {
          // a warp's heads may be of several kinds: every lane runs both
          // kinds that occur among them, writing only its own
          const bool any_k = __any_sync(0xffffffffu, slot >= 0 && !is_v);
          const bool any_v = __any_sync(0xffffffffu, slot >= 0 && is_v);
          if (any_k)
            store_q4<D, false, !kInterleaved>(static_cast<uint8_t*>(p.k_pool), a[u], b[u], c0[u], c1[u], item,
                                              is_v ? -1 : slot, h, p);
          if (any_v)
            store_q4<D, true, false>(static_cast<uint8_t*>(p.v_pool), a[u], b[u], c0[u], c1[u], item,
                                     is_v ? slot : -1, h, p);
        } else if (slot >= 0) {
          const int64_t blk = slot >> p.block_shift;
          const int64_t row = ((blk * p.num_kv_heads + h) << p.block_shift) + (slot & (p.block_size - 1));
          T* dst = static_cast<T*>(is_v ? p.v_pool : p.k_pool) + row * D;
          store16(dst + c0[u] * N, a[u]);
          store16(dst + c1[u] * N, b[u]);
        }
      }
    }
    __syncthreads();  // cs is rewritten for the next tile
  }
}

// How the plain 4-bit append and read spread a token's `per_token` items over
// threads: a thread keeps its item (a piece of one head) in every token it
// visits, so that only the slot changes and nothing is divided per token;
// grid.x walks tokens, grid.y the items beyond a block's width.
constexpr int kRowThreads = 256;
struct RowShare {
  int item;             // -1: this thread has none
  int64_t first, step;  // its tokens: first, first + step, ...
  __device__ __forceinline__ explicit RowShare(int per_token) {
    const int width = min(per_token, kRowThreads), side = kRowThreads / width;
    const int mine = threadIdx.x / width;
    item = blockIdx.y * width + (threadIdx.x - mine * width);
    if (mine >= side || item >= per_token) item = -1;
    first = static_cast<int64_t>(blockIdx.x) * side + mine;
    step = static_cast<int64_t>(gridDim.x) * side;
  }
};

dim3 row_grid(int per_token, int64_t num_tokens, int tokens_per_thread) {
  const int width = std::min(per_token, kRowThreads), side = kRowThreads / width;
  const int64_t run = static_cast<int64_t>(side) * tokens_per_thread;
  return dim3(static_cast<unsigned>(std::min<int64_t>((num_tokens + run - 1) / run, 1 << 30)),
              static_cast<unsigned>((per_token + width - 1) / width));
}

// Quantises new rows: a thread takes the same 16 dims of K and of V; four
// neighbouring threads hold a group. About 10 instructions an element beside
// 2.6 bytes moved: 16384 rows of 8 heads of 128 take 21 us (floor 13).
constexpr int kAppendCtasPerSm = 3;  // 70 to 78 registers; measured 41.1 us (with the read) against 45.4 for 4, 43.3 for 12
template <int D>
__global__ void __launch_bounds__(kRowThreads)
    kv_append_q4_kernel(const __nv_bfloat16* __restrict__ k_new, const __nv_bfloat16* __restrict__ v_new,
                        int64_t k_stride, int64_t v_stride, const int64_t* __restrict__ slots, int num_tokens,
                        int num_kv_heads, int block_shift, int64_t num_slots, uint8_t* __restrict__ k_pool,
                        uint8_t* __restrict__ v_pool, uint32_t* dev_err) {
  using Geo = Q4Geo<D>;
  constexpr int C = D / 16;
  const RowShare sh(num_kv_heads * C);
  if (sh.item < 0) return;  // (four neighbours leave together)
  const uint32_t quad = 0xfu << (threadIdx.x & 28);
  const int item = sh.item % C, h = sh.item / C;
  Vec16 next[2][2];
  int64_t next_slot = -1;
  auto load = [&](int64_t t) {  // the next token's rows, while this one's are quantised
    if (t >= num_tokens) return;
    next_slot = slots[t];
    const __nv_bfloat16* k = k_new + t * k_stride + sh.item * 16;
    const __nv_bfloat16* v = v_new + t * v_stride + sh.item * 16;
    next[0][0] = load16(k);
    next[0][1] = load16(k + 8);
    next[1][0] = load16(v);
    next[1][1] = load16(v + 8);
  };
  load(sh.first);
  for (int64_t t = sh.first; t < num_tokens; t += sh.step) {
    const Vec16 x[2][2] = {{next[0][0], next[0][1]}, {next[1][0], next[1][1]}};
    const int64_t slot = next_slot;
    load(t + sh.step);
    if (slot < 0) continue;
    if (slot >= num_slots) {
      if (sh.item == 0) report(dev_err, PA_DEVERR_SLOT);
      continue;
    }
    const Q4Place<D> at(slot, h, num_kv_heads, block_shift);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint32_t s = min_bf16x2(spread8(x[kv][0]), spread8(x[kv][1]));
      s = min_bf16x2(s, __shfl_xor_sync(quad, s, 1));
      s = min_bf16x2(s, __shfl_xor_sync(quad, s, 2));
      const Quant g = group_params(s);
      uint8_t* pool = kv ? v_pool : k_pool;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = 2 * item + i;
        const int word = kv ? Geo::v_word(at.tok, c) : Geo::k_word(at.tok, c);
        *reinterpret_cast<uint32_t*>(pool + at.row + word) = codes8(x[kv][i], g);
      }
      if ((item & 3) == 0) *reinterpret_cast<uint32_t*>(pool + at.params + (item >> 2) * 4) = g.param;
    }
  }
}

// Values of 4-bit rows, one fp32 multiply-add each, which for bf16 is rounded a
// second time (a product and a minimum far apart would have to be split to save
// that, at most 2^-24 of the value): a thread takes the same eight dims of K and of
// V, kGatherUnroll tokens at a time (16384 rows of 8 heads of 128 with their
// append: 43.4 us for one, 41.0 for two, 41.3 for four). Bound: the 16-bit
// stores, behind a slot and then a row load.
constexpr int kGatherUnroll = 2;

template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads)
    kv_gather_q4_kernel(const uint8_t* __restrict__ k_pool, const uint8_t* __restrict__ v_pool,
                        const int64_t* __restrict__ slots, int num_tokens, int num_kv_heads, int block_shift,
                        int64_t num_slots, T* __restrict__ k_out, T* __restrict__ v_out, uint32_t* dev_err) {
  using Geo = Q4Geo<D>;
  constexpr int C = D / 8;
  const RowShare sh(num_kv_heads * C);
  if (sh.item < 0) return;
  const int c = sh.item % C, h = sh.item / C;
  for (int64_t t0 = sh.first; t0 < num_tokens; t0 += sh.step * kGatherUnroll) {
    int64_t tok_at[kGatherUnroll];
    uint32_t w[kGatherUnroll][2], q[kGatherUnroll][2];
#pragma unroll
    for (int u = 0; u < kGatherUnroll; ++u) {
      const int64_t t = t0 + u * sh.step;
      tok_at[u] = -1;
      if (t >= num_tokens) continue;
      const int64_t slot = slots[t];
      if (slot < 0) continue;
      if (slot >= num_slots) {
        if (sh.item == 0) report(dev_err, PA_DEVERR_SLOT);
        continue;
      }
      tok_at[u] = t;
      const Q4Place<D> at(slot, h, num_kv_heads, block_shift);
      w[u][0] = *reinterpret_cast<const uint32_t*>(k_pool + at.row + Geo::k_word(at.tok, c));
      w[u][1] = *reinterpret_cast<const uint32_t*>(v_pool + at.row + Geo::v_word(at.tok, c));
      q[u][0] = *reinterpret_cast<const uint32_t*>(k_pool + at.params + (c >> 3) * 4);
      q[u][1] = *reinterpret_cast<const uint32_t*>(v_pool + at.params + (c >> 3) * 4);
    }
#pragma unroll
    for (int u = 0; u < kGatherUnroll; ++u) {
      if (tok_at[u] < 0) continue;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        T* out = (kv ? v_out : k_out) + (tok_at[u] * num_kv_heads + h) * D + c * 8;
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)  // 2^23 + code, exactly
          f[j] = fmaf(__uint_as_float(0x4b000000u | ((w[u][kv] >> (4 * j)) & 15u)) - 8388608.f, bf16_lo(q[u][kv]),
                      bf16_hi(q[u][kv]));
        if constexpr (sizeof(T) == 2) {
          store16(out, VecOf<T>::narrow(f));
        } else {
          reinterpret_cast<float4*>(out)[0] = make_float4(f[0], f[1], f[2], f[3]);
          reinterpret_cast<float4*>(out)[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T, int D, bool kInterleaved, bool kQ4>
void launch_rope(RopeArgs p, cudaStream_t stream) {
  const int sms = sm_count();
  const int heads = p.num_q_heads + 2 * p.num_kv_heads;
  // Four tokens a tile amortise the cos/sin of one pair a thread over all
  // heads once the tiles still fill the GPU; a decode step takes a token a
  // tile and spreads its heads over grid.y so that no thread has two rounds.
  p.tile_tokens = p.num_tokens >= 8 * sms ? 4 : 1;
  const int64_t tiles = (static_cast<int64_t>(p.num_tokens) + p.tile_tokens - 1) / p.tile_tokens;
  const int64_t items = static_cast<int64_t>(p.tile_tokens) * heads * (D / (2 * VecOf<T>::N));
  const int64_t rounds = (items + kRopeThreads * kUnroll - 1) / (kRopeThreads * kUnroll);
  int gy = 1;
  while (gy < rounds && tiles * gy < 4 * sms) ++gy;
  // One tile a CTA: a grid of 8 CTAs per SM walking the tiles leaves some with 4
  // tiles and others with 3 at 16384 tokens.
  const int64_t gx = std::min<int64_t>(tiles, 1 << 30);
  const size_t smem = static_cast<size_t>(p.tile_tokens) * (p.rotary_dim / 2) * sizeof(float2);
  rope_append_kernel<T, D, kInterleaved, kQ4>
      <<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), kRopeThreads, smem, stream>>>(p);
}

template <typename T, int D, bool kQ4>
void pick_layout(const RopeArgs& p, bool interleaved, cudaStream_t stream) {
  if (interleaved) launch_rope<T, D, true, kQ4>(p, stream);
  else launch_rope<T, D, false, kQ4>(p, stream);
}

template <typename T, bool kQ4>
void pick_dim(const RopeArgs& p, int head_dim, bool interleaved, cudaStream_t stream) {
  if (head_dim == 64) pick_layout<T, 64, kQ4>(p, interleaved, stream);
  else if (head_dim == 128) pick_layout<T, 128, kQ4>(p, interleaved, stream);
  else pick_layout<T, 256, kQ4>(p, interleaved, stream);
}

template <int D>
void launch_append(const RopeArgs& p, cudaStream_t stream) {
  // As many CTAs as are resident, each walking its tokens a load ahead.
  dim3 grid = row_grid(p.num_kv_heads * (D / 16), p.num_tokens, 1);
  grid.x = std::min<unsigned>(grid.x, std::max<unsigned>(1u, kAppendCtasPerSm * sm_count() / grid.y));
  kv_append_q4_kernel<D><<<grid, kRowThreads, 0, stream>>>(
      static_cast<const __nv_bfloat16*>(p.k), static_cast<const __nv_bfloat16*>(p.v), p.k_stride, p.v_stride, p.slots,
      p.num_tokens, p.num_kv_heads, p.block_shift, p.num_slots, static_cast<uint8_t*>(p.k_pool),
      static_cast<uint8_t*>(p.v_pool), p.dev_err);
}

void pick_append(const RopeArgs& p, int head_dim, cudaStream_t stream) {
  if (head_dim == 64) launch_append<64>(p, stream);
  else if (head_dim == 128) launch_append<128>(p, stream);
  else launch_append<256>(p, stream);
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// Checks and launches rope_append and the two 4-bit appends (rotary_dim 0 and
// no q for the plain one).
pa_status_t run_rope(RopeArgs p, int head_dim, bool interleaved, int num_blocks, pa_dtype_t dtype, bool q4,
                     cudaStream_t stream) {
  if (p.num_tokens < 0) return fail(PA_ERR_INVALID_ARG, "num_tokens < 0");
  if (p.num_q_heads < 0 || p.num_kv_heads <= 0 || num_blocks <= 0)
    return fail(PA_ERR_INVALID_ARG, "head and block counts must be positive");
  if (dtype != PA_F32 && dtype != PA_BF16) return fail(PA_ERR_INVALID_ARG, "unknown dtype");
  if (q4 && dtype != PA_BF16) return fail(PA_ERR_UNSUPPORTED, "the 4-bit cache takes bf16 keys and values");
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(PA_ERR_UNSUPPORTED, "head_dim %d (64, 128 or 256)", head_dim);
  if (p.block_size != 16 && p.block_size != 32)
    return fail(PA_ERR_UNSUPPORTED, "block_size %d (16 or 32)", p.block_size);
  if (p.rotary_dim < 0 || p.rotary_dim > head_dim || p.rotary_dim % 2 != 0)
    return fail(PA_ERR_INVALID_ARG, "rotary_dim (%d) must be even and at most head_dim", p.rotary_dim);
  if (p.rotary_dim % 16 != 0)
    return fail(PA_ERR_UNSUPPORTED, "rotary_dim (%d) must be a multiple of 16", p.rotary_dim);
  if (!std::isfinite(p.mscale)) return fail(PA_ERR_INVALID_ARG, "mscale is not finite");
  if (p.num_tokens == 0) return ok();
  if (p.k == nullptr || p.v == nullptr || p.slots == nullptr || p.k_pool == nullptr || p.v_pool == nullptr ||
      (p.num_q_heads > 0 && (p.q == nullptr || p.q_out == nullptr)) ||
      (p.rotary_dim > 0 && (p.positions == nullptr || p.inv_freq == nullptr)))
    return fail(PA_ERR_INVALID_ARG, "NULL pointer");
  const int eb = dtype == PA_F32 ? 4 : 2;
  const int64_t qrow = static_cast<int64_t>(p.num_q_heads) * head_dim;
  const int64_t krow = static_cast<int64_t>(p.num_kv_heads) * head_dim;
  if ((p.num_q_heads > 0 && p.q_stride < qrow) || p.k_stride < krow || p.v_stride < krow)
    return fail(PA_ERR_INVALID_ARG, "a token stride is shorter than the token's heads");
  if ((p.q_stride * eb) % 16 != 0 || (p.k_stride * eb) % 16 != 0 || (p.v_stride * eb) % 16 != 0)
    return fail(PA_ERR_INVALID_ARG, "token strides must be multiples of 16 bytes");
  if (!aligned16(p.q) || !aligned16(p.k) || !aligned16(p.v) || !aligned16(p.q_out) || !aligned16(p.k_pool) ||
      !aligned16(p.v_pool))
    return fail(PA_ERR_INVALID_ARG, "q, k_new, v_new, q_out and pools must be 16-byte aligned");
  if (q4 && static_cast<int64_t>(p.num_kv_heads) * head_dim >= (int64_t(1) << 24))  // (the append's grid.y)
    return fail(PA_ERR_UNSUPPORTED, "too many heads");
  // One item's indices are 32-bit.
  if (4 * (static_cast<int64_t>(p.num_q_heads) + 2 * static_cast<int64_t>(p.num_kv_heads)) * 32 >= (int64_t(1) << 30))
    return fail(PA_ERR_UNSUPPORTED, "too many heads");
  if (p.num_q_heads > 0) {
    // q_out may be q itself (each thread writes what it alone has read), and
    // nothing else that the call reads or writes: CTAs run in any order.
    const size_t n = static_cast<size_t>(p.num_tokens), last = n - 1;
    const size_t out = n * qrow * eb;
    const bool same = p.q == p.q_out && p.q_stride == qrow;
    if ((!same && overlap(p.q_out, out, p.q, (last * p.q_stride + qrow) * eb)) ||
        overlap(p.q_out, out, p.k, (last * p.k_stride + krow) * eb) ||
        overlap(p.q_out, out, p.v, (last * p.v_stride + krow) * eb))
      return fail(PA_ERR_INVALID_ARG, "q_out overlaps an input (it may only be q itself, contiguous)");
    const size_t pool = q4 ? static_cast<size_t>(num_blocks) * p.num_kv_heads * pa_q4_tile_bytes(p.block_size, head_dim)
                           : static_cast<size_t>(num_blocks) * p.block_size * krow * eb;
    if (overlap(p.q_out, out, p.k_pool, pool) || overlap(p.q_out, out, p.v_pool, pool) ||
        overlap(p.q_out, out, p.slots, n * 8) ||
        (p.rotary_dim > 0 && (overlap(p.q_out, out, p.positions, n * 4) ||
                              overlap(p.q_out, out, p.inv_freq, static_cast<size_t>(p.rotary_dim) * 2))))
      return fail(PA_ERR_INVALID_ARG, "q_out overlaps a pool, the slots, the positions or the frequencies");
  }
  p.num_slots = static_cast<int64_t>(num_blocks) * p.block_size;
  p.block_shift = p.block_size == 16 ? 4 : 5;
  if (q4 && p.num_q_heads == 0 && p.rotary_dim == 0) pick_append(p, head_dim, stream);
  else if (q4) pick_dim<__nv_bfloat16, true>(p, head_dim, interleaved, stream);
  else if (dtype == PA_BF16) pick_dim<__nv_bfloat16, false>(p, head_dim, interleaved, stream);
  else pick_dim<float, false>(p, head_dim, interleaved, stream);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return fail(PA_ERR_CUDA, "rope_append launch: %s", cudaGetErrorString(err));
  return ok();
}

template <typename T, int D>
void launch_gather(const void* k_pool, const void* v_pool, const int64_t* slots, int T_, int H, int bs,
                   int64_t num_slots, void* k_out, void* v_out, uint32_t* err, cudaStream_t st) {
  kv_gather_q4_kernel<T, D><<<row_grid(H * (D / 8), T_, kGatherUnroll), kRowThreads, 0, st>>>(
      static_cast<const uint8_t*>(k_pool), static_cast<const uint8_t*>(v_pool), slots, T_, H, bs == 16 ? 4 : 5, num_slots,
      static_cast<T*>(k_out), static_cast<T*>(v_out), err);
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" {

size_t pa_q4_tile_bytes(int block_size, int head_dim) {
  if ((block_size != 16 && block_size != 32) || (head_dim != 64 && head_dim != 128 && head_dim != 256)) return 0;
  return static_cast<size_t>(block_size / 16) * 9 * head_dim;
}

pa_status_t pa_rope_frequencies(int rotary_dim, double base, pa_rope_scaling_t scaling, double factor,
                                int original_context, double beta_fast, double beta_slow, float* inv_freq,
                                float* mscale) {
  if (inv_freq == nullptr || mscale == nullptr) return fail(PA_ERR_INVALID_ARG, "NULL pointer");
  if (rotary_dim <= 0 || rotary_dim % 2 != 0) return fail(PA_ERR_INVALID_ARG, "rotary_dim must be positive and even");
  if (!(base > 1.0) || !std::isfinite(base)) return fail(PA_ERR_INVALID_ARG, "base must be above 1");
  if (scaling != PA_ROPE_NONE && scaling != PA_ROPE_LINEAR && scaling != PA_ROPE_NTK && scaling != PA_ROPE_YARN)
    return fail(PA_ERR_INVALID_ARG, "unknown scaling");
  if (scaling != PA_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(PA_ERR_INVALID_ARG, "factor must be at least 1");
  if (scaling == PA_ROPE_NTK && rotary_dim == 2)
    return fail(PA_ERR_INVALID_ARG, "base stretching needs rotary_dim above 2");
  if (scaling == PA_ROPE_YARN && (original_context <= 0 || !(beta_slow > 0.0) || !(beta_fast > beta_slow) ||
                                  !std::isfinite(beta_fast)))
    return fail(PA_ERR_INVALID_ARG, "the ramp needs original_context > 0 and beta_fast > beta_slow > 0");
  const double rd = rotary_dim;
  if (scaling == PA_ROPE_NTK) base *= std::pow(factor, rd / (rd - 2.0));
  double low = 0.0, high = 0.0;
  if (scaling == PA_ROPE_YARN) {
    // the (fractional) pair that makes `turns` turns over the original context
    auto dim = [&](double turns) {
      return rd * std::log(original_context / (turns * 2.0 * M_PI)) / (2.0 * std::log(base));
    };
    low = std::max(std::floor(dim(beta_fast)), 0.0);
    high = std::min(std::ceil(dim(beta_slow)), rd - 1.0);
  }
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rd);
    if (scaling == PA_ROPE_LINEAR) f /= factor;
    if (scaling == PA_ROPE_YARN) {
      const double r = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001)));
      f = f / factor * r + f * (1.0 - r);
    }
    inv_freq[i] = static_cast<float>(f);
  }
  *mscale = scaling == PA_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return ok();
}

pa_status_t pa_rope_append(const void* q, const void* k_new, const void* v_new, int64_t q_stride,
                           int64_t k_stride, int64_t v_stride, const int32_t* positions,
                           const float* inv_freq, const int64_t* slot_mapping, int num_tokens,
                           int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim, int interleaved,
                           float mscale, int block_size, int num_blocks, pa_dtype_t dtype, void* q_out,
                           void* k_pool, void* v_pool, uint32_t* dev_err, void* stream) {
  PA_NVTX_RANGE("pa_rope_append");
  RopeArgs p{q, k_new, v_new, q_stride, k_stride, v_stride, positions, inv_freq, slot_mapping, q_out, k_pool,
             v_pool, dev_err, num_tokens, num_q_heads, num_kv_heads, rotary_dim, block_size, mscale, 0, 0, 0};
  return run_rope(p, head_dim, interleaved != 0, num_blocks, dtype, false, static_cast<cudaStream_t>(stream));
}

pa_status_t pa_rope_append_q4(const void* q, const void* k_new, const void* v_new, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, const int32_t* positions,
                              const float* inv_freq, const int64_t* slot_mapping, int num_tokens,
                              int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim,
                              int interleaved, float mscale, int block_size, int num_blocks,
                              pa_dtype_t dtype, void* q_out, void* k_pool, void* v_pool, uint32_t* dev_err,
                              void* stream) {
  PA_NVTX_RANGE("pa_rope_append_q4");
  RopeArgs p{q, k_new, v_new, q_stride, k_stride, v_stride, positions, inv_freq, slot_mapping, q_out, k_pool,
             v_pool, dev_err, num_tokens, num_q_heads, num_kv_heads, rotary_dim, block_size, mscale, 0, 0, 0};
  return run_rope(p, head_dim, interleaved != 0, num_blocks, dtype, true, static_cast<cudaStream_t>(stream));
}

pa_status_t pa_kv_append_q4(const void* k_new, const void* v_new, int64_t k_stride, int64_t v_stride,
                            const int64_t* slot_mapping, int num_tokens, int num_kv_heads, int head_dim,
                            int block_size, int num_blocks, pa_dtype_t dtype, void* k_pool, void* v_pool,
                            uint32_t* dev_err, void* stream) {
  PA_NVTX_RANGE("pa_kv_append_q4");
  RopeArgs p{nullptr, k_new, v_new, 0, k_stride, v_stride, nullptr, nullptr, slot_mapping, nullptr, k_pool,
             v_pool, dev_err, num_tokens, 0, num_kv_heads, 0, block_size, 1.f, 0, 0, 0};
  return run_rope(p, head_dim, false, num_blocks, dtype, true, static_cast<cudaStream_t>(stream));
}

pa_status_t pa_kv_gather_q4(const void* k_pool, const void* v_pool, const int64_t* slot_mapping,
                            int num_tokens, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                            pa_dtype_t dtype, void* k_out, void* v_out, uint32_t* dev_err, void* stream) {
  PA_NVTX_RANGE("pa_kv_gather_q4");
  if (num_tokens < 0) return fail(PA_ERR_INVALID_ARG, "num_tokens < 0");
  if (num_kv_heads <= 0 || num_blocks <= 0) return fail(PA_ERR_INVALID_ARG, "sizes must be positive");
  if (dtype != PA_F32 && dtype != PA_BF16) return fail(PA_ERR_INVALID_ARG, "unknown dtype");
  if (pa_q4_tile_bytes(block_size, head_dim) == 0)
    return fail(PA_ERR_UNSUPPORTED, "no 4-bit cache for head_dim=%d block_size=%d", head_dim, block_size);
  if (static_cast<int64_t>(num_kv_heads) * head_dim >= (int64_t(1) << 24))  // (grid.y)
    return fail(PA_ERR_UNSUPPORTED, "too many heads");
  if (num_tokens == 0) return ok();
  if (k_pool == nullptr || v_pool == nullptr || slot_mapping == nullptr || k_out == nullptr || v_out == nullptr)
    return fail(PA_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k_out) || !aligned16(v_out))
    return fail(PA_ERR_INVALID_ARG, "pools and outputs must be 16-byte aligned");
  const int64_t slots = static_cast<int64_t>(num_blocks) * block_size;
  const size_t out = static_cast<size_t>(num_tokens) * num_kv_heads * head_dim * (dtype == PA_F32 ? 4 : 2);
  const size_t pool = static_cast<size_t>(num_blocks) * num_kv_heads * pa_q4_tile_bytes(block_size, head_dim);
  const size_t row_slots = static_cast<size_t>(num_tokens) * 8;
  if (overlap(k_out, out, v_out, out)) return fail(PA_ERR_INVALID_ARG, "k_out and v_out share memory");
  for (const void* o : {k_out, v_out})
    if (overlap(o, out, k_pool, pool) || overlap(o, out, v_pool, pool) || overlap(o, out, slot_mapping, row_slots))
      return fail(PA_ERR_INVALID_ARG, "an output shares memory with a pool or the slots");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto go = [&](auto elt) {
    using T = decltype(elt);
    if (head_dim == 64)
      launch_gather<T, 64>(k_pool, v_pool, slot_mapping, num_tokens, num_kv_heads, block_size, slots, k_out, v_out, dev_err, st);
    else if (head_dim == 128)
      launch_gather<T, 128>(k_pool, v_pool, slot_mapping, num_tokens, num_kv_heads, block_size, slots, k_out, v_out, dev_err, st);
    else
      launch_gather<T, 256>(k_pool, v_pool, slot_mapping, num_tokens, num_kv_heads, block_size, slots, k_out, v_out, dev_err, st);
  };
  if (dtype == PA_BF16) go(__nv_bfloat16{});
  else go(float{});
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return fail(PA_ERR_CUDA, "kv_gather_q4 launch: %s", cudaGetErrorString(err));
  return ok();
}

}  // extern "C"
