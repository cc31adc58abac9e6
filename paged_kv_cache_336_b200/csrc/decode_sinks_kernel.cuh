// Balanced split decode over a sliding window with sinks, for sm_100a
// (templates; instantiated in decode_inst_*.cu), and the per-sequence unit
// lists that the 4-bit decode kernel shares.
//
// What is computed: softmax(scale * K_s q) V_s over tokens t < ctx with
// t >= ctx - window or t < num_sinks; a logit of -inf weighs nothing, and a row of
// nothing but such logits is zeros, as one without a token.
// How: paged_decode_stream_kernel's cut (every warp of a persistent grid an equal
// run of a KV head's list of 16-token units, pieces merged by lse_merge_kernel),
// over lists that hold the sinks' units and then the window's, so that no other
// block is read; short windows and small batches are cut sequence by sequence
// (SinksArgs::seq_cut).
// Bound: 8 sequences of 100,000 to 131,072 tokens, window 4096 + 4, 64 heads
// over 8 in bf16: 30.4 us in graph replays (floor 20.6): 14 units a warp behind the
// launch, the lists and the first loads, then the merge.
// Rounding: the 16-bit decode's, weights to bf16 for the product with the values;
// logits, sums and the merge in fp32.
#pragma once

#include "decode_stream_kernel.cuh"

namespace pagedkv {

// Running maximum before the first token, and of a piece without weight (every
// block id bad, logits of -inf or NaN): the lowest finite value. From -inf the
// first step would take 2^(-inf - -inf), a NaN, where its logits are -inf.
constexpr float kNoTokens = -3.402823466e38f;

struct SinksArgs : DecodeArgs {
  int num_sinks;  // first tokens that stay visible beside the window
  // Lists per KV head: with fp32's CUDA-core math a KV head's group may be cut
  // into several lists of fewer query heads (num_kv_heads and group are then
  // those of the lists), each reading the head's K and V.
  int head_tiles;
  // Non-zero: each sequence's units are cut into so many equal pieces, for as
  // many neighbouring warps of one CTA (a divisor of its consumers), which merge
  // them there; no merge kernel follows.
  int seq_cut;
};

// A sliding window with sinks (the first a.num_sinks tokens stay visible): the
// list of a sequence whose window starts at token `ftok` begins with the
// ceil(num_sinks / 16) units of its sinks. Where the sinks end inside the
// window's first unit that unit is listed twice, once for each of its two
// visible runs of tokens; where they reach the window, the whole context is
// visible and there are no sink units.
constexpr int kSinkFlag = 1 << 30;  // beside a first unit: sink units precede it
__device__ __forceinline__ bool sinks_apart(const SinksArgs& a, int ftok) { return a.num_sinks < ftok; }
__device__ __forceinline__ int sink_units(const SinksArgs& a, int first_unit) {
  return (first_unit & kSinkFlag) ? (a.num_sinks + 15) / 16 : 0;
}

// Every sequence's units: first_unit[B] (-1: nothing to read) and the exclusive
// prefix sum prefix[B + 1], in shared memory, built by all threads of a CTA
// of W warps; returns the number of units of each KV head's list and of the
// longest sequence. kPad places without units follow each sequence's units in
// the list, so that an equal cut of the list also shares out what a sequence
// costs besides its units.
struct UnitLists {
  int total, longest;
};

template <int W, int kPad = 0>
__device__ __forceinline__ UnitLists build_unit_lists(const SinksArgs& a, int bs, int* prefix, int* first_unit) {
  constexpr int NT = 32 * W;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = a.num_seqs;
  const int max_tokens = a.max_blocks_per_seq * bs;
  __shared__ int warp_tot[W];
  __shared__ int warp_max_units[W];
  const int chunk = (B + NT - 1) / NT;
  const int lo = min(B, tid * chunk);
  const int hi = min(B, lo + chunk);
  int mine = 0, biggest = 0;
  for (int i = lo; i < hi; ++i) {
    const int raw = a.context_lens[i];
    const int ctx = clamp_ctx(raw, max_tokens);
    if (ctx != raw && blockIdx.x == 0) report(a.dev_err, PA_DEVERR_CONTEXT_LEN);
    const int ub = stream_first_unit(a, i, ctx, bs);
    int u = ub < 0 ? 1 : (ctx + 15) / 16 - ub;
    first_unit[i] = ub;
    const int ftok = first_token(a, ctx);
    if (ftok > 0) {
      first_unit[i] = sinks_apart(a, ftok) ? ub | kSinkFlag : 0;
      u = sinks_apart(a, ftok) ? u + (a.num_sinks + 15) / 16 : (ctx + 15) / 16;
    }
    mine += u + kPad;
    biggest = max(biggest, u);
  }
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += v;
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) biggest = max(biggest, __shfl_xor_sync(0xffffffffu, biggest, off));
  if (lane == 31) warp_tot[warp] = incl;
  if (lane == 0) warp_max_units[warp] = biggest;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < warp; ++w) base += warp_tot[w];
  int run = base + incl - mine;
  for (int i = lo; i < hi; ++i) {
    prefix[i] = run;
    const int fu = first_unit[i];
    int u = 1;
    if (fu >= 0) u = (clamp_ctx(a.context_lens[i], max_tokens) + 15) / 16 - (fu & ~kSinkFlag) + sink_units(a, fu);
    run += u + kPad;
  }
  if (tid == NT - 1) prefix[B] = base + incl;
  __syncthreads();
  int umax = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) umax = max(umax, warp_max_units[w]);
  return UnitLists{prefix[B], umax};
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::kThreads)
    paged_decode_sinks_kernel(const __grid_constant__ CUtensorMap tm_k,
                               const __grid_constant__ CUtensorMap tm_v, const SinksArgs a) {
  using T = typename Cfg::Elt;
  using Geo = typename Cfg::Geo;
  constexpr int W = Cfg::W;
  constexpr int NS = Cfg::NS;
  constexpr int BS = Cfg::BS;
  constexpr int UR = Cfg::UR;
  constexpr int UPB = Cfg::UPB;
  constexpr int D = Cfg::D;
  using WarpT = typename std::conditional<Cfg::kMma, MmaWarp<Cfg>, SimtWarp<Cfg>>::type;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::kRingBytes);
  int* misc = reinterpret_cast<int*>(smem + Cfg::kRingBytes + Cfg::kBarBytes);
  int* prefix = misc + StreamCfg<Cfg>::kMiscInts;  // [B + 1] units (per KV head) before sequence s
  int* first_unit = prefix + a.num_seqs + 1;      // [B] first unit read, -1: nothing to read

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int B = a.num_seqs;
  const int Hkv = a.num_kv_heads;
  const int G = a.group;
  const int max_tokens = a.max_blocks_per_seq * BS;

  // The merge grid (a programmatic dependent) may be scheduled now; it waits
  // on the device for this grid's completion before it reads anything.
  grid_dependents_launch();

  if (tid == 0) {
    for (int i = 0; i < W * NS; ++i) mbar_init(&bars[i], 1);
    fence_barrier_init();
    tma_prefetch_descriptor(&tm_k);
    tma_prefetch_descriptor(&tm_v);
  }

  const UnitLists lists = build_unit_lists<W>(a, BS, prefix, first_unit);
  const int U = lists.total;
  const int umax = lists.longest;
  int h, gi = 0, g0, g1, C;  // this warp's list, its group, its units, and how the list is cut
  int seq = 0, piece = 0;    // with seq_cut: its sequence and piece
  if (a.seq_cut > 0) {
    const int item = static_cast<int>(blockIdx.x) * (W / a.seq_cut) + warp / a.seq_cut;
    h = item % Hkv;
    seq = item / Hkv;
    piece = warp % a.seq_cut;
    const int first = prefix[min(seq, B)], end = prefix[min(seq + 1, B)];
    C = (end - first + a.seq_cut - 1) / a.seq_cut;
    g0 = min(first + piece * C, end);
    g1 = min(g0 + C, end);
  } else {
    const int wg = static_cast<int>(blockIdx.x) * W + warp;
    const int groups = static_cast<int>(gridDim.x) * W / Hkv;
    h = wg % Hkv;
    gi = wg / Hkv;
    C = max((U + groups - 1) / groups, (umax + a.max_pieces - 2) / (a.max_pieces - 1));
    const int64_t g_begin = static_cast<int64_t>(gi) * C;
    g0 = static_cast<int>(g_begin < U ? g_begin : U);
    g1 = gi < groups ? static_cast<int>(g_begin + C < U ? g_begin + C : U) : g0;
  }
  const int kv_heads = Hkv / a.head_tiles, kv_head = h / a.head_tiles;  // of the pools
  const int nj = g1 - g0;
  if (nj <= 0 && a.seq_cut <= 1) return;

  // Sequence of unit g of a KV head's list (last s with prefix[s] <= g) and
  // the unit's index within the sequence's units.
  auto locate = [&](int g, int& s, int& un) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= g) lo = mid; else hi = mid - 1;
    }
    s = lo;
    un = g - prefix[s];
  };

  // TMA row of unit g of head h's list (>= 0), -1 for a unit with nothing to
  // read, -2 for a block id outside the pool.
  auto unit_row = [&](int g) -> int {
    if (g >= g1) return -1;
    int s, un;
    locate(g, s, un);
    const int fu = first_unit[s];
    if (fu < 0) return -1;
    const int ns = sink_units(a, fu);
    const int u = un < ns ? un : (fu & ~kSinkFlag) + un - ns;
    const int phys = a.block_tables[static_cast<int64_t>(s) * a.max_blocks_per_seq + u / UPB];
    if (phys < 0 || phys >= a.num_blocks) return -2;
    return (phys * kv_heads + kv_head) * BS + (u % UPB) * UR;
  };

  const uint64_t policy = l2_policy(a.l2_hint);
  uint8_t* my_ring = ring + warp * NS * Cfg::kStageBytes;
  uint64_t* my_bars = bars + warp * NS;
  int y_cur = unit_row(g0 + lane);
  int y_nxt = unit_row(g0 + 32 + lane);
  int win = 0;
  uint32_t bad = 0;  // bit per stage: nothing to compute (no data or a bad block id)

  auto issue = [&](int j) {
    const int c = j >> 5;
    if (c != win) {  // advance the window of unit rows by 32 units
      y_cur = y_nxt;
      y_nxt = unit_row(g0 + (c + 1) * 32 + lane);
      win = c;
    }
    const int y = __shfl_sync(0xffffffffu, y_cur, j & 31);
    const uint32_t stage = static_cast<uint32_t>(j) % NS;
    bad = (y >= 0) ? (bad & ~(1u << stage)) : (bad | (1u << stage));
    if (lane == 0) {
      uint64_t* bar = &my_bars[stage];
      fence_proxy_async_smem();
      if (y >= 0) {
        uint8_t* kdst = my_ring + stage * Cfg::kStageBytes;
        uint8_t* vdst = kdst + Geo::kTileBytes;
        mbar_arrive_expect_tx(bar, 2 * Geo::kTileBytes);
#pragma unroll
        for (int c2 = 0; c2 < Geo::kChunks; ++c2) {
          tma_load_2d(kdst + c2 * Geo::kChunkBytes, &tm_k, bar, c2 * Geo::kBoxCols, y, policy);
          tma_load_2d(vdst + c2 * Geo::kChunkBytes, &tm_v, bar, c2 * Geo::kBoxCols, y, policy);
        }
      } else {
        if (y == -2) report(a.dev_err, PA_DEVERR_BLOCK_ID);
        mbar_arrive(bar);  // completes the phase with no data
      }
    }
  };

  const int npre = min(NS, nj);
  for (int j = 0; j < npre; ++j) issue(j);

  // ---- consume the warp's units, segment by segment ---------------------------------
  WarpT st;
  int s = 0, un = 0;
  if (nj > 0) locate(g0, s, un);
  int us = prefix[s + 1] - prefix[s];
  int seg_start = g0 - un;  // index of the segment's first unit in h's list
  int ctx = 0, ftok = 0, ub = 0, ns = 0;  // ns: sink units at the segment's head
  const int64_t q_seq_stride = static_cast<int64_t>(a.num_q_heads) * D;
  auto begin_segment = [&]() {
    ctx = clamp_ctx(a.context_lens[s], max_tokens);
    ftok = first_token(a, ctx);
    ub = first_unit[s];
    ns = ub < 0 ? 0 : sink_units(a, ub);
    if (ub >= 0) ub &= ~kSinkFlag;
    if (!sinks_apart(a, ftok)) ftok = 0;
    const T* q_group = reinterpret_cast<const T*>(a.q) + static_cast<int64_t>(s) * q_seq_stride +
                       static_cast<int64_t>(h) * G * D;
    if (s + 1 < B && seg_start + us < g1) {
      // the next segment's query rows (G x D contiguous): into L2 now
      const char* nq = reinterpret_cast<const char*>(q_group + q_seq_stride);
      const int lines = (G * D * static_cast<int>(sizeof(T)) + 127) / 128;
      for (int i = lane; i < lines; i += 32) prefetch_l2(nq + i * 128);
    }
    if constexpr (Cfg::kMma) {
      st.begin(q_group, G, a.scale_log2, lane);
    } else {
      st.begin(q_group, a.scale_log2, lane);
    }
    for (float& m : st.m) m = kNoTokens;
    if (un == 0 && a.seq_cut == 0) {  // this warp holds the segment's first piece: record the count
      const int pieces = (seg_start + us - 1) / C - seg_start / C + 1;
      if (lane == 0) a.seg_pieces[static_cast<int64_t>(s) * Hkv + h] = pieces;
    }
  };
  // Writes the segment out: final rows when this warp covered all of it, else
  // the partial slot of this warp's piece.
  auto end_segment = [&](bool reached_end) {
    const int piece = gi - seg_start / C;
    const bool whole = reached_end && seg_start >= g0;
    const int64_t row0 = static_cast<int64_t>(s) * a.num_q_heads + static_cast<int64_t>(h) * G;
    if constexpr (Cfg::kMma) {
      const int g = lane >> 2;
      if (whole) {
        T* o = reinterpret_cast<T*>(a.out) + row0 * D;
        st.store_final(o + g * D, o + (g + 8) * D, g < G, g + 8 < G, lane);
      } else {
        const int64_t pr0 = g < G ? (row0 + g) * a.max_partitions + piece : -1;
        const int64_t pr1 = g + 8 < G ? (row0 + g + 8) * a.max_partitions + piece : -1;
        st.store_partials(a, pr0, pr1, lane);
      }
    } else {
      if (whole) {
        st.store_final(reinterpret_cast<T*>(a.out) + row0 * D, lane);
      } else {
        st.store_partials(a, row0 * a.max_partitions + piece, a.max_partitions, lane);
      }
    }
  };

  if (nj > 0) begin_segment();
  bool timed_out = false;
  int j = 0;
  for (; j < nj; ++j) {
    if (un == us) {  // the previous unit ended its segment: move to the next one
      end_segment(true);
      seg_start += us;
      ++s;
      us = prefix[s + 1] - prefix[s];
      un = 0;
      begin_segment();
    }
    const uint32_t stage = static_cast<uint32_t>(j) % NS;
    const uint32_t parity = (static_cast<uint32_t>(j) / NS) & 1u;
    const bool okw = mbar_wait_bounded(&my_bars[stage], parity, a.dev_err);
    if (!__all_sync(0xffffffffu, okw)) {
      timed_out = true;
      break;
    }
    if (!(bad & (1u << stage))) {
      const bool sink = un < ns;
      const int u0 = (sink ? un : ub + un - ns) * UR;   // first token of the unit
      const int nvalid = min(UR, (sink ? a.num_sinks : ctx) - u0);
      const int nfirst = sink ? 0 : ftok - u0;          // > 0 only inside the window's first unit
      if (nfirst < nvalid) {
        uint8_t* kt = my_ring + stage * Cfg::kStageBytes;
        st.block(kt, kt + Geo::kTileBytes, nfirst, nvalid, lane);
      }
    }
    __syncwarp();
    ++un;
    if (j + NS < nj) issue(j + NS);
  }
  if (timed_out) {
    // Give copies still in flight a bounded chance to land before leaving.
    for (int jj = j; jj < min(nj, j + NS); ++jj)
      mbar_wait_bounded(&my_bars[jj % NS], (jj / NS) & 1u, a.dev_err);
  } else if (a.seq_cut <= 1) {
    end_segment(un == us);
  }
  if (a.seq_cut <= 1) return;

  // ---- pieces of one sequence, merged in shared memory: a warp's state takes the
  // place of its ring, whose last copies it has used ----------------------------------
  constexpr int kRows = Cfg::kRowsMax;
  static_assert(kRows * (D + 2) * 4 <= NS * Cfg::kStageBytes, "a warp's state fits its ring");
  auto state = [&](int w) { return reinterpret_cast<float*>(ring + w * NS * Cfg::kStageBytes); };  // m, l, values
  float* mine = state(warp);
  if (nj <= 0) {
    if (lane < kRows) {
      mine[lane] = kNoTokens;
      mine[kRows + lane] = -1.f;  // (a sum is at least 0, or NaN)
    }
  } else if constexpr (Cfg::kMma) {
    st.publish(mine, mine + kRows, mine + 2 * kRows, G, lane);
  } else {
    st.publish(mine, mine + kRows, mine + 2 * kRows, lane);
  }
  __syncthreads();
  if (seq >= B) return;
  for (int r = piece; r < G; r += a.seq_cut) {
    const int w0 = warp - piece;
    // A piece whose logits are all NaN has the maximum of one without a token
    // (fmaxf passes over NaN), but sums of NaN, which any weight keeps.
    float top = kNoTokens;
    for (int p = 0; p < a.seq_cut; ++p) top = fmaxf(top, state(w0 + p)[r]);
    float sum = 0.f, acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
    for (int p = 0; p < a.seq_cut; ++p) {
      const float* from = state(w0 + p);
      if (from[kRows + r] < 0.f) continue;  // no unit: its values may be anything
      const float wt = fast_exp2(from[r] - top);
      sum = fmaf(from[kRows + r], wt, sum);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) acc[i] = fmaf(from[2 * kRows + r * D + lane + 32 * i], wt, acc[i]);
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    T* out = reinterpret_cast<T*>(a.out) + (static_cast<int64_t>(seq) * a.num_q_heads + static_cast<int64_t>(h) * G + r) * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) out[lane + 32 * i] = Elt<T>::from_f32(acc[i] * inv);
  }
}

}  // namespace pagedkv
