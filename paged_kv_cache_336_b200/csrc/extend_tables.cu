// Block tables, slots and positions of a step built on the GPU from request
// lengths (pa_extend_tables, see include/pagedkv.h).
//
// What is computed. Sequence s holds ctx_s tokens in have_s = ceil(ctx_s / bs)
// blocks and receives new_s tokens, so it needs
//   need_s = ceil((ctx_s + new_s) / bs) - have_s
// blocks. With the exclusive prefix sums N_s (need), R_s (blocks of leaving
// sequences) and Q_s (new tokens), in sequence order:
//   table[s][have_s + j] = queue[(head + N_s + j) mod cap],      j < need_s
//   queue[(head + count + R_s + j) mod cap] = j-th held block of s,  s leaves
//   token Q_s + i: position ctx_s + i, slot table[s][p / bs] * bs + p % bs
// which is the host block manager's policy (a FIFO queue, all or nothing;
// "What is PagedAttention?", How It Works) without reference counts.
//
// How. One launch. Every CTA builds the three prefix sums of the whole batch
// in shared memory (at most 4096 sequences: a few loads per thread), reaches
// the same verdict on whether the call can be met, and then writes its share
// of the tokens (four per thread: one 16-byte store of positions, two of
// slots), new table entries and returned blocks, each found by a binary
// search in the sums. No CTA reads what another writes: a token in a new
// block takes its id from the queue, not from the table, and the queue's
// read and written places are disjoint because count + returned <= cap.
// Bound (graph replays; a call's host time is 10 us): launch latency and three
// dependent global round trips for a decode step (256 sequences 5.2 us); for a
// prefill wave the sums and table reads that every CTA repeats, then 12 bytes a
// token (512 sequences, 465,000 tokens, some sequences leaving: 10.3 us).
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>

#include "device_common.cuh"
#include "pa_internal.h"

namespace pagedkv {
namespace {

constexpr int kExtThreads = 256;
constexpr int kExtMaxSeqs = 4096;
constexpr int kLeaves = static_cast<int>(0x80000000u);  // flag beside a sequence's sum of returned blocks

struct ExtendArgs {
  int32_t* tables;
  const int32_t* ctx;
  const int32_t* new_lens;
  int32_t* queue;
  const int32_t* state;
  int num_seqs, mbs, bs, cap, max_tokens;
  int32_t* ctx_out;
  int32_t* query_start;
  int32_t* positions;
  int64_t* slots;
  int32_t* state_out;
  uint32_t* dev_err;
};

__device__ __forceinline__ int blocks_of(int tokens, int bs) { return (tokens + bs - 1) / bs; }
__device__ __forceinline__ bool in_pool(int id, int cap) { return id >= 0 && id < cap; }

// Last s with prefix[s] <= x, for prefix[0] = 0 and x < prefix[n].
__device__ __forceinline__ int find_seq(const int* prefix, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kExtThreads) extend_tables_kernel(const ExtendArgs a) {
  extern __shared__ int sm[];
  const int B = a.num_seqs;
  int* qs = sm;               // [B + 1] new tokens before sequence s
  int* ns = qs + B + 1;       // [B + 1] blocks taken before s
  int* rs = ns + B + 1;       // [B] blocks returned before s, kLeaves if s itself leaves
  int* cs = rs + B;           // [B] context lengths
  __shared__ int64_t tot[3][kExtThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs = a.bs;
  const int64_t max_ctx = static_cast<int64_t>(a.mbs) * bs;

  // ---- prefix sums; refusals ------------------------------------------------------
  const int chunk = (B + kExtThreads - 1) / kExtThreads;
  const int lo = min(B, tid * chunk), hi = min(B, lo + chunk);
  const int head = a.state[0], count = a.state[1];
  int64_t v[3] = {0, 0, 0};
  int bad = 0, leaves = 0;
  for (int i = lo; i < hi; ++i) {
    const int c = a.ctx[i], n = a.new_lens[i];
    cs[i] = c;
    qs[i] = n;  // until the running sums take its place below
    if (c < 0 || n < -1 || static_cast<int64_t>(c) + max(n, 0) > max_ctx) bad = 1;
    if (n < 0) leaves = 1;
  }
  uint32_t refused = __syncthreads_or(bad) ? PA_DEVERR_CONTEXT_LEN : 0u;
  // Blocks of the leaving sequences, a warp per sequence: entries of -1
  // (released before a window) were returned before.
  if (__syncthreads_or(leaves && refused == 0)) {
    // The leaving sequences are dealt to the warps in turn: in batch order a
    // warp could meet several of them while others meet none.
    __shared__ int num_gone;
    if (tid == 0) num_gone = 0;
    __syncthreads();
    for (int i = lo; i < hi; ++i)
      if (qs[i] < 0) ns[atomicAdd(&num_gone, 1)] = i;  // (ns is not in use yet; any order does)
    __syncthreads();
    for (int k = warp; k < num_gone; k += kExtThreads / 32) {
      const int s = ns[k];
      const int32_t* row = a.tables + static_cast<int64_t>(s) * a.mbs;
      const int have = blocks_of(cs[s], bs);
      int held = 0;
      for (int j0 = 0; j0 < have; j0 += 256) {  // eight loads in flight
        int id[8];
#pragma unroll
        for (int v = 0; v < 8; ++v) id[v] = j0 + 32 * v + lane < have ? row[j0 + 32 * v + lane] : -1;
#pragma unroll
        for (int v = 0; v < 8; ++v) held += in_pool(id[v], a.cap);
      }
      held = __reduce_add_sync(0xffffffffu, held);
      if (lane == 0) rs[s] = held;
    }
    __syncthreads();
  }
  auto item = [&](int i, int (&x)[3]) {
    const int c = cs[i], n = qs[i];
    x[0] = max(n, 0);
    x[1] = n > 0 ? blocks_of(c + n, bs) - blocks_of(c, bs) : 0;
    x[2] = n < 0 ? rs[i] : 0;
  };
  if (refused == 0) {
    for (int i = lo; i < hi; ++i) {
      int x[3];
      item(i, x);
      for (int k = 0; k < 3; ++k) v[k] += x[k];
    }
  }
  int64_t incl[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    incl[k] = v[k];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl[k], off);
      if (lane >= off) incl[k] += up;
    }
    if (lane == 31) tot[k][warp] = incl[k];
  }
  __syncthreads();
  int64_t total[3], before[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    int64_t base = 0, all = 0;
    for (int w = 0; w < kExtThreads / 32; ++w) {
      if (w < warp) base += tot[k][w];
      all += tot[k][w];
    }
    before[k] = base + incl[k] - v[k];
    total[k] = all;
  }
  if (head < 0 || head >= a.cap || count < 0 || count > a.cap || count + total[2] > a.cap)
    refused |= PA_DEVERR_FREE_QUEUE;
  else if (total[1] > count)
    refused |= PA_DEVERR_NO_FREE_BLOCKS;
  if (total[0] > a.max_tokens) refused |= PA_DEVERR_NUM_TOKENS;

  const int64_t stride = static_cast<int64_t>(gridDim.x) * kExtThreads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kExtThreads + tid;
  if (refused) {  // nothing is taken: padding tokens, lengths as they were
    for (int64_t i = first; i < a.max_tokens; i += stride) {
      a.positions[i] = 0;
      a.slots[i] = -1;
    }
    for (int64_t i = first; i <= B; i += stride) {
      a.query_start[i] = 0;
      if (i < B) a.ctx_out[i] = a.ctx[i];
    }
    if (first == 0) {
      a.state_out[0] = head;
      a.state_out[1] = count;
      report(a.dev_err, refused);
    }
    return;
  }
  int run[3] = {static_cast<int>(before[0]), static_cast<int>(before[1]), static_cast<int>(before[2])};
  for (int i = lo; i < hi; ++i) {
    const int c = cs[i], n = qs[i];
    int x[3];
    item(i, x);
    qs[i] = run[0];
    ns[i] = run[1];
    rs[i] = run[2] | (n < 0 ? kLeaves : 0);
    for (int k = 0; k < 3; ++k) run[k] += x[k];
    if (blockIdx.x == 0) {
      a.ctx_out[i] = n < 0 ? 0 : c + n;
      a.query_start[i] = qs[i];
    }
  }
  const int T = static_cast<int>(total[0]), taken = static_cast<int>(total[1]),
            returned = static_cast<int>(total[2]);
  if (tid == kExtThreads - 1) {
    qs[B] = T;
    ns[B] = taken;
    if (blockIdx.x == 0) {
      a.query_start[B] = T;
      const int64_t nh = (static_cast<int64_t>(head) + taken) % a.cap;
      a.state_out[0] = static_cast<int>(nh);
      a.state_out[1] = count - taken + returned;
    }
  }
  __syncthreads();

  auto queue_at = [&](int i) {  // place of the i-th block taken by this call
    int64_t at = static_cast<int64_t>(head) + i;
    if (at >= a.cap) at -= a.cap;
    return a.queue + at;
  };

  // ---- positions and slots, four tokens per thread -----------------------------------
  const int64_t quads = (static_cast<int64_t>(a.max_tokens) + 3) / 4;
  for (int64_t qd = first; qd < quads; qd += stride) {
    const int t0 = static_cast<int>(qd * 4);
    int pos[4], id[4];
    int64_t slot[4];
    int s = t0 < T ? find_seq(qs, B, t0) : B;
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // the four block ids are asked for together
      const int t = t0 + k;
      pos[k] = 0;
      id[k] = INT_MIN;
      if (t >= T) continue;
      while (t >= qs[s + 1]) ++s;
      const int c = cs[s];
      pos[k] = c + (t - qs[s]);
      const int b = pos[k] / bs, have = blocks_of(c, bs);
      const int32_t* src = b < have ? a.tables + static_cast<int64_t>(s) * a.mbs + b : queue_at(ns[s] + b - have);
      id[k] = *src;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      slot[k] = -1;
      if (in_pool(id[k], a.cap)) slot[k] = static_cast<int64_t>(id[k]) * bs + pos[k] % bs;
      else if (t0 + k < T) report(a.dev_err, PA_DEVERR_BLOCK_ID);
    }
    if (t0 + 4 <= a.max_tokens) {
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      reinterpret_cast<longlong2*>(a.slots + t0)[0] = make_longlong2(slot[0], slot[1]);
      reinterpret_cast<longlong2*>(a.slots + t0)[1] = make_longlong2(slot[2], slot[3]);
    } else {
      for (int k = 0; t0 + k < a.max_tokens; ++k) {
        a.positions[t0 + k] = pos[k];
        a.slots[t0 + k] = slot[k];
      }
    }
  }

  // ---- new table entries; blocks of leaving sequences back to the queue ---------------
  // (from the last thread and warp on: a step with few tokens leaves those idle above)
  for (int64_t i = stride - 1 - first; i < taken; i += stride) {
    const int s = find_seq(ns, B, static_cast<int>(i));
    const int have = blocks_of(cs[s], bs);
    a.tables[static_cast<int64_t>(s) * a.mbs + have + (i - ns[s])] = *queue_at(static_cast<int>(i));
  }
  if (returned > 0) {
    const int warps = gridDim.x * (kExtThreads / 32);
    for (int s = warps - 1 - (blockIdx.x * (kExtThreads / 32) + warp); s < B; s += warps) {
      if (!(rs[s] & kLeaves)) continue;
      const int32_t* row = a.tables + static_cast<int64_t>(s) * a.mbs;
      const int have = blocks_of(cs[s], bs);
      int64_t at = static_cast<int64_t>(head) + count + (rs[s] & ~kLeaves);
#pragma unroll 4
      for (int j0 = 0; j0 < have; j0 += 32) {
        const int id = j0 + lane < have ? row[j0 + lane] : -1;
        const bool mine = in_pool(id, a.cap);
        if (!mine && id != -1) report(a.dev_err, PA_DEVERR_BLOCK_ID);
        const uint32_t all = __ballot_sync(0xffffffffu, mine);
        if (mine) a.queue[(at + __popc(all & ((1u << lane) - 1u))) % a.cap] = id;
        at += __popc(all);
      }
    }
  }
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" pa_status_t pa_extend_tables(int32_t* block_tables, const int32_t* context_lens,
                                        const int32_t* new_lens, int num_seqs, int max_blocks_per_seq,
                                        int block_size, int32_t* free_queue, int num_blocks,
                                        const int32_t* queue_state, int max_tokens,
                                        int32_t* context_lens_out, int32_t* query_start,
                                        int32_t* positions, int64_t* slot_mapping,
                                        int32_t* queue_state_out, uint32_t* dev_err, void* stream) {
  PA_NVTX_RANGE("pa_extend_tables");
  if (num_seqs < 0 || max_tokens < 0) return fail(PA_ERR_INVALID_ARG, "num_seqs and max_tokens must be >= 0");
  if (num_seqs > kExtMaxSeqs)
    return fail(PA_ERR_UNSUPPORTED, "pa_extend_tables takes at most %d sequences", kExtMaxSeqs);
  if (max_blocks_per_seq <= 0 || block_size <= 0 || num_blocks <= 0)
    return fail(PA_ERR_INVALID_ARG, "max_blocks_per_seq, block_size and num_blocks must be positive");
  if (static_cast<int64_t>(max_blocks_per_seq) * block_size >= (int64_t(1) << 31) - block_size)
    return fail(PA_ERR_INVALID_ARG, "max_blocks_per_seq * block_size must be < 2^31");
  if (free_queue == nullptr || queue_state == nullptr || queue_state_out == nullptr || query_start == nullptr)
    return fail(PA_ERR_INVALID_ARG, "NULL pointer");
  if (num_seqs > 0 && (block_tables == nullptr || context_lens == nullptr || new_lens == nullptr ||
                       context_lens_out == nullptr))
    return fail(PA_ERR_INVALID_ARG, "NULL pointer");
  if (max_tokens > 0 && (positions == nullptr || slot_mapping == nullptr))
    return fail(PA_ERR_INVALID_ARG, "NULL positions or slot_mapping");
  if ((reinterpret_cast<uintptr_t>(positions) & 15u) != 0 || (reinterpret_cast<uintptr_t>(slot_mapping) & 15u) != 0)
    return fail(PA_ERR_INVALID_ARG, "positions and slot_mapping must be 16-byte aligned");
  // Every CTA reads the lengths and the queue's state while others write the
  // outputs, so none of them may share memory.
  const size_t nb = static_cast<size_t>(num_seqs) * 4;
  struct Range {
    const void* p;
    size_t n;
  };
  const Range ins[] = {{context_lens, nb}, {new_lens, nb}, {queue_state, 8}};
  const Range outs[] = {{context_lens_out, nb},
                        {query_start, nb + 4},
                        {positions, static_cast<size_t>(max_tokens) * 4},
                        {slot_mapping, static_cast<size_t>(max_tokens) * 8},
                        {queue_state_out, 8},
                        {free_queue, static_cast<size_t>(num_blocks) * 4},
                        {block_tables, static_cast<size_t>(num_seqs) * max_blocks_per_seq * 4}};
  for (size_t i = 0; i < sizeof(outs) / sizeof(outs[0]); ++i) {
    for (const Range& r : ins)
      if (r.n > 0 && outs[i].n > 0 && overlap(r.p, r.n, outs[i].p, outs[i].n))
        return fail(PA_ERR_INVALID_ARG, "an output shares memory with context_lens, new_lens or queue_state");
    for (size_t j = i + 1; j < sizeof(outs) / sizeof(outs[0]); ++j)
      if (outs[i].n > 0 && outs[j].n > 0 && overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
        return fail(PA_ERR_INVALID_ARG, "two outputs share memory");
  }
  ExtendArgs a{block_tables, context_lens, new_lens, free_queue, queue_state, num_seqs,
               max_blocks_per_seq, block_size, num_blocks, max_tokens, context_lens_out, query_start,
               positions, slot_mapping, queue_state_out, dev_err};
  // Four tokens a thread; enough CTAs for the new blocks of a batch without
  // tokens as well. At most two CTAs per SM: each repeats the prefix sums
  // (four take 12.8 us instead of 11.7 for 512 sequences with 465,000 tokens).
  const int64_t work = std::max<int64_t>((static_cast<int64_t>(max_tokens) + 3) / 4, num_seqs);
  const int grid = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((work + kExtThreads - 1) / kExtThreads, 2 * sm_count())));
  const size_t smem = (static_cast<size_t>(num_seqs) * 4 + 2) * sizeof(int);
  // Without the opt-in dynamic and static shared memory (some 200 bytes here)
  // together may take 48 KB.
  constexpr size_t kStaticRoom = 1024;
  if (smem + kStaticRoom > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(extend_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>((kExtMaxSeqs * 4 + 2) * sizeof(int)));
    if (e != cudaSuccess) return fail(PA_ERR_CUDA, "extend_tables: %s", cudaGetErrorString(e));
  }
  extend_tables_kernel<<<grid, kExtThreads, smem, static_cast<cudaStream_t>(stream)>>>(a);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return fail(PA_ERR_CUDA, "extend_tables launch: %s", cudaGetErrorString(err));
  return ok();
}
