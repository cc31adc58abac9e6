// Instances of the 4-bit decode kernel (bf16 queries, groups 1..16).
#include "decode_dispatch.h"
#include "decode_q4_kernel.cuh"

namespace pagedkv {

template <int BS, int D, int W, int US, int NS>
static DecodeInstance make_q4() {
  using Cfg = Q4Cfg<BS, D, W, US, NS>;
  DecodeInstance r;
  r.kernel = reinterpret_cast<const void*>(&paged_decode_q4_kernel<Cfg>);
  r.merge = reinterpret_cast<const void*>(&lse_merge_kernel<__nv_bfloat16, D>);
  r.threads = Cfg::kThreads;
  r.fixed_smem = Cfg::kFixedSmem;
  r.stages = Cfg::NS;
  r.warps = Cfg::W;
  r.launch_regs = Cfg::kLaunchRegs;
  r.name = "mma_q4";
  return r;
}

// Consumer warps x units a step x ring slots (of a step's K or V). Measured at
// head_dim 128 on 8 x 131072 tokens / 256 ragged sequences, before the lists'
// padding: 12 x 4 x 3 260 / 107 us; 12 x 3 x 4 275 / 109; 8 x 4 x 4 274 / 112;
// 12 x 2 x 4 307 / 124 (per-step work over fewer units). A fourth slot gains
// 1.5% and leaves no room for the lists of 4096 sequences.
// head_dim 64, where a unit is half the bytes, so steps of more units carry the
// per-step work: 12 x 8 x 3 155 / 66 us; 12 x 6 x 4 162 / 68; 12 x 4 x 4 186 /
// 75; 12 x 4 x 6 185 / 75.
// head_dim 256 needs 232 registers, so 8 warps; 4 x 131072 / 128 ragged:
// 8 x 3 x 3 248 / 98 us; 8 x 2 x 4 258 / 105; 8 x 2 x 3 261 / 104; 8 x 4 x 2
// 250 / 106 (and it spills).
// (All with one power of two for the value scales; one for each group costs 1 to
// 2%: 249 / 97 us at head_dim 128, 157 / 66 at 64, 253 / 100 at 256.)
template <int BS>
static bool pick(int head_dim, DecodeInstance* out) {
  if (head_dim == 64) { *out = make_q4<BS, 64, 12, 8, 3>(); return true; }
  if (head_dim == 128) { *out = make_q4<BS, 128, 12, 4, 3>(); return true; }
  if (head_dim == 256) { *out = make_q4<BS, 256, 8, 3, 3>(); return true; }
  return false;
}

bool find_decode_q4(int head_dim, int block_size, DecodeInstance* out) {
  if (block_size == 16) return pick<16>(head_dim, out);
  if (block_size == 32) return pick<32>(head_dim, out);
  return false;
}

}  // namespace pagedkv
