// Instances of the 4-bit decode kernel (bf16 queries, groups 1..16).
#include <cstdlib>
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

template <int BS>
static bool pick(int head_dim, DecodeInstance* out) {
  if (head_dim == 64) { *out = make_q4<BS, 64, 12, 4, 4>(); return true; }
  if (head_dim == 128) {
    const char* e = std::getenv("Q4SHAPE");
    const int v = e ? std::atoi(e) : 0;
    if constexpr (BS == 16) {
    if (v == 1) { *out = make_q4<BS, 128, 8, 4, 4>(); return true; }
    if (v == 2) { *out = make_q4<BS, 128, 12, 3, 4>(); return true; }
    if (v == 3) { *out = make_q4<BS, 128, 12, 3, 3>(); return true; }
    if (v == 4) { *out = make_q4<BS, 128, 8, 4, 3>(); return true; }
    if (v == 5) { *out = make_q4<BS, 128, 12, 2, 4>(); return true; }
    }
    *out = make_q4<BS, 128, 12, 4, 3>(); return true; }
  if (head_dim == 256) { *out = make_q4<BS, 256, 8, 2, 4>(); return true; }
  return false;
}

bool find_decode_q4(int head_dim, int block_size, DecodeInstance* out) {
  if (block_size == 16) return pick<16>(head_dim, out);
  if (block_size == 32) return pick<32>(head_dim, out);
  return false;
}

}  // namespace pagedkv
