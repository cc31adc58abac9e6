// Layout and arithmetic of the 4-bit KV cache, shared by its append, read
// and attention kernels (the layout is specified in include/pagedkv.h).
//
// A (block, KV head) tile of one pool is block_size / 16 sub-tiles of 16
// tokens. A sub-tile is 16 code rows of D / 2 bytes, then 16 x (D / 64)
// pairs (scale, minimum) in bf16: 9 D bytes in all, contiguous, a multiple
// of 16 bytes, so that the attention kernel moves one sub-tile with one bulk
// copy. Eight consecutive dims (8-aligned) of a token are one 32-bit word
// of eight codes, the lowest dim in the lowest nibble; the words of a row
// stand in the order in which the attention kernel's lanes read them:
//   K: a lane of quarter t = (d >> 4) & 3 takes the dims 16 t .. 16 t + 15 of
//      every 64-dim group, so each quarter's words are adjacent;
//   V: a lane of octet g = (d >> 3) & 7 takes the dims 8 g .. 8 g + 7 of every
//      group, so each octet's words are adjacent; octets are permuted by the
//      token so that the eight rows that a warp reads together lie in
//      different shared-memory banks (the K rows of head_dim 256 likewise).
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

namespace pagedkv {

template <int D>
struct Q4Geo {
  static_assert(D == 64 || D == 128 || D == 256, "head_dim 64, 128 or 256");
  static constexpr int kGroups = D / 64;            // (scale, min) pairs per token
  static constexpr int kRowBytes = D / 2;           // codes of one token
  static constexpr int kCodeBytes = 16 * kRowBytes; // codes of one sub-tile
  static constexpr int kParamRow = kGroups * 4;     // (scale, min) of one token
  static constexpr int kSubBytes = 9 * D;           // one sub-tile
  static_assert(kCodeBytes + 16 * kParamRow == kSubBytes && kSubBytes % 16 == 0, "sub-tile size");

  // Byte offset in a token's code row of the word of dims 8 c .. 8 c + 7.
  __host__ __device__ static constexpr int k_word(int tok, int c) {
    const int grp = c >> 3, t = (c >> 1) & 3, w = 2 * grp + (c & 1);
    if (D == 64) return t * 8 + w * 4;
    const int panel = (w >> 2) ^ (D == 256 ? (tok & 1) : 0);
    return panel * 64 + t * 16 + (w & 3) * 4;
  }
  __host__ __device__ static constexpr int v_turn(int tok) {
    return D == 64 ? 0 : D == 128 ? 4 * ((tok >> 1) & 1) : 2 * (tok & 3);
  }
  __host__ __device__ static constexpr int v_word(int tok, int c) {
    const int grp = c >> 3, g = c & 7;
    return (g ^ v_turn(tok)) * (D / 16) + grp * 4;
  }
  template <bool kValue>
  __host__ __device__ static constexpr int word(int tok, int c) {
    return kValue ? v_word(tok, c) : k_word(tok, c);
  }
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace pagedkv
