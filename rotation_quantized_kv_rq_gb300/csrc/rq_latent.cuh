// The cache of latents (storage contract: include/rq.h): where a token's bytes stand.
//
// A page is four planes of codes (128 dims each), a plane of position parts and the exponent bytes, P rows of 128 bytes
// to a plane.  A row's 16-byte chunks stand at chunk ^ (row % 8): eight rows are as they stand an operand of the tensor
// cores with the 128-byte swizzle, for scores (a row a token, K along dims) and for the weighted sum (N along dims, K along
// tokens) alike, so a bulk copy brings operands and nothing is rearranged or widened.
#pragma once

#include <stdint.h>

#include "rq_internal.h"

namespace rq {
namespace latent {

constexpr int kNanExp = 255;  // exponent byte of a token that reads as NaN

// Byte of 16-byte chunk `chunk` (0 to 7) of row r in a plane.
__device__ __forceinline__ uint32_t chunk_at(int r, int chunk) {
  return (uint32_t)(r * 128 + ((chunk ^ (r & 7)) << 4));
}
__device__ __forceinline__ size_t page_at(int page, int page_size) {
  return (size_t)page * (uint32_t)(page_size * kLatentTokenBytes);
}
// 2^E of an exponent byte; NaN for byte 255, other bytes brought into the range of scales.
__device__ __forceinline__ float scale_of_byte(uint32_t byte) {
  const int e = min(max((int)byte - 127, kMinExp), kMaxExp);
  return __uint_as_float(byte == kNanExp ? 0x7FFFFFFFu : (uint32_t)(e + 127) << 23);
}

}  // namespace latent
}  // namespace rq
