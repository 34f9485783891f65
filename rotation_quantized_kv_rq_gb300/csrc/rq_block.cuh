// The 8-bit block-scaled cache (storage contract: include/rq.h): where a block's bytes stand, and
// the conversions between e4m3 codes and wider types.
//
// A block is 16 tokens of one kv head, 4112 bytes, so that one bulk copy brings a whole tile of the
// attention kernels: 16 is the M of their MMA over tokens and the K of their MMA over values.  Its
// byte order is the order of those MMAs' A fragments: with lane = 4 g + t, the 16 bytes at 16 *
// (32 u + lane) are all lane's, so every read of a tile is 16 contiguous bytes a lane, free of bank
// conflicts, and needs no rearranging.
//   keys,   unit u = 2 (r / 8) + d / 64: token r = 8 (u / 2) + g, dims 64 (u % 2) + 16 t .. + 15
//   values, unit u: dims 32 u + 4 g .. + 3, four bytes each: tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "rq_internal.h"

namespace rq {
namespace block {

constexpr int kValues = 2048;  // offset of the value codes
constexpr int kExps = 4096;    // the key scale's exponent byte, then the value scale's

// Two e4m3 codes (low byte first) as fp16, exactly.
__device__ __forceinline__ uint32_t widen2(uint32_t codes) {
  uint32_t h;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(h) : "r"(codes));
  return h;
}
__device__ __forceinline__ uint32_t widen2_hi(uint32_t codes) {
  uint32_t h;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}" : "=r"(h) : "r"(codes));
  return h;
}
// Four f32 to e4m3 codes, x0 in the low byte: round to nearest even, past 448 to 448, NaN to NaN.
__device__ __forceinline__ uint32_t code4(float x0, float x1, float x2, float x3) {
  uint32_t w;
  asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
      " mov.b32 %0, {lo, hi};\n}"
      : "=r"(w)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return w;
}
// Four codes times 2^-shift (1 <= shift), rounded to codes again.  The product is exact in fp16
// down to 2^-24; below that both round to zero.
__device__ __forceinline__ uint32_t shrink4(uint32_t codes, int shift) {
  const __half2 s = __half2half2(__float2half_rn(exp2f((float)-shift)));  // 0 past 2^-24
  uint32_t a = widen2(codes), b = widen2_hi(codes), w;
  __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&a), s), y = __hmul2(*reinterpret_cast<const __half2*>(&b), s);
  a = *reinterpret_cast<const uint32_t*>(&x), b = *reinterpret_cast<const uint32_t*>(&y);
  asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f16x2 lo, %1;\n cvt.rn.satfinite.e4m3x2.f16x2 hi, %2;\n"
      " mov.b32 %0, {lo, hi};\n}"
      : "=r"(w)
      : "r"(a), "r"(b));
  return w;
}

// The scale's exponent for a largest magnitude `amax` (finite): the smallest E with amax <= 448 *
// 2^E, 448 = 1.75 * 2^8, read off amax's own bits; subnormal amax (and 0) get the smallest scale.
__device__ __forceinline__ int exp_of(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kMinExp), kMaxExp);
}
// A stored exponent byte; any byte is brought into the range of scales.
__device__ __forceinline__ int exp_of_byte(uint32_t byte) { return min(max((int)byte - 127, kMinExp), kMaxExp); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }  // |e| <= 126

// The softmax weights, rounded to fp16 for their product with the values: 2^(score + EV - m), where m is a
// running maximum of score + EV less kLift, moved where a score is past it by more than kReach.  So the largest
// weight of a row stands between 2^kLift and 2^kReach, near the top of fp16's range, and its smallest steps,
// 2^-24, are 2^-31 of it or less: a token below half of that is lost from the product (not from the
// weights' sum), at most 2^-32 of the largest, 2^-12 for 2^20 such tokens, where the largest itself is rounded
// by up to 2^-11.
constexpr float kLift = 7.f, kReach = 15.f;  // (a maximum of 2^26 and more, 8 apart, gives a lift of 8 or 0)
constexpr float kNone = -3.402823466e38f;    // m before any visible token: no finite score is below

// A query row as an fp16 operand is the row times `down`; its scores are the products times `factor` times a
// block's key scale.  A bf16 row is brought by a power of two to a largest magnitude `top` of 2^14 .. 2^15, an
// fp16 row (BF16 false) is taken as it is; sm: the softmax scale times log2(e).
// factor is at least 2^-66, so that with a key scale (2^-60 at least) it stays above 0 in f32: a score that the
// mask made minus infinity has to stay that, and a row of zeros over keys of zeros would come to -inf * 0.
// For smaller rows the operand is smaller instead.  It is then off by 2^-25 at most, which moves a score by
// 2^-25 * 448 * 128 * 2^-65 * 2^60 < 2^-14 at the largest key scale there is (2^60), 2^-66 at 2^8.
// (An fp16 row meets the bound only below sm = 2^-66, where its scores come to 2^-26 at most either way.)
struct RowScale {
  float down, factor;
};
template <bool BF16>
__device__ __forceinline__ RowScale row_scale(float top, float sm) {
  constexpr int kLeast = -66;
  RowScale r{1.f, sm};
  if (BF16) {
    const int least = kLeast + 14 + 127 - (int)(__float_as_uint(sm) >> 23);
    const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, max(least, -100)), 127);
    r.down = pow2(14 - e);
    r.factor *= pow2(e - 14);
  }
  r.factor = fmaxf(r.factor, pow2(kLeast));
  return r;
}

}  // namespace block
}  // namespace rq
