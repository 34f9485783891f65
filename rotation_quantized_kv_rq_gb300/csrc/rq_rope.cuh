// Per-head norms and position rotation of query and key rows: device code shared by the pass over
// queries and keys (rq_rope.cu) and the 8-bit append that applies it on the way
// (rq_block_append.cu).
//
// A row (one token, one head) of 128 values is held by a half-warp: lane j holds two runs of four
// dims, o0 .. o0 + 3 and o1 .. o1 + 3, chosen so that both values of its four rotation pairs are
// its own (no exchange) and both runs are aligned 8-byte loads that a half-warp makes whole
// 32-byte sectors of.
//   y = x / sqrt(mean(x^2) + eps) * w                      (in f32; the sum over the half-warp)
//   (a, b) -> scale * (a cos t - b sin t, a sin t + b cos t),   t = position * frequency
// The angle: a frequency is kept as its fraction of a turn in 64 fixed-point bits, f / (2 pi) *
// 2^64, and position * that, modulo 2^64, is the angle's fraction of a turn: the wrap of the
// integer product is the range reduction, exact at every position (|error| <= |position| * 2^-65
// turns, 2^-34 at 2^31), where position * frequency in f32 would be off by 0.06 rad at 2^20.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "rq_internal.h"

namespace rq {
namespace rope {

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two f32 operations in one instruction (half the issue slots; the rate is the same).
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void split2(uint64_t d, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(d));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Where lane j of a half-warp stands in a row.
struct Lane {
  int o0, o1;  // its two runs of four dims
  int pair;    // its four pairs: pair .. pair + 3, or -1 (dims past rotary_dim)
};
template <bool INTERLEAVED>
__device__ __forceinline__ Lane lane_of(int j, int rotary_dim) {
  Lane l;
  const int half = rotary_dim >> 1, p = 4 * j;
  if (INTERLEAVED) {  // pairs (2i, 2i + 1)
    l.o0 = 8 * j;
    l.o1 = 8 * j + 4;
  } else if (p < half) {  // pairs (i, i + rotary_dim / 2)
    l.o0 = p;
    l.o1 = p + half;
  } else {
    l.o0 = rotary_dim + 2 * (p - half);
    l.o1 = l.o0 + 4;
  }
  l.pair = p < half ? p : -1;
  return l;
}

// cos and sin (times the rotation's scale) of pair p at token t.
__device__ __forceinline__ float2 cos_sin(const RopeTable& r, int p, const int32_t* positions, long long n,
                                          long long t) {
  const ulonglong2 e = __ldg(reinterpret_cast<const ulonglong2*>(r.pairs) + p);  // (turns per position, axis)
  const int32_t pos = __ldg(positions + (long long)e.y * n + t);
  const uint64_t turns = (uint64_t)(int64_t)pos * e.x;
  const int32_t frac = (int32_t)((turns + 0x80000000ull) >> 32);  // signed fraction of a turn, * 2^32
  float s, c;
  sincospif((float)frac * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
  return make_float2(c * r.scale, s * r.scale);
}

template <typename T>
__device__ __forceinline__ void load8(uint2 (&raw)[2], const T* row, const Lane& l) {
  raw[0] = *reinterpret_cast<const uint2*>(row + l.o0);  // plain loads: the row may be written in place
  raw[1] = *reinterpret_cast<const uint2*>(row + l.o1);
}
template <typename T>
__device__ __forceinline__ void widen8(float (&x)[8], const uint2 (&raw)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = unpack2<T>(raw[i].x), b = unpack2<T>(raw[i].y);
    x[4 * i] = a.x, x[4 * i + 1] = a.y, x[4 * i + 2] = b.x, x[4 * i + 3] = b.y;
  }
}

// 1 / sqrt(mean(x^2) + eps) of the row.  All lanes of the half-warp call it.
__device__ __forceinline__ float inv_rms(const float (&x)[8], float eps) {
  uint64_t s2 = 0ull;
#pragma unroll
  for (int i = 0; i < 8; i += 2) s2 = fma2(f2(x[i], x[i + 1]), f2(x[i], x[i + 1]), s2);
  float ss, hi;
  split2(s2, ss, hi);
  ss += hi;
  const uint32_t mask = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
  return __frsqrt_rn(fmaf(ss, 1.f / kHeadDim, eps));
}
// The lane's eight weights.
__device__ __forceinline__ void load_weights(float (&w)[8], const float* weight, const Lane& l) {
  const float4 w0 = __ldg(reinterpret_cast<const float4*>(weight + l.o0));
  const float4 w1 = __ldg(reinterpret_cast<const float4*>(weight + l.o1));
  w[0] = w0.x, w[1] = w0.y, w[2] = w0.z, w[3] = w0.w, w[4] = w1.x, w[5] = w1.y, w[6] = w1.z, w[7] = w1.w;
}
__device__ __forceinline__ void scale8(float (&x)[8], float r, const float (&w)[8]) {
  const uint64_t r2 = f2(r, r);
#pragma unroll
  for (int i = 0; i < 8; i += 2) split2(mul2(f2(x[i], x[i + 1]), mul2(r2, f2(w[i], w[i + 1]))), x[i], x[i + 1]);
}

// Turns the lane's four pairs; cs[i] = (cos, sin) of pair l.pair + i.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn8(float (&x)[8], const float2 (&cs)[4], const Lane& l) {
  if (l.pair < 0) return;
  if (INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = x[2 * i], v = x[2 * i + 1];
      x[2 * i] = u * cs[i].x - v * cs[i].y;
      x[2 * i + 1] = u * cs[i].y + v * cs[i].x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint64_t c = f2(cs[i].x, cs[i + 1].x), s = f2(cs[i].y, cs[i + 1].y), ns = f2(-cs[i].y, -cs[i + 1].y);
      const uint64_t u = f2(x[i], x[i + 1]), v = f2(x[4 + i], x[5 + i]);
      split2(fma2(u, c, mul2(v, ns)), x[i], x[i + 1]);
      split2(fma2(u, s, mul2(v, c)), x[4 + i], x[5 + i]);
    }
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* row, const float (&x)[8], const Lane& l) {
  *reinterpret_cast<uint2*>(row + l.o0) = make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]));
  *reinterpret_cast<uint2*>(row + l.o1) = make_uint2(pack2<T>(x[4], x[5]), pack2<T>(x[6], x[7]));
}

// Heads first, first + step, ... of one token's rows at src to dst: norm (weight: the norm's, null for
// none) and rotation.  Loads of four rows are in flight together.  In place is safe: a row is read by
// the half-warp that writes it, before it writes.
template <typename T, bool INTERLEAVED>
__device__ __forceinline__ void turn_rows(const T* src, T* dst, int first, int step, int heads, const float* weight,
                                          float eps, const float2 (&cs)[4], const Lane& l) {
  constexpr int kBatch = 4;
  if (first >= heads) return;
  float w[8];
  if (weight) load_weights(w, weight, l);
  src += first * kHeadDim;
  dst += first * kHeadDim;
  const int stride = step * kHeadDim;
  for (int left = (heads - first + step - 1) / step; left > 0; left -= kBatch) {
    uint2 raw[kBatch][2];
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (u < left) load8(raw[u], src + u * stride, l);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (u >= left) break;
      float x[8];
      widen8<T>(x, raw[u]);
      if (weight) scale8(x, inv_rms(x, eps), w);
      turn8<INTERLEAVED>(x, cs, l);
      store8(dst + u * stride, x, l);
    }
    src += kBatch * stride;
    dst += kBatch * stride;
  }
}

}  // namespace rope
}  // namespace rq
