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

// Two f32 values in one 64-bit register pair and two operations in one instruction (half the issue
// slots at the same rate).  A lane's eight values stay in four such pairs throughout: packing and
// unpacking around single operations would cost more moves than it saves.
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
  // quarter turns, and what is left of one (|left| <= 1/8 turn) before the rounding to 24 bits: an
  // angle of half a turn rounded as it is would be off by 9e-8 rad, a third of all the f32 error here
  const int32_t frac = (int32_t)((turns + 0x80000000ull) >> 32);  // signed fraction of a turn, * 2^32
  const uint32_t quarter = ((uint32_t)frac + 0x20000000u) >> 30;
  const int32_t left = (int32_t)((uint32_t)frac - (quarter << 30));
  float s, c;
  sincospif((float)left * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
  if (quarter & 1) {  // (c, s) turned by a quarter: (-s, c)
    const float t = c;
    c = -s;
    s = t;
  }
  if (quarter & 2) c = -c, s = -s;
  return make_float2(c * r.scale, s * r.scale);
}
// Cosines, sines and negated sines of the lane's pairs, two to a word.
struct Angles {
  uint64_t c[2], s[2], n[2];
};
__device__ __forceinline__ Angles angles_of(const float4& c, const float4& s) {
  Angles a;
  a.c[0] = f2(c.x, c.y), a.c[1] = f2(c.z, c.w);
  a.s[0] = f2(s.x, s.y), a.s[1] = f2(s.z, s.w);
  a.n[0] = f2(-s.x, -s.y), a.n[1] = f2(-s.z, -s.w);
  return a;
}
__device__ __forceinline__ void cos_sin4(float4& c, float4& s, const RopeTable& r, int p, const int32_t* positions,
                                         long long n, long long t) {
  const float2 a0 = cos_sin(r, p, positions, n, t), a1 = cos_sin(r, p + 1, positions, n, t);
  const float2 a2 = cos_sin(r, p + 2, positions, n, t), a3 = cos_sin(r, p + 3, positions, n, t);
  c = make_float4(a0.x, a1.x, a2.x, a3.x);
  s = make_float4(a0.y, a1.y, a2.y, a3.y);
}

template <typename T>
__device__ __forceinline__ void load8(uint2 (&raw)[2], const T* row, const Lane& l) {
  raw[0] = *reinterpret_cast<const uint2*>(row + l.o0);  // plain loads: the row may be written in place
  raw[1] = *reinterpret_cast<const uint2*>(row + l.o1);
}
// The lane's eight values: dims (o0, o0 + 1), (o0 + 2, o0 + 3), (o1, o1 + 1), (o1 + 2, o1 + 3).
template <typename T>
__device__ __forceinline__ void widen8(uint64_t (&x)[4], const uint2 (&raw)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = unpack2<T>(raw[i].x), b = unpack2<T>(raw[i].y);
    x[2 * i] = f2(a.x, a.y);
    x[2 * i + 1] = f2(b.x, b.y);
  }
}

// 1 / sqrt(mean(x^2) + eps) of the row.  All lanes of the half-warp call it.
__device__ __forceinline__ float inv_rms(const uint64_t (&x)[4], float eps) {
  uint64_t s2 = mul2(x[0], x[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s2 = fma2(x[i], x[i], s2);
  float ss, hi;
  split2(s2, ss, hi);
  ss += hi;
  const uint32_t mask = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
  return __frsqrt_rn(fmaf(ss, 1.f / kHeadDim, eps));
}
// The lane's eight weights.
__device__ __forceinline__ void load_weights(uint64_t (&w)[4], const float* weight, const Lane& l) {
  const float4 w0 = __ldg(reinterpret_cast<const float4*>(weight + l.o0));
  const float4 w1 = __ldg(reinterpret_cast<const float4*>(weight + l.o1));
  w[0] = f2(w0.x, w0.y), w[1] = f2(w0.z, w0.w), w[2] = f2(w1.x, w1.y), w[3] = f2(w1.z, w1.w);
}
__device__ __forceinline__ void scale8(uint64_t (&x)[4], float r, const uint64_t (&w)[4]) {
  const uint64_t r2 = f2(r, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = mul2(x[i], mul2(r2, w[i]));
}

// Turns the lane's four pairs.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn8(uint64_t (&x)[4], const Angles& a, const Lane& l) {
  if (l.pair < 0) return;
  if (INTERLEAVED) {  // pair i = x[i]
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float u, v, c0, c1, s0, s1;
      split2(x[i], u, v);
      split2(a.c[i >> 1], c0, c1);
      split2(a.s[i >> 1], s0, s1);
      const float c = i & 1 ? c1 : c0, s = i & 1 ? s1 : s0;
      x[i] = f2(u * c - v * s, u * s + v * c);
    }
  } else {  // pair 2 i + k = (half k of x[i], half k of x[i + 2])
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint64_t u = x[i], v = x[i + 2];
      x[i] = fma2(u, a.c[i], mul2(v, a.n[i]));
      x[i + 2] = fma2(u, a.s[i], mul2(v, a.c[i]));
    }
  }
}

template <typename T>
__device__ __forceinline__ uint32_t narrow2(uint64_t x) {
  float lo, hi;
  split2(x, lo, hi);
  return pack2<T>(lo, hi);
}
template <typename T>
__device__ __forceinline__ void store8(T* row, const uint64_t (&x)[4], const Lane& l) {
  *reinterpret_cast<uint2*>(row + l.o0) = make_uint2(narrow2<T>(x[0]), narrow2<T>(x[1]));
  *reinterpret_cast<uint2*>(row + l.o1) = make_uint2(narrow2<T>(x[2]), narrow2<T>(x[3]));
}

// Heads first, first + step, ... of one token's rows at src to dst: norm (weight: the norm's, null for
// none) and rotation.  Loads of four rows are in flight together.  In place is safe: a row is read by
// the half-warp that writes it, before it writes.
template <typename T, bool INTERLEAVED>
__device__ __forceinline__ void turn_rows(const T* src, T* dst, int first, int step, int heads, const float* weight,
                                          float eps, const Angles& cs, const Lane& l) {
  constexpr int kBatch = 4;
  if (first >= heads) return;
  uint64_t w[4];
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
      uint64_t x[4];
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
