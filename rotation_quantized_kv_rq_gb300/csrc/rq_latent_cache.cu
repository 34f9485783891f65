// Append to the cache of latents, with the latent's norm and the position rotation on the way and the same tokens'
// queries turned in the same launch, and reading the cache back.
//
// append: y = c / sqrt(mean c^2 + eps) w, p = rot(k_pe), E the least exponent with |y| <= 448 2^E and |p| <= 2^15 2^E; codes
// e4m3(y 2^-E), parts p 2^-E in 16 bits.  A row is a warp's, 16 dims to a lane, so that sums and maxima stay in it and a token's
// bytes are written by one warp.  In long calls the warp turns the token's queries too, with the angles it has; in short ones
// they have warps of their own (64 tokens x 128 heads: 2.8 us, a chain of latencies).  32,768 tokens x 16 heads: 44 us, 4.4 TB/s, 66%
// of the copy rate: 69% of the issue slots are taken, and what stalls the rest first are the loads.
// read: a warp takes four rows, whose bytes are in flight together: 16 x 1K-16K tokens in 44 us, 5.7 TB/s, 85%; 1,500 in 3.2.
#include "../../include/rq.h"
#include "rq_block.cuh"
#include "rq_latent.cuh"
#include "rq_rope.cuh"

namespace rq {
namespace {

using namespace rope;
using namespace latent;

constexpr int kThreads = 256;
constexpr uint32_t kInf = 0x7F800000u;
constexpr uint32_t kMostCode = (kMaxExp + 8 + 127) << 23 | 0x600000u;  // 448 * 2^kMaxExp
constexpr uint32_t kMostPart = (uint32_t)(kMaxExp + 15 + 127) << 23;   // 2^15 * 2^kMaxExp

// The smallest E with top <= 2^(15 + E), within the range of scales.
__device__ __forceinline__ int exp_of_part(float top) {
  const uint32_t b = __float_as_uint(top);
  return min(max((int)(b >> 23) - 127 - 15 + ((b & 0x7FFFFFu) != 0u ? 1 : 0), kMinExp), kMaxExp);
}

// A position part, 64 dims, is held by a half-warp, lane j dims 4j .. 4j + 3.  Pairs (2i, 2i + 1) are a lane's own; of
// pairs (i, i + rotary_dim / 2) the other half is rotary_dim / 8 lanes away.
struct Turn {
  float c[4], s[4];  // of the pair of each of the four dims; s negated where the dim is a pair's first
  int other;         // lane of the half-warp that holds the other halves; -1: past rotary_dim
};
// All lanes of the warp call it: lane l computes pair l's cosine and sine, and takes those of its own pairs from others.
template <bool INTERLEAVED>
__device__ __forceinline__ Turn turn_of(const RopeTable& r, int lane, const int32_t* positions, long long n, long long t) {
  const int j = lane & 15;
  float2 mine = make_float2(1.f, 0.f);
  if (2 * lane < r.rotary_dim) mine = cos_sin(r, lane, positions, n, t);
  const int away = r.rotary_dim >> 3;
  const bool turns = 4 * j < r.rotary_dim, first = INTERLEAVED || j < away;
  Turn u;
  u.other = !turns ? -1 : INTERLEAVED ? j : first ? j + away : j - away;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int pair = INTERLEAVED ? 2 * j + (i >> 1) : 4 * (first ? j : j - away) + i;
    u.c[i] = __shfl_sync(0xffffffffu, mine.x, pair & 31);
    const float sn = __shfl_sync(0xffffffffu, mine.y, pair & 31);
    u.s[i] = (INTERLEAVED ? (i & 1) == 0 : first) ? -sn : sn;
  }
  return u;
}
// All lanes of the warp call it.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn4(float (&x)[4], const Turn& u) {
  float y[4];
  if (INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = x[i ^ 1];
  } else {
    const int from = (threadIdx.x & 16) | (u.other < 0 ? (threadIdx.x & 15) : u.other);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], from);
  }
  if (u.other < 0) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = fmaf(y[i], u.s[i], x[i] * u.c[i]);
}

// s += x; returns what the rounding leaves.
__device__ __forceinline__ float plus(float& s, float x) {
  const float sum = s + x, of_x = sum - s, left = (s - (sum - of_x)) + (x - of_x);
  s = sum;
  return left;
}

// Two sums; `left` gathers what the roundings leave.
__device__ __forceinline__ void plus2(uint64_t& s, uint64_t x, uint64_t& left) {
  asm("{\n .reg .b64 sum, of_x, of_s, a, b;\n add.rn.f32x2 sum, %0, %2;\n sub.rn.f32x2 of_x, sum, %0;\n sub.rn.f32x2 of_s, sum, of_x;\n"
      " sub.rn.f32x2 a, %0, of_s;\n sub.rn.f32x2 b, %2, of_x;\n add.rn.f32x2 a, a, b;\n add.rn.f32x2 %1, %1, a;\n mov.b64 %0, sum;\n}"
      : "+l"(s), "+l"(left)
      : "l"(x));
}

template <typename T>
__device__ __forceinline__ void widen4(float (&x)[4], const uint2& w) {
  const float2 a = unpack2<T>(w.x), b = unpack2<T>(w.y);
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}

// Queries of heads first .. last - 1 of token t, two heads to the warp at a time.
template <typename T, bool INTERLEAVED>
__device__ __forceinline__ void turn_heads(const LatentAppendArgs& a, long long t, int first, int last, const Turn& u) {
  const int j = threadIdx.x & 15, half = threadIdx.x >> 4 & 1;
  const T* src = reinterpret_cast<const T*>(a.q.x) + t * a.q.stride + 4 * j;
  T* dst = reinterpret_cast<T*>(const_cast<void*>(a.q_out.x)) + t * a.q_out.stride + 4 * j;
  constexpr int kBatch = 8;
  for (int h0 = first; h0 < last; h0 += 2 * kBatch) {
    uint2 raw[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + 2 * i + half;
      raw[i] = h < last ? *reinterpret_cast<const uint2*>(src + h * a.q.head_stride) : make_uint2(0u, 0u);  // (may be in place)
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (h0 + 2 * i >= last) break;
      const int h = h0 + 2 * i + half;
      float x[4];
      widen4<T>(x, raw[i]);
      turn4<INTERLEAVED>(x, u);
      if (h < last)
        *reinterpret_cast<uint2*>(dst + h * a.q_out.head_stride) = make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]));
    }
  }
}

// Warp (token, part): part 0 codes the token's latent and position part, part i turns queries of heads per * (i - 1) .. ; with
// one part, that warp turns all of them.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 4) latent_append_kernel(const LatentPool pool, const LatentAppendArgs a, int parts, int per) {
  const int lane = threadIdx.x & 31, j = lane & 15, half = lane >> 4;
  const long long w = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const long long t = parts == 1 ? w : w / parts;
  if (t >= a.n) return;
  const int part = (int)(w - t * parts);
  // a coding warp's rows are on their way while the angles are computed
  const int slot = part == 0 ? __ldg(a.slots + t) : -1;
  uint4 r0 = make_uint4(0u, 0u, 0u, 0u), r1 = r0;
  uint2 rp = make_uint2(0u, 0u);
  if (part == 0) {
    const uint4* row = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.c) + t * a.c_stride) + 2 * lane;
    r0 = __ldg(row), r1 = __ldg(row + 1);
    rp = __ldg(reinterpret_cast<const uint2*>(reinterpret_cast<const T*>(a.k_pe) + t * a.k_pe_stride) + j);
  }
  Turn u;
  u.other = -1;
  if (a.rope.rotary_dim > 0) u = turn_of<INTERLEAVED>(a.rope, lane, a.positions, a.n, t);
  if (part > 0) {
    turn_heads<T, INTERLEAVED>(a, t, (part - 1) * per, min(a.q.heads, part * per), u);
    return;
  }
  if (parts == 1) turn_heads<T, INTERLEAVED>(a, t, 0, a.q.heads, u);
  if (slot < 0) return;
  if (slot >= pool.num_pages * pool.page_size) {
    if (lane == 0 && a.status) atomicOr(a.status, RQ_STATUS_BAD_SLOT);
    return;
  }
  // the latent: 16 dims to a lane, one chunk of codes
  float x[16];
  {
    const uint32_t w8[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = unpack2<T>(w8[i]);
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  if (a.weight) {
    // The sum, the factor and the products with what their roundings leave, the last rounded to odd, so that a code moves only for a
    // value at the very middle of two: a step of 2^-4 multiplies what rounding moves.  Of 16.8 million codes none is off the
    // definition's; with plain float32 sums and products 3 to 17 were (41 us, with these 44).
    float ss, ss_lo;
    {
      uint64_t sum[2], left = 0ull;  // squares of values of 8 or 11 bits are exact
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t v = f2(x[2 * i], x[2 * i + 1]), q = mul2(v, v);
        if (i < 2)
          sum[i] = q;
        else
          plus2(sum[i & 1], q, left);
      }
      plus2(sum[0], sum[1], left);
      float other, other_lo;
      split2(sum[0], ss, other);
      split2(left, ss_lo, other_lo);
      ss_lo += other_lo + plus(ss, other);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float other = __shfl_xor_sync(0xffffffffu, ss, o), lo = __shfl_xor_sync(0xffffffffu, ss_lo, o);
      ss_lo = (ss_lo + lo) + plus(ss, other);
    }
    float m = ss * (1.f / kLatentDim);
    const float m_lo = fmaf(ss_lo, 1.f / kLatentDim, plus(m, a.eps)), r = __frsqrt_rn(m);
    const float mr = m * r, r_lo = 0.5f * r * (fmaf(-mr, r, 1.f) - fmaf(m, r, -mr) * r - m_lo * r * r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 w4 = __ldg(reinterpret_cast<const float4*>(a.weight) + 4 * lane + i);
      const float wt[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float y = x[4 * i + k] * wt[k], y_lo = fmaf(x[4 * i + k], wt[k], -y);
        // (the factor is a square root's: a product that is a float to the last bit is rare, and may go either way from a middle)
        x[4 * i + k] = __uint_as_float(__float_as_uint(__fmaf_rz(y, r, fmaf(y, r_lo, y_lo * r))) | 1u);
      }
    }
  }
  float p[4];
  widen4<T>(p, rp);
  turn4<INTERLEAVED>(p, u);
  uint32_t top_c = 0u, top_p = 0u;  // magnitudes order as their bits do, NaN above infinity above the rest
#pragma unroll
  for (int i = 0; i < 16; ++i) top_c = max(top_c, __float_as_uint(x[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int i = 0; i < 4; ++i) top_p = max(top_p, __float_as_uint(p[i]) & 0x7FFFFFFFu);
  top_c = __reduce_max_sync(0xffffffffu, top_c);
  top_p = __reduce_max_sync(0xffffffffu, top_p);
  const bool bad = max(top_c, top_p) >= kInf;
  if (lane == 0 && a.status) {
    const int fault = bad ? RQ_STATUS_NOT_FINITE : top_c > kMostCode || top_p > kMostPart ? RQ_STATUS_NORM_OVERFLOW : 0;
    if (fault) atomicOr(a.status, fault);
  }
  const int e = max(block::exp_of(__uint_as_float(top_c)), exp_of_part(__uint_as_float(top_p)));
  const float down = block::pow2(-e);
  uint4 codes = make_uint4(0u, 0u, 0u, 0u);
  uint2 pe = make_uint2(0u, 0u);
  if (!bad) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= down;
    codes = make_uint4(block::code4(x[0], x[1], x[2], x[3]), block::code4(x[4], x[5], x[6], x[7]),
                       block::code4(x[8], x[9], x[10], x[11]), block::code4(x[12], x[13], x[14], x[15]));
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = fminf(fmaxf(p[i] * down, -32768.f), 32768.f);
    pe = make_uint2(pack2<T>(p[0], p[1]), pack2<T>(p[2], p[3]));
  }
  const int P = pool.page_size, r = slot % P;
  uint8_t* const page = const_cast<uint8_t*>(pool.pages) + page_at(slot / P, P);
  *reinterpret_cast<uint4*>(page + (lane >> 3) * 128 * P + chunk_at(r, lane & 7)) = codes;
  if (half == 0) *reinterpret_cast<uint2*>(page + 512 * P + chunk_at(r, j >> 1) + 8 * (j & 1)) = pe;
  if (lane == 0) page[640 * P + r] = (uint8_t)(bad ? kNanExp : e + 127);
}

// A warp reads four rows: their sequences and pages are looked up by a lane each, then their bytes are in flight together.  (Eight,
// with half the warps: 48 us where four take 44.)
constexpr int kRows = 4;
template <typename T>
__global__ void __launch_bounds__(kThreads) latent_read_kernel(const LatentPool pool, const LatentReadArgs a) {
  const int lane = threadIdx.x & 31, P = pool.page_size;
  const long long row0 = (((long long)blockIdx.x * kThreads + threadIdx.x) >> 5) * kRows;
  if (row0 >= a.n) return;
  const uint8_t* at = nullptr;  // page of the lane's row, and the row's offset in it
  int r = 0;
  {
    const long long row = row0 + (lane & (kRows - 1));
    int lo = 0, hi = a.B - 1;  // the last sequence that starts at or before the row
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(a.offsets + mid) <= row) lo = mid; else hi = mid - 1;
    }
    const long long first = __ldg(a.offsets + lo), end = __ldg(a.offsets + lo + 1);
    if (row < a.n && row >= first && row < end) {
      const long long pos = (a.starts ? (long long)__ldg(a.starts + lo) : 0) + (row - first);
      int fault = 0;
      if (pos < 0 || pos >= (long long)a.max_pages * P || first < 0) {
        fault = RQ_STATUS_BAD_LEN;
      } else {
        const int page = __ldg(a.block_table + (size_t)lo * a.max_pages + pos / P);
        r = (int)(pos % P);
        if (page < 0 || page >= pool.num_pages)
          fault = RQ_STATUS_BAD_PAGE;
        else
          at = pool.pages + page_at(page, P);
      }
      if (fault && a.status) atomicOr(a.status, fault);
    }
  }
  uint4 code[kRows];
  float scale[kRows];
  uint32_t there = __ballot_sync(0xffffffffu, at != nullptr);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const uint8_t* page = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, (unsigned long long)at, i));
    const int ri = __shfl_sync(0xffffffffu, r, i);
    if (there >> i & 1) {
      code[i] = __ldg(reinterpret_cast<const uint4*>(page + (lane >> 3) * 128 * P + chunk_at(ri, lane & 7)));
      scale[i] = scale_of_byte(__ldg(page + 640 * P + ri));
    }
  }
  uint4 part[kRows / 4];  // four rows at a time, a chunk of eight values to a lane
#pragma unroll
  for (int i = 0; i < kRows; i += 4) {
    const int k = i + (lane >> 3);
    const uint8_t* page = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, (unsigned long long)at, k));
    const int rk = __shfl_sync(0xffffffffu, r, k);
    if (there >> k & 1) part[i / 4] = __ldg(reinterpret_cast<const uint4*>(page + 512 * P + chunk_at(rk, lane & 7)));
  }
  T* const c = reinterpret_cast<T*>(a.c);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (!(there >> i & 1)) continue;
    const uint32_t w[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
    uint32_t y[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 lo = unpack2<__half>(block::widen2(w[k])), hi = unpack2<__half>(block::widen2_hi(w[k]));
      y[2 * k] = pack2<T>(lo.x * scale[i], lo.y * scale[i]);
      y[2 * k + 1] = pack2<T>(hi.x * scale[i], hi.y * scale[i]);
    }
    uint4* dst = reinterpret_cast<uint4*>(c + (size_t)(row0 + i) * kLatentDim) + 2 * lane;
    dst[0] = make_uint4(y[0], y[1], y[2], y[3]);
    dst[1] = make_uint4(y[4], y[5], y[6], y[7]);
  }
#pragma unroll
  for (int i = 0; i < kRows; i += 4) {
    const int q4 = lane >> 3, k = i + q4;
    if (!(there >> k & 1)) continue;
    const float s = q4 < 2 ? (q4 == 0 ? scale[i] : scale[i + 1]) : (q4 == 2 ? scale[i + 2] : scale[i + 3]);
    const uint32_t w[4] = {part[i / 4].x, part[i / 4].y, part[i / 4].z, part[i / 4].w};
    uint32_t y[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 f = unpack2<T>(w[q]);
      y[q] = pack2<T>(f.x * s, f.y * s);
    }
    *reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.k_pe) + (size_t)(row0 + k) * kPositionDim + 8 * (lane & 7)) =
        make_uint4(y[0], y[1], y[2], y[3]);
  }
}

}  // namespace

cudaError_t launch_latent_append(const LatentPool& pool, const LatentAppendArgs& a, int num_sms, cudaStream_t stream) {
  // One warp a token, so that the angles are computed once, where that fills the SMs; else queries in warps of 16 heads.
  const int per = 16, parts = a.q.heads == 0 || a.n >= 16ll * num_sms ? 1 : 1 + (a.q.heads + per - 1) / per;
  const long long ctas = (a.n * parts * 32 + kThreads - 1) / kThreads;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)ctas;
  if (pool.bf16) {
    if (a.rope.interleaved)
      latent_append_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, stream>>>(pool, a, parts, per);
    else
      latent_append_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, stream>>>(pool, a, parts, per);
  } else {
    if (a.rope.interleaved)
      latent_append_kernel<__half, true><<<grid, kThreads, 0, stream>>>(pool, a, parts, per);
    else
      latent_append_kernel<__half, false><<<grid, kThreads, 0, stream>>>(pool, a, parts, per);
  }
  return cudaGetLastError();
}

cudaError_t launch_latent_read(const LatentPool& pool, const LatentReadArgs& a, cudaStream_t stream) {
  const unsigned grid = (unsigned)(((long long)(a.n + kRows - 1) / kRows * 32 + kThreads - 1) / kThreads);
  if (pool.bf16)
    latent_read_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(pool, a);
  else
    latent_read_kernel<__half><<<grid, kThreads, 0, stream>>>(pool, a);
  return cudaGetLastError();
}

}  // namespace rq
