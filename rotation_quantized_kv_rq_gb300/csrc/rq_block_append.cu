// Append to the 8-bit block-scaled cache, with the key's norm and position rotation on the way and
// the queries of the same tokens turned in the same launch.
//
// A block's key scale (and value scale) is 2^E with the smallest E that holds the largest magnitude
// of its tokens.  Tokens arrive a few at a time, so E can only be known so far: the first token of
// a block starts it anew, a later one raises it if it must, and the codes already there are then
// divided by the power of two in place.  Codes are floating point, so that division is exact but
// for codes it makes subnormal (below 2^-14 of the scale's largest value).
//
// Work is split by runs: consecutive tokens of the call in consecutive slots of one block.  One warp
// codes a run's keys or its values of one head, so that a block's scale is one reduction in one warp
// and no atomics order anything; the run's tokens all belong to one block by construction.  No two runs
// that are written share a block: a run that starts inside a block is dropped, and reported, where the
// call has tokens of that block elsewhere (of two runs at most one starts it).  To know that, such a run's CTA
// looks through all the call's slots; prompts have one such run a sequence.
//
// What bounds it: 512 bytes in and 257 out a (token, kv head), and the queries' rows in and out.  32,768
// tokens x (32 + 8) heads, 739 MB: 164 us (4.5 TB/s, 67% of the copy rate).  The queries, in a launch of
// their own, run at rq_rope.cu's rate; the coding of keys and values is bound by its latencies at 16 warps
// an SM (128 registers hold a warp's 16 rows; issue in 47% of the cycles).  Neither 20% fewer instructions
// (whole blocks apart from parts of one), nor more CTAs an SM with the rows read again, was faster.  64
// single tokens x 72 heads: 6.2 us, the chain slot - row - norm - largest value - old scale - codes.  The look
// for tokens elsewhere is beside that chain in short calls (0.1 to 0.4 us) and ahead of one CTA's work a sequence in
// prompts (32,768 tokens from inside a block 162.8 -> 163.1 us; 8,000 of one head, 64 threads, 20 -> 25).
#include "../../include/rq.h"
#include "rq_block.cuh"
#include "rq_rope.cuh"

namespace rq {
namespace {

using namespace rope;
using namespace block;

constexpr int kMaxWarps = 8;
// Tokens from which a CTA takes 16 of them.  Device time, us, 32 and 8 heads, one token or 16 to a CTA:
// 1,024 x 1 token 28 | 72; 128 x 8 17.6 | 29.5; 256 x 8 28.3 | 29.6; 1 x 1,500 20.4 | 23.4; 1 x 2,048 25 | 23.6;
// 1 x 8,000 (one head) 55 | 27; 1 x 16,000 143 | 90.  The slots say how long the runs are, and they
// are on the device: a call with as many tokens is taken for a prompt's, unless each is a sequence's by the
// call's form (a decode step).  Single tokens given by slots pay for it up to some 3,500 of them: 2,048 x 1 52 | 77,
// 3,000 x 1 92 | 106, 4,096 x 1 133 | 115.
constexpr int kLongAppend = 2048;
constexpr int kSplitAppend = 8192;  // tokens from which the queries have a launch of their own

constexpr uint32_t kInf = 0x7F800000u;
constexpr uint32_t kMost = (kMaxExp + 8 + 127) << 23 | 0x600000u;  // 448 * 2^kMaxExp: larger values are stored as that

__device__ __forceinline__ uint32_t code4(uint64_t a, uint64_t b) {
  float x0, x1, x2, x3;
  split2(a, x0, x1);
  split2(b, x2, x3);
  return block::code4(x0, x1, x2, x3);
}

// The scale's exponent for values whose largest magnitude over the warp has the bits `top`, or, if
// that is not finite, for the finite ones among them (a second look, given by `finite_top`).  What the
// values have that d_status reports is added to `faults`.
template <typename F>
__device__ __forceinline__ int warp_exp(uint32_t top, int& faults, F finite_top) {
  top = __reduce_max_sync(0xffffffffu, top);
  if (top > kMost) {
    if (top >= kInf) {
      faults |= RQ_STATUS_NOT_FINITE;
      top = __reduce_max_sync(0xffffffffu, finite_top());
    }
    if (top > kMost) faults |= RQ_STATUS_NORM_OVERFLOW;
  }
  return exp_of(__uint_as_float(top));
}

// Token t's slot, or -1: padding, past the call's end, or a fault (reported once, by `report`).
__device__ __forceinline__ int slot_of(const Geometry& g, const BlockAppendArgs& a, long long t, bool report) {
  if (t < 0 || t >= a.in.n) return -1;
  int fault = 0, s;
  if (a.slots != nullptr) {
    s = __ldg(a.slots + t);
    if (s >= g.num_pages * g.page_size) fault = RQ_STATUS_BAD_SLOT;
  } else {
    const int len = __ldg(a.seq_lens + t), cap = a.max_pages * g.page_size;
    s = -1;
    if (len < 0 || len > cap) {
      fault = RQ_STATUS_BAD_LEN;
    } else if (len > 0) {
      const int page = __ldg(a.block_table + t * a.max_pages + (len - 1) / g.page_size);
      if (page < 0 || page >= g.num_pages)
        fault = RQ_STATUS_BAD_PAGE;
      else
        s = page * g.page_size + (len - 1) % g.page_size;
    }
  }
  if (fault) {
    if (report && a.status) atomicOr(a.status, fault);
    return -1;
  }
  return s;
}

// The slots of a call in groups of four (16-byte loads between ends of up to three): groups i, i + threads, ...,
// N of them, in flight together, and the ends with group threadIdx.x.
template <int N>
struct SlotQuads {
  int4 v[N];
  int ends[2];
  long long count;  // groups of the call
  __device__ __forceinline__ static int head(const int32_t* slots, long long n) {
    return (int)min(n, (long long)((4 - ((uintptr_t)slots >> 2 & 3)) & 3));
  }
  __device__ __forceinline__ void load(const int32_t* slots, long long n, long long i) {
    const int h = head(slots, n);
    count = (n - h) / 4;
    const int4* p = reinterpret_cast<const int4*>(slots + h);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const long long at = i + u * (int)blockDim.x;
      v[u] = at < count ? __ldg(p + at) : make_int4(-1, -1, -1, -1);
    }
    const long long tail = h + 4 * count + i;
    ends[0] = i < h ? __ldg(slots + i) : -1;
    ends[1] = tail < n ? __ldg(slots + tail) : -1;
  }
  template <typename F>
  __device__ __forceinline__ void each(const int32_t* slots, long long n, long long i, F f) const {  // f(token, slot)
    const int h = head(slots, n);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const long long t = h + 4 * (i + u * (int)blockDim.x);
      f(t, v[u].x), f(t + 1, v[u].y), f(t + 2, v[u].z), f(t + 3, v[u].w);
    }
    f(i, ends[0]), f(h + 4 * count + i, ends[1]);
  }
};
// Whether the token at distance d from a run's first, in slot s0, has its slot s in the run's block, but not the slot
// of a token that continues the run.  (Behind a gap there may be one that would continue it: it starts a run
// of its own, and this one is elsewhere to that.)  So of two runs of a block that both start inside it the later is dropped.
__device__ __forceinline__ bool elsewhere(long long d, int s, int s0) {
  return s >= 0 && s / kBlockTokens == s0 / kBlockTokens && (d < 0 || s != s0 + d);
}

// Rows `off` .. off + cnt - 1 of a block's keys from tokens t0 .. (head h).  cs: cosines and sines
// of token t0 + i at cs[i].  Returns the exponent.  The rows
// stay in registers as they came (32, where the turned f32 values would take 64 and leave an SM one
// CTA): they are turned once for the largest magnitude and again for the codes.
template <typename T, bool INTERLEAVED>
__device__ __forceinline__ int append_keys(const BlockAppendArgs& a, uint8_t* blk, int h, long long t0, int off,
                                           int cnt, int e_old, const float4 (*cs)[2][16], int lane, int& faults) {
  const int j = lane & 15, half = lane >> 4;
  const Lane l = lane_of<INTERLEAVED>(j, a.in.rope.rotary_dim);
  const T* src = reinterpret_cast<const T*>(a.in.k.x) + (long long)h * kHeadDim;
  const bool norm = a.in.k.weight != nullptr;
  uint2 raw[8][2];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (2 * i + half < cnt) load8(raw[i], src + (t0 + 2 * i + half) * a.in.k.stride, l);
  uint64_t w[4];
  float inv[8];
  if (norm) load_weights(w, a.in.k.weight, l);
  auto turned = [&](uint64_t (&x)[4], int i, bool first) {
    widen8<T>(x, raw[i]);
    if (norm) {
      if (first) inv[i] = inv_rms(x, a.in.eps);
      scale8(x, inv[i], w);
    }
    if (l.pair >= 0) turn8<INTERLEAVED>(x, angles_of(cs[2 * i + half][0][j], cs[2 * i + half][1][j]), l);
  };
  auto largest = [](uint32_t m, uint64_t x) {  // of the magnitudes' bits
    return max(max(m, (uint32_t)x & 0x7FFFFFFFu), (uint32_t)(x >> 32) & 0x7FFFFFFFu);
  };
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (2 * i + half < cnt) {
      uint64_t x[4];
      turned(x, i, true);
#pragma unroll
      for (int k = 0; k < 4; ++k) top = largest(top, x[k]);
    }
  }
  const int e_new = warp_exp(top, faults, [&]() {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (2 * i + half < cnt) {
        uint64_t x[4];
        turned(x, i, false);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t u = (uint32_t)(x[k >> 1] >> (32 * (k & 1))) & 0x7FFFFFFFu;
          m = max(m, u < kInf ? u : 0u);
        }
      }
    }
    return m;
  });
  const int e = off == 0 ? e_new : max(e_old, e_new);
  if (off > 0 && e > e_old) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint4* p = reinterpret_cast<uint4*>(blk) + 32 * u + lane;
      uint4 c = *p;
      c.x = shrink4(c.x, e - e_old), c.y = shrink4(c.y, e - e_old);
      c.z = shrink4(c.z, e - e_old), c.w = shrink4(c.w, e - e_old);
      *p = c;
    }
    __syncwarp();  // the rows below overwrite some of these bytes
  }
  const uint64_t s2 = f2(pow2(-e), pow2(-e));
  auto place = [&](int d) { return ((d >> 6) * 32 + ((d & 63) >> 4)) * 16 + (d & 15); };  // of token 0
  uint8_t* const d0 = blk + place(l.o0);
  uint8_t* const d1 = blk + place(l.o1);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (2 * i + half < cnt) {
      const int r = off + 2 * i + half, at = (r >> 3) * 1024 + (r & 7) * 64;
      uint64_t x[4];
      turned(x, i, false);
      *reinterpret_cast<uint32_t*>(d0 + at) = code4(mul2(x[0], s2), mul2(x[1], s2));
      *reinterpret_cast<uint32_t*>(d1 + at) = code4(mul2(x[2], s2), mul2(x[3], s2));
    }
  }
  return e;
}

__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b, __half) {  // per half: max(a, |b|), NaN if any is
  const __half2 m = __hmax2_nan(*reinterpret_cast<const __half2*>(&a), __habs2(*reinterpret_cast<const __half2*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&m);
}
__device__ __forceinline__ uint32_t abs_max2(uint32_t a, uint32_t b, __nv_bfloat16) {
  const __nv_bfloat162 m =
      __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a), __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// The same of values.  Lane 4 g + t takes tokens 2t, 2t + 1, 2t + 8, 2t + 9 and of each the dims 32 u + 4 g
// .. + 3, which are unit u of its 16 bytes in the block: a store of the warp is 512 bytes in a row, a
// load 64 of four rows.  Bytes of rows outside the run stay as they are.
template <typename T>
__device__ __forceinline__ int append_values(const BlockAppendArgs& a, uint8_t* blk, int h, long long t0, int off,
                                             int cnt, int e_old, int lane, int& faults) {
  const int g4 = 4 * (lane >> 2), t2 = 2 * (lane & 3);
  uint2 raw[4][4];  // [token][unit]
  uint32_t mask = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = t2 + (i & 1) + 8 * (i >> 1);
    const bool here = r >= off && r < off + cnt;
    const T* src = reinterpret_cast<const T*>(a.v) + (t0 + r - off) * a.v_stride + (long long)h * kHeadDim + g4;
    if (here) mask |= 0xFFu << (8 * i);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      raw[i][u] = make_uint2(0u, 0u);
      if (here) raw[i][u] = __ldg(reinterpret_cast<const uint2*>(src + 32 * u));
    }
  }
  uint32_t m2 = 0u;
#pragma unroll
  for (int i = 0; i < 16; ++i) m2 = abs_max2(abs_max2(m2, raw[i >> 2][i & 3].x, T()), raw[i >> 2][i & 3].y, T());
  const float2 m = unpack2<T>(m2);
  const uint32_t top = max(__float_as_uint(m.x) & 0x7FFFFFFFu, __float_as_uint(m.y) & 0x7FFFFFFFu);
  const int e_new = warp_exp(top, faults, [&]() {
    uint32_t f = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 p = unpack2<T>(raw[i >> 2][i & 3].x), q = unpack2<T>(raw[i >> 2][i & 3].y);
      const float x[4] = {p.x, p.y, q.x, q.y};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t u = __float_as_uint(x[k]) & 0x7FFFFFFFu;
        f = max(f, u < kInf ? u : 0u);
      }
    }
    return f;
  });
  const int e = off == 0 ? e_new : max(e_old, e_new);
  const bool grow = off > 0 && e > e_old;
  if (mask == 0u && !grow) return e;
  const uint64_t s2 = f2(pow2(-e), pow2(-e));
  uint4* const dst = reinterpret_cast<uint4*>(blk + kValues) + lane;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = unpack2<T>(raw[i][u].x), q = unpack2<T>(raw[i][u].y);
      w[i] = code4(mul2(f2(p.x, p.y), s2), mul2(f2(q.x, q.y), s2));  // one token, four dims
    }
    // to one dim, four tokens: a 4 x 4 transpose of bytes
    const uint32_t a0 = __byte_perm(w[0], w[1], 0x5140), a1 = __byte_perm(w[2], w[3], 0x5140);
    const uint32_t b0 = __byte_perm(w[0], w[1], 0x7362), b1 = __byte_perm(w[2], w[3], 0x7362);
    uint4 c = make_uint4(__byte_perm(a0, a1, 0x5410), __byte_perm(a0, a1, 0x7632), __byte_perm(b0, b1, 0x5410),
                         __byte_perm(b0, b1, 0x7632));
    if (mask != 0xFFFFFFFFu) {
      uint4 o = dst[32 * u];
      if (grow) {
        o.x = shrink4(o.x, e - e_old), o.y = shrink4(o.y, e - e_old);
        o.z = shrink4(o.z, e - e_old), o.w = shrink4(o.w, e - e_old);
      }
      c.x = (c.x & mask) | (o.x & ~mask), c.y = (c.y & mask) | (o.y & ~mask);
      c.z = (c.z & mask) | (o.z & ~mask), c.w = (c.w & mask) | (o.w & ~mask);
    }
    dst[32 * u] = c;
  }
  return e;
}

// The runs that start among a CTA's W = 16 tokens.
constexpr int kFilterWords = 512;
struct Runs {
  int at[16], cnt[16], slot[16], num;  // first token (of the CTA's), tokens, first slot; runs
  uint32_t inside, apart;  // first tokens of runs that start inside a block; of them those whose block has tokens elsewhere
  uint32_t filter[kFilterWords];  // bits of those blocks' numbers modulo 16,384
  __device__ __forceinline__ uint32_t maybe(int s) const {  // (padding: past all blocks)
    const uint32_t blk = (uint32_t)s / kBlockTokens;
    return filter[(blk >> 5) % kFilterWords] >> (blk & 31) & 1;
  }
};
// Drops, and reports, the runs that start inside a block that has tokens elsewhere in the call; `apart` already
// holds those with tokens among the kSeen of the CTA's first.  By the whole CTA.  (Not inlined: that cost the
// kernel's loop 4 to 28%, in calls without such runs too.)
template <int kSeen>
__device__ __noinline__ void drop_apart(Runs& runs, const int32_t* slots, long long n, long long base, int32_t* status) {
  const int tid = threadIdx.x;
  uint32_t mine = 0u;
  constexpr int N = 4;
  SlotQuads<N> quads;
  for (long long i = tid;; i += N * blockDim.x) {
    quads.load(slots, n, i);
    uint32_t hits = 0u;  // all looks at the filter together, no branch between
    int at = 0;
    quads.each(slots, n, i, [&](long long t, int s) {
      hits |= (t < base || t >= base + kSeen ? runs.maybe(s) : 0u) << at++;
    });
    if (hits != 0u) {
      at = 0;
      quads.each(slots, n, i, [&](long long t, int s) {
        if (!(hits >> at++ & 1)) return;
        for (int r = 0; r < runs.num; ++r)
          if ((runs.inside >> runs.at[r] & 1) && elsewhere(t - base - runs.at[r], s, runs.slot[r])) mine |= 1u << runs.at[r];
      });
    }
    if (i - tid + N * blockDim.x >= quads.count) break;
  }
  mine = __reduce_or_sync(0xffffffffu, mine);
  if ((tid & 31) == 0 && mine != 0u) atomicOr(&runs.apart, mine);
  __syncthreads();
  if (runs.apart == 0u) return;
  if (tid == 0) {  // what is left of the runs
    int kept = 0;
    for (int i = 0; i < runs.num; ++i) {
      if (runs.apart >> runs.at[i] & 1) continue;
      runs.at[kept] = runs.at[i], runs.cnt[kept] = runs.cnt[i], runs.slot[kept] = runs.slot[i];
      ++kept;
    }
    runs.num = kept;
    if (status) atomicOr(status, RQ_STATUS_BAD_ORDER);
  }
  __syncthreads();
}

// A CTA takes the runs that start among its W tokens, and those W tokens' queries.  W = 1 spreads a
// decode step's single tokens over the SMs; W = 16 (long appends) makes one block of a run a
// CTA's work.  blockIdx.y splits the heads.
template <typename T, bool INTERLEAVED, int W>
__global__ void __launch_bounds__(32 * kMaxWarps, 2) block_append_kernel(const Geometry g, const BlockAppendArgs a) {
  constexpr int kTokens = W == 1 ? 16 : 32;  // a run reaches at most 15 tokens past its first
  __shared__ float4 cs[kTokens][2][16];  // [token][cosines, sines][j]: pairs 4j .. 4j + 3
  __shared__ Runs runs;  // (W = 1: one run, nothing of its filter)
  __shared__ int reach;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const long long base = (long long)blockIdx.x * W;
  const int hw = tid >> 4, hws = blockDim.x >> 4, j = tid & 15;
  auto angles = [&](int i) {  // cosines and sines of token base + i, by a half-warp
    if (4 * j < a.in.rope.rotary_dim >> 1 && base + i < a.in.n) {
      float4 c, s;
      cos_sin4(c, s, a.in.rope, 4 * j, a.in.positions, a.in.n, base + i);
      cs[i][0][j] = c;
      cs[i][1][j] = s;
    }
  };
  // W = 1: the first of the call's slots, loaded beside the rest of the opening
  int slot0 = -1, before = -1;
  SlotQuads<1> quads;
  if (W == 1 && a.slots != nullptr) {
    slot0 = __ldg(a.slots + base);
    if (base > 0) before = __ldg(a.slots + base - 1);
    quads.load(a.slots, a.in.n, tid);
  }
  if (warp == 0) {
    const int s = lane < kTokens ? slot_of(g, a, base + lane, lane < W && blockIdx.y == 0) : -1;
    int prev = __shfl_up_sync(0xffffffffu, s, 1);
    if (lane == 0) prev = slot_of(g, a, base - 1, false);
    const bool cont = s >= 0 && s % kBlockTokens != 0 && prev == s - 1;
    const uint32_t conts = __ballot_sync(0xffffffffu, cont);
    const uint32_t leads = __ballot_sync(0xffffffffu, lane < W && s >= 0 && !cont);
    int cnt = 0;
    if (leads >> lane & 1) {
      const uint32_t after = lane < 31 ? conts >> (lane + 1) : 0u;
      cnt = __ffs(~after);  // 1 + the tokens that continue it
      const int i = __popc(leads & ((1u << lane) - 1u));
      runs.at[i] = lane, runs.cnt[i] = cnt, runs.slot[i] = s;
    }
    const int ends = __reduce_max_sync(0xffffffffu, cnt > 0 ? lane + cnt : 0);
    if (W > 1) {
      const bool in = (leads >> lane & 1) && s % kBlockTokens != 0 && a.slots != nullptr;
      const uint32_t ins = __ballot_sync(0xffffffffu, in);
      uint32_t apart = 0u;
      if (ins != 0u) {
        for (int i = lane; i < kFilterWords; i += 32) runs.filter[i] = 0u;
        __syncwarp();
        if (in) atomicOr(&runs.filter[(s / kBlockTokens >> 5) % kFilterWords], 1u << (s / kBlockTokens & 31));
        // among these tokens: those of the block, but for later ones in the slots of tokens that continue the run
        const uint32_t same = __match_any_sync(0xffffffffu, s >= 0 ? s / kBlockTokens : -1 - lane);
        const uint32_t line = __match_any_sync(0xffffffffu, s >= 0 ? s - lane : INT32_MIN + lane);
        apart = __ballot_sync(0xffffffffu, in && (same & ~(line & 0xffffffffu << lane)) != 0u);
      }
      if (lane == 0) runs.inside = ins, runs.apart = apart;
    }
    if (lane == 0) runs.num = __popc(leads), reach = ends;
  } else {  // meanwhile the angles of the W tokens
    for (int i = hw - 2; i < W; i += hws - 2) angles(i);
  }
  bool dropped = false;  // W = 1: the run (a decode step's tokens are each a sequence's: no look)
  if (W == 1) {
    bool other = false;
    if (slot0 > 0 && slot0 % kBlockTokens != 0 && before != slot0 - 1) {
      auto look = [&](long long t, int s) { other = other || elsewhere(t - base, s, slot0); };
      quads.each(a.slots, a.in.n, tid, look);
      SlotQuads<1> more;
      for (long long i = tid + blockDim.x; i < quads.count; i += blockDim.x) {
        more.load(a.slots, a.in.n, i);
        more.each(a.slots, a.in.n, i, look);
      }
    }
    dropped = __syncthreads_or(other);
    if (dropped && tid == 0 && blockIdx.y == 0 && runs.num > 0 && a.status) atomicOr(a.status, RQ_STATUS_BAD_ORDER);
  } else {
    __syncthreads();
  }
  if (reach > W) {  // a run goes on past them
    for (int i = W + hw; i < reach; i += hws) angles(i);
    __syncthreads();
  }
  if (W > 1 && runs.inside != 0u) drop_apart<kTokens>(runs, a.slots, a.in.n, base, a.status);

  int faults = 0;
  const int items = dropped ? 0 : 2 * runs.num * g.num_kv_heads;  // (run, keys or values, head)
  for (int it = blockIdx.y * warps + warp; it < items; it += gridDim.y * warps) {
    const int run = it / (2 * g.num_kv_heads), of = it % (2 * g.num_kv_heads), h = of % g.num_kv_heads;
    const bool keys = of < g.num_kv_heads;
    const int at = runs.at[run], cnt = runs.cnt[run], slot = runs.slot[run], off = slot % kBlockTokens;
    uint8_t* blk = a.pages + ((size_t)(slot / g.page_size) * g.num_kv_heads + h) * g.page_bytes +
                   (size_t)(slot % g.page_size / kBlockTokens) * kBlockBytes;
    uint8_t* const exp_at = blk + kExps + (keys ? 0 : 1);
    const int e_old = off > 0 ? exp_of_byte(*exp_at) : kMinExp;
    const int e = keys ? append_keys<T, INTERLEAVED>(a, blk, h, base + at, off, cnt, e_old, cs + at, lane, faults)
                       : append_values<T>(a, blk, h, base + at, off, cnt, e_old, lane, faults);
    if (lane == 0) *exp_at = (uint8_t)(e + 127);
  }
  if (faults && a.status) atomicOr(a.status, faults);

  if (a.in.q.heads > 0) {
    const Lane l = lane_of<INTERLEAVED>(j, a.in.rope.rotary_dim);
    // W = 16: a half-warp takes a token's heads; W = 1: the half-warps share the token's heads
    const int i0 = W == 1 ? 0 : hw, h0 = W == 1 ? blockIdx.y * hws + hw : blockIdx.y;
    for (int i = i0; i < W && base + i < a.in.n; i += hws) {
      Angles p;
      if (l.pair >= 0) p = angles_of(cs[i][0][j], cs[i][1][j]);
      turn_rows<T, INTERLEAVED>(reinterpret_cast<const T*>(a.in.q.x) + (base + i) * a.in.q.stride,
                                reinterpret_cast<T*>(a.in.q.out) + (base + i) * a.in.q.out_stride, h0,
                                W == 1 ? gridDim.y * hws : gridDim.y, a.in.q.heads, a.in.q.weight, a.in.eps, p, l);
    }
  }
}

template <typename T, bool INTERLEAVED>
void launch(const Geometry& g, const BlockAppendArgs& a, int num_sms, cudaStream_t stream) {
  const int hkv = g.num_kv_heads, hq = a.in.q.heads;
  int warps = hkv < 2 ? 2 : (2 * hkv > kMaxWarps ? kMaxWarps : 2 * hkv);
  if (a.in.n < kLongAppend || a.slots == nullptr) {
    if (hq > 0) warps = kMaxWarps;
    const int most = max((2 * hkv + warps - 1) / warps, (hq + 2 * warps - 1) / (2 * warps));
    long long split = (2LL * num_sms + a.in.n - 1) / a.in.n;
    split = split > most ? most : split;
    block_append_kernel<T, INTERLEAVED, 1><<<dim3((unsigned)a.in.n, (unsigned)split), 32 * warps, 0, stream>>>(g, a);
  } else {
    block_append_kernel<T, INTERLEAVED, 16><<<dim3((unsigned)((a.in.n + 15) / 16), 1), 32 * warps, 0, stream>>>(g, a);
  }
}

}  // namespace

cudaError_t launch_block_append(const Geometry& g, BlockAppendArgs a, int num_sms, cudaStream_t stream) {
  if (a.in.n <= 0) return cudaSuccess;
  if (a.in.n >= kSplitAppend && a.in.q.heads > 0) {
    // long calls turn the queries in a launch of their own, with twice this kernel's warps on an SM
    NormRopeArgs q = a.in;
    q.k = RowsDev{};
    q.bf16 = g.bf16;
    const cudaError_t e = launch_norm_rope(q, num_sms, stream);
    if (e != cudaSuccess) return e;
    a.in.q = RowsDev{};
  }
  if (g.bf16) {
    if (a.in.rope.interleaved)
      launch<__nv_bfloat16, true>(g, a, num_sms, stream);
    else
      launch<__nv_bfloat16, false>(g, a, num_sms, stream);
  } else {
    if (a.in.rope.interleaved)
      launch<__half, true>(g, a, num_sms, stream);
    else
      launch<__half, false>(g, a, num_sms, stream);
  }
  return cudaGetLastError();
}

}  // namespace rq
