// Extend (prefill) attention over the 8-bit block-scaled cache: T new tokens per sequence, each
// attending to the cached prefix and causally to the new tokens, on the 5th-generation tensor cores.
//
// The mathematics is rq_block_attention.cu's (value scales in the weights' exponents, a running
// maximum of score + EV that moves past a margin only).  What bounds it is the tensor cores' rate:
// 4 * 128 flops a (query row, token) against 257 cache bytes a token that 256 rows share.
//
// A CTA (one per SM) takes 256 query rows of one (sequence, kv head), two blocks of 128, and walks
// the cache in tiles of 64 tokens, its warps specialised and coupled through mbarriers:
//   softmax (warps 0-7, a thread per row): reads its row of S from tensor memory, applies scales and
//     mask, writes fp16 weights over S;
//   codes (warps 8-11): widen a tile's key and value codes (exact) into fp16 shared-memory operands,
//     loading the next tile's codes meanwhile;
//   MMA (one thread of warp 12; warps 13-15 only fill the warpgroup, 16 warps have 128 registers
//     a thread where 17 would have 96): O_b += W_b V(t) and behind it S_b(t + 1) = Q_b K(t + 1)^T, one block
//     on the tensor cores while the other is in its softmax.  Q and W come from tensor memory (O 2 x
//     128 columns, Q 2 x 64, S 2 x 64 with W over it: all 512), so that shared memory has only K and
//     V to feed: 64 of its 128 bytes a cycle.
// The order of tokens inside a tile is free as long as S's columns and V's rows agree.  It is the one
// in which the cache holds values: column 32 p + 8 t + 4 b + i is token {2t, 2t + 1, 2t + 8, 2t + 9}[i]
// of block 2 p + b, so that a thread's 16 bytes of two blocks' value codes become four whole 16-byte
// chunks of V^T, stored without bank conflicts, and no byte is ever shuffled.
//
// Work is cut evenly: tiles of all units (sequence, 256 rows, kv head) in order, one range per CTA.
// A unit that spans ranges is joined by the last of its CTAs to finish, in the ranges' order.
// Every wait is bounded: one that runs out sets RQ_STATUS_TIMEOUT and an abort flag every role polls.
#include <math_constants.h>

#include <type_traits>

#include "../../include/rq.h"
#include "rq_block.cuh"
#include "rq_rope.cuh"
#include "rq_tc.cuh"

namespace rq {
namespace {

using namespace block;
using namespace tc;

constexpr int kSoftWarps = 8, kCodeWarps = 4, kThreads = 512;
constexpr int kHalf = 128, kRows = 2 * kHalf;  // rows of a block (M of the MMAs), of a CTA
constexpr int kTok = 64;                       // tokens of a tile
constexpr int kStages = 4;                     // K and V operand rings
constexpr int kScaleSlots = 8;                 // tiles whose scales are kept
constexpr uint32_t kOperand = 16384;           // bytes of a K or V stage
constexpr int kSmem = 2 * kStages * (int)kOperand + 1024 + 1024;  // + alignment, + the part below
constexpr int kScanThreads = 512;
constexpr float kMargin = 8.f;      // log2 slack of the running maximum
constexpr float kNone = -1e30f;     // running maximum before any visible token
constexpr float kLarge = 1048576.f; // |maximum| from which weights are formed in two roundings
constexpr int kMinTiles = 8;        // a CTA's least work, while there is enough
// tensor-memory columns
constexpr uint32_t kColQ = 256, kColS = 384;
// floats of a fragment's slot: 256 rows x 128 (as [dim / 4][row][4]), then the rows' m and l
constexpr size_t kSlotFloats = (size_t)kRows * kHeadDim + 2 * kRows;

struct Misc {  // shared, after the operands
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t s_full[2], p_full[2], o_done[2], drain;
  uint32_t tmem;
  int abort;
  float scales[kScaleSlots][3][4];  // per block of a tile: 2^EK, EV, 2^-EV
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpair(uint64_t d, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(d));
}
__device__ __forceinline__ void fma2(float& x, float& y, uint64_t f, uint64_t b) {  // (x, y) = (x, y) * f + b
  uint64_t d = pair(x, y);
  asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(d) : "l"(f), "l"(b));
  unpair(d, x, y);
}
__device__ __forceinline__ void add2(uint64_t& a, float x, float y) {
  const uint64_t d = pair(x, y);
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(d));
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
// Place of column c inside its tile: the token's offset.
__host__ __device__ constexpr int token_of(int c) {
  const int i = c & 3, t = c >> 3 & 3;
  return 32 * (c >> 5) + 16 * (c >> 2 & 1) + 2 * t + (i & 1) + 8 * (i >> 1);
}

// One unit's geometry: 256 rows rb of sequence b.
struct Unit {
  int len, tiles;
};
__device__ __forceinline__ Unit unit_of(const AttnArgs& a, int group, int cap, int b, int rb, bool report) {
  Unit u;
  u.len = __ldg(a.seq_lens + b);
  if (u.len < 0 || u.len > cap || (u.len > 0 && u.len < a.T)) {
    if (report && a.status) atomicOr(a.status, RQ_STATUS_BAD_LEN);
    u.len = u.len < 0 ? 0 : min(u.len, cap);
  }
  const int last = min(a.rows, (rb + 1) * kRows) - 1;
  const int end = max(0, min(u.len, u.len - a.T + last / group + 1));
  u.tiles = max(1, (end + kTok - 1) / kTok);  // rows that see nothing are written too
  return u;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) extend_kernel(const Geometry g, const AttnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Misc ms;
  __shared__ long long s_scan[kScanThreads], s_begin;
  __shared__ int s_item, s_last;
  __shared__ int nan_from[kHeadDim];  // first position with a NaN value in a dim
  uint8_t* const ops = smem_raw + (1024 - (smem_addr(smem_raw) & 1023) & 1023);
  const uint32_t k_ring = smem_addr(ops), v_ring = k_ring + kStages * kOperand;
  volatile int* const abort_flag = &ms.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = a.max_pages * g.page_size, n_rb = (a.rows + kRows - 1) / kRows;
  const long long n_items = (long long)a.B * n_rb;  // (sequence, rows): num_kv_heads units each

  // ---- the CTA's range of tiles ----
  long long mine = 0, chunk = (n_items + kScanThreads - 1) / kScanThreads;
  if (tid < kScanThreads) {
    for (long long i = tid * chunk; i < min(n_items, (tid + 1) * chunk); ++i)
      mine += unit_of(a, g.group, cap, (int)(i / n_rb), (int)(i % n_rb), blockIdx.x == 0).tiles;
    s_scan[tid] = mine;
  }
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&ms.k_full[i]), 32 * kCodeWarps);
      mbar_init(smem_addr(&ms.v_full[i]), 32 * kCodeWarps);
      mbar_init(smem_addr(&ms.k_empty[i]), 1);
      mbar_init(smem_addr(&ms.v_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&ms.s_full[i]), 1);
      mbar_init(smem_addr(&ms.p_full[i]), kHalf);
      mbar_init(smem_addr(&ms.o_done[i]), 1);
    }
    mbar_init(smem_addr(&ms.drain), 1);
    ms.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid < kHeadDim) nan_from[tid] = INT32_MAX;
  __syncthreads();
  for (int o = 1; o < kScanThreads; o <<= 1) {
    const long long v = tid >= o && tid < kScanThreads ? s_scan[tid - o] : 0;
    __syncthreads();
    if (tid < kScanThreads) s_scan[tid] += v;
    __syncthreads();
  }
  const long long total = s_scan[kScanThreads - 1] * g.num_kv_heads;
  const long long parts = min((long long)gridDim.x, max(1ll, total / kMinTiles));
  if ((long long)blockIdx.x >= parts) return;
  auto part_begin = [&](long long c) { return c * total / parts; };
  auto part_of = [&](long long x) { return ((x + 1) * parts - 1) / total; };
  long long x = part_begin(blockIdx.x);
  const long long end = part_begin(blockIdx.x + 1ll);
  if (tid < kScanThreads) {
    const long long before = (s_scan[tid] - mine) * g.num_kv_heads;
    if (x >= before && x < s_scan[tid] * g.num_kv_heads) {
      long long at = before, i = tid * chunk;
      for (;; ++i) {
        const long long n =
            (long long)unit_of(a, g.group, cap, (int)(i / n_rb), (int)(i % n_rb), false).tiles * g.num_kv_heads;
        if (x < at + n) break;
        at += n;
      }
      s_begin = at;
      s_item = (int)i;
    }
  }
  __syncwarp();
  if (warp == 0) tmem_alloc(smem_addr(&ms.tmem), 512);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *(volatile uint32_t*)&ms.tmem;
  long long at = s_begin;
  int item = s_item;

  uint32_t done_tiles = 0;  // tiles of the fragments before: ring positions and parities
  bool ok = true;           // this role has not given up
  while (x < end) {
    // ---- the fragment: tiles r0 .. r1 - 1 of kv head h, rows rb of sequence b ----
    const int b = item / n_rb, rb = item % n_rb;
    const Unit un = unit_of(a, g.group, cap, b, rb, false);
    const int len = un.len, tiles = un.tiles;
    const int h = (int)((x - at) / tiles), r0 = (int)((x - at) % tiles);
    const int r1 = (int)min((long long)tiles, r0 + (end - x)), n = r1 - r0;
    const int32_t* table = a.block_table + (size_t)b * a.max_pages;
    const int blk = warp >> 2 & 1, brow = 32 * (warp & 3) + lane;  // softmax: row block, row in it (= lane of tensor memory)
    const int row = rb * kRows + kHalf * blk + brow;
    const bool valid = row < a.rows;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const int qj = valid ? row / g.group : 0, head = h * g.group + (valid ? row % g.group : 0);
    const size_t row_at = (((size_t)b * a.T + qj) * g.num_q_heads + head) * kHeadDim;
    float q_scale = g.sm_scale * 1.44269504088896340736f, m_run = kNone, l_run = 0.f;

    // the code loads of a tile, units of 16 bytes (rq_block.cuh): code warp dw takes the keys of block dw
    // and half of the dims of the values of blocks p16 and p16 + 1
    const int dw = warp & 3, p16 = dw & 2;
    auto block_at = [&](int t, int blk16) -> const uint8_t* {  // block blk16 of tile t, or null past the sequence
      const int p = t * kTok + 16 * blk16;
      if (p >= len) return nullptr;
      int page = __ldg(table + p / g.page_size);
      if (page < 0 || page >= g.num_pages) {
        if (a.status) atomicOr(a.status, RQ_STATUS_BAD_PAGE);
        page = 0;
      }
      return a.pages + ((size_t)page * g.num_kv_heads + h) * g.page_bytes + (size_t)(p % g.page_size / 16) * kBlockBytes;
    };
    const uint8_t *src_a = nullptr, *src_b = nullptr;  // blocks p16 and p16 + 1 of the tile
    auto look_up = [&](int t) {
      if (t >= r1) return;
      src_a = block_at(t, p16);
      src_b = block_at(t, p16 + 1);
    };
    uint4 kraw[4], vraw[4];
    uint32_t raw_exps = 0;
    auto load = [&]() {  // from the blocks looked up
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      const uint8_t* own = dw & 1 ? src_b : src_a;
#pragma unroll
      for (int u = 0; u < 4; ++u) kraw[u] = own ? __ldg(reinterpret_cast<const uint4*>(own) + 32 * u + lane) : zero;
      raw_exps = own ? __ldg(reinterpret_cast<const uint16_t*>(own + kExps)) : 0x7F7Fu;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at16 = kValues / 16 + 32 * (2 * (dw & 1) + i) + lane;
        vraw[2 * i] = src_a ? __ldg(reinterpret_cast<const uint4*>(src_a) + at16) : zero;
        vraw[2 * i + 1] = src_b ? __ldg(reinterpret_cast<const uint4*>(src_b) + at16) : zero;
      }
    };
    if (warp >= kSoftWarps && warp < kSoftWarps + kCodeWarps) {
      look_up(r0);
      load();
      look_up(r0 + 1);
    }

    // ---- Q of the row into tensor memory: fp16 as it is; a bf16 row by a power of two ----
    if (warp < kSoftWarps) {
      const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q) + row_at);
      float down = 1.f;
      if constexpr (!std::is_same<T, __half>::value) {
        float top = 0.f;
        if (valid)
#pragma unroll 4
          for (int c = 0; c < 16; ++c) {
            const uint4 v = __ldg(src + c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = rope::unpack2<T>(word(v, k));
              top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          }
        const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 127);
        down = pow2(14 - e);
        q_scale *= pow2(e - 14);
      }
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        uint32_t qw[16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 v = valid ? __ldg(src + 4 * cc + c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w = word(v, k);
            if constexpr (!std::is_same<T, __half>::value) {
              const float2 f = rope::unpack2<T>(w);
              w = rope::pack2<__half>(f.x * down, f.y * down);
            }
            qw[4 * c + k] = w;
          }
        }
        tmem_st16u(tmem + lane_off + kColQ + 64 * blk + 16 * cc, qw);
      }
      tmem_wait_st();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();

    const uint32_t t_base = done_tiles;
    if (warp < kSoftWarps) {
      // ================= softmax: one thread per row =================
      const int qpos = valid ? len - a.T + qj : -1;
      const uint32_t s_cols = tmem + lane_off + kColS + 64 * blk, o_cols = tmem + lane_off + 128 * blk;
      for (int t = 0; t < n && ok; ++t) {
        const uint32_t k = t_base + t;
        const int t0 = (r0 + t) * kTok;
        // S_b(t) complete: so is every MMA issued before it, W_b(t - 1) V included
        ok = __all_sync(0xffffffffu, role_wait(smem_addr(&ms.s_full[blk]), k & 1, abort_flag));
        if (!ok) break;
        fence_after_sync();
        float s[kTok];
#pragma unroll
        for (int c = 0; c < kTok / 16; ++c) {
          float v[16];
          tmem_ld16(s_cols + 16 * c, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) s[16 * c + i] = v[i];
        }
        const float4* sc = reinterpret_cast<const float4*>(ms.scales[k % kScaleSlots]);
        const float4 ks4 = sc[0], ev4 = sc[1], dn4 = sc[2];
        const float ks[4] = {ks4.x, ks4.y, ks4.z, ks4.w}, ev[4] = {ev4.x, ev4.y, ev4.z, ev4.w};
        const float dn[4] = {dn4.x, dn4.y, dn4.z, dn4.w};
        tmem_wait_ld();
        const bool large = __any_sync(0xffffffffu, fabsf(m_run) > kLarge && m_run != kNone);
        const float base = m_run == kNone || large ? 0.f : m_run;
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // block q of the tile: columns 32 (q / 2) + 4 (q % 2) + 8 t + i
          const uint64_t f = pair(q_scale * ks[q], q_scale * ks[q]), d = pair(ev[q] - base, ev[q] - base);
#pragma unroll
          for (int t4 = 0; t4 < 4; ++t4) {
            const int c = 32 * (q >> 1) + 4 * (q & 1) + 8 * t4;
            fma2(s[c], s[c + 1], f, d);
            fma2(s[c + 2], s[c + 3], f, d);
          }
        }
        if (t0 + kTok - 1 > qpos) {  // mask what the row may not see
#pragma unroll
          for (int c = 0; c < kTok; ++c)
            if (t0 + token_of(c) > qpos) s[c] = -CUDART_INF_F;
        }
        float tm[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < kTok - 4; c += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i) tm[i] = max3(tm[i], s[c + i], s[c + 4 + i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) tm[i] = fmaxf(tm[i], s[kTok - 4 + i]);
        // relative to `base`: the running maximum, or 0 (none yet, or the large case)
        const float top = fmaxf(max3(tm[0], tm[1], tm[2]), tm[3]);
        float alpha = 1.f, shift = large ? -m_run : 0.f;
        if (top > (m_run == kNone ? -CUDART_INF_F : m_run - base + kMargin)) {
          const float m_new = top + base;
          alpha = ex2(m_run - m_new);
          shift = base - m_new;
          m_run = m_new;
        }
        if (__any_sync(0xffffffffu, shift != 0.f)) {
          const uint64_t one = pair(1.f, 1.f), d = pair(shift, shift);
#pragma unroll
          for (int c = 0; c < kTok; c += 2) fma2(s[c], s[c + 1], one, d);
        }
        l_run *= alpha;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pw[16];
          uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float w0 = ex2(s[32 * half + c]), w1 = ex2(s[32 * half + c + 1]);
            add2(sum[c >> 2 & 1], w0, w1);
            pw[c >> 1] = rope::pack2<__half>(w0, w1);
          }
          tmem_st16u(s_cols + 16 * half, pw);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float lo, hi;
            unpair(sum[q], lo, hi);
            l_run = fmaf(lo + hi, dn[2 * half + q], l_run);
          }
        }
        if (t > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {  // O *= alpha (the warp's rows)
#pragma unroll 1
          for (int c = 0; c < kHeadDim / 16; ++c) {
            float v[16];
            tmem_ld16(o_cols + 16 * c, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= alpha;
            tmem_st16(o_cols + 16 * c, v);
          }
        }
        tmem_wait_st();
        fence_before_sync();
        mbar_arrive(smem_addr(&ms.p_full[blk]));
      }
      if (ok)
        ok = __all_sync(0xffffffffu, role_wait(smem_addr(&ms.o_done[blk]), (t_base + n - 1) & 1, abort_flag));
      fence_after_sync();
      if (!ok && lane == 0 && a.status) atomicOr(a.status, RQ_STATUS_TIMEOUT);
    } else if (warp < kSoftWarps + kCodeWarps) {
      // ================= codes =================
      const int g8 = lane >> 2, t4 = lane & 3;
      for (int t = 0; t < n && ok; ++t) {
        const uint32_t k = t_base + t, st = k % kStages;
        const int t0 = (r0 + t) * kTok;
        if (k >= kStages &&
            !(ok = __all_sync(0xffffffffu, role_wait(smem_addr(&ms.k_empty[st]), (k / kStages - 1) & 1, abort_flag))))
          break;
        {  // unit u: token 8 (u / 2) + g8, dims 64 (u % 2) + 16 t4 ..; the token's row is its column of S
          uint8_t* const dst = ops + st * kOperand;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = 32 * (dw >> 1) + 8 * (g8 >> 1) + 4 * (dw & 1) + (g8 & 1) + 2 * (u >> 1);
            uint8_t* const atom = dst + (u & 1) * 8192;
            *reinterpret_cast<uint4*>(atom + sw128(r, 2 * t4)) =
                make_uint4(widen2(kraw[u].x), widen2_hi(kraw[u].x), widen2(kraw[u].y), widen2_hi(kraw[u].y));
            *reinterpret_cast<uint4*>(atom + sw128(r, 2 * t4 + 1)) =
                make_uint4(widen2(kraw[u].z), widen2_hi(kraw[u].z), widen2(kraw[u].w), widen2_hi(kraw[u].w));
          }
          // k_empty: S(t - 4) of both blocks is done, which was issued behind W(t - 5) V: both softmaxes
          // are past the scales of tile t - 5, and so of t - 8, whose slot this is
          if (lane == 0) {
            const int ev = exp_of_byte(raw_exps >> 8);
            ms.scales[k % kScaleSlots][0][dw] = pow2(exp_of_byte(raw_exps & 0xFF));
            ms.scales[k % kScaleSlots][1][dw] = (float)ev;
            ms.scales[k % kScaleSlots][2][dw] = pow2(-ev);
          }
          fence_async_smem();
          mbar_arrive(smem_addr(&ms.k_full[st]));
        }
        if (k >= kStages &&
            !(ok = __all_sync(0xffffffffu, role_wait(smem_addr(&ms.v_empty[st]), (k / kStages - 1) & 1, abort_flag))))
          break;
        uint32_t bad = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) bad |= __vcmpeq4(word(vraw[i], k4) & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        if (__any_sync(0xffffffffu, bad != 0u || t0 + kTok > len)) {
          // bytes past the sequence may be anything; a NaN value goes to the rows that see it at the end
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // vraw[2 i + b]: block p16 + b, dims 32 (2 (dw % 2) + i) + 4 g8 ..
            uint32_t w[4];
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4) {
              w[k4] = word(vraw[i], k4);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int p = t0 + 16 * (p16 + (i & 1)) + 2 * t4 + (c & 1) + 8 * (c >> 1);
                const bool isnan = (w[k4] >> (8 * c) & 0x7Fu) == 0x7Fu;
                if (isnan && p < len) atomicMin(&nan_from[32 * (2 * (dw & 1) + (i >> 1)) + 4 * g8 + k4], p);
                if (isnan || p >= len) w[k4] &= ~(0xFFu << (8 * c));
              }
            }
            vraw[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        uint8_t* const dst = ops + (kStages + st) * kOperand;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {
            const int d = 32 * (2 * (dw & 1) + i) + 4 * g8 + k4;
            const uint32_t wa = word(vraw[2 * i], k4), wb = word(vraw[2 * i + 1], k4);
            *reinterpret_cast<uint4*>(dst + sw128(d, t4 + 4 * (dw >> 1))) =
                make_uint4(widen2(wa), widen2_hi(wa), widen2(wb), widen2_hi(wb));
          }
        }
        fence_async_smem();
        mbar_arrive(smem_addr(&ms.v_full[st]));
        if (t + 1 < n) {
          load();
          look_up(r0 + t + 2);
        }
      }
      if (!ok && lane == 0 && a.status) atomicOr(a.status, RQ_STATUS_TIMEOUT);
    } else if (tid == 32 * (kSoftWarps + kCodeWarps)) {
      // ================= MMA issue (one thread) =================
      const uint32_t id_s = idesc_f16(kHalf, kTok), id_o = idesc_f16(kHalf, kHeadDim);
      bool issued = false;
      auto s_mmas = [&](int bb, uint32_t kb) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          umma_f16_ts(tmem + kColS + 64 * bb, tmem + kColQ + 64 * bb + 8 * ks, sdesc(kb + (ks >> 2) * 8192 + (ks & 3) * 32),
                      id_s, ks > 0);
        umma_commit(smem_addr(&ms.s_full[bb]));
        issued = true;
      };
      auto wait_k = [&](uint32_t k) { return role_wait(smem_addr(&ms.k_full[k % kStages]), (k / kStages) & 1, abort_flag); };
      if (ok && (ok = wait_k(t_base))) {
        fence_after_sync();
        s_mmas(0, k_ring + t_base % kStages * kOperand);
        s_mmas(1, k_ring + t_base % kStages * kOperand);
        umma_commit(smem_addr(&ms.k_empty[t_base % kStages]));
      }
      for (int t = 0; t < n && ok; ++t) {
        const uint32_t k = t_base + t, vs = k % kStages, ks1 = (k + 1) % kStages;
        const bool next = t + 1 < n;
        if (!(ok = role_wait(smem_addr(&ms.v_full[vs]), (k / kStages) & 1, abort_flag))) break;
        if (next && !(ok = wait_k(k + 1))) break;
#pragma unroll 1
        for (int bb = 0; bb < 2; ++bb) {
          if (!(ok = role_wait(smem_addr(&ms.p_full[bb]), k & 1, abort_flag))) break;
          fence_after_sync();
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_f16_ts(tmem + 128 * bb, tmem + kColS + 64 * bb + 8 * ks, sdesc(v_ring + vs * kOperand + ks * 32), id_o,
                        t > 0 || ks > 0);
          umma_commit(smem_addr(&ms.o_done[bb]));
          if (next) s_mmas(bb, k_ring + ks1 * kOperand);  // over the same columns, behind the MMAs that read them
        }
        if (!ok) break;
        umma_commit(smem_addr(&ms.v_empty[vs]));
        if (next) umma_commit(smem_addr(&ms.k_empty[ks1]));
      }
      if (!ok) {
        if (issued) {  // nothing may be running when the tensor memory is freed
          umma_commit(smem_addr(&ms.drain));
          for (int i = 0; i < kWaitLimit; ++i)
            if (mbar_test(smem_addr(&ms.drain), 0u)) break;
        }
        if (a.status) atomicOr(a.status, RQ_STATUS_TIMEOUT);
      }
    }
    done_tiles += n;
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (ms.abort) break;  // uniform: read after the barrier, and no role raises it between here and there

    // ---- write the rows, or the fragment's part of them ----
    const bool whole = r0 == 0 && r1 == tiles;
    const long long u0 = at + (long long)h * tiles, cf = part_of(u0), cl = part_of(u0 + tiles - 1);
    auto slot_of = [&](long long c) {  // range c's first fragment, or the last of the unit's first range
      return a.ws + (2 * c + (c == cf && part_begin(c) != u0 ? 1 : 0)) * kSlotFloats;
    };
    auto store16 = [&](int c, const float (&y)[16]) {  // dims 16 c .. of the thread's row
      uint4* const dst = reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.out) + row_at) + 2 * c;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        dst[i] = make_uint4(rope::pack2<T>(y[8 * i], y[8 * i + 1]), rope::pack2<T>(y[8 * i + 2], y[8 * i + 3]),
                            rope::pack2<T>(y[8 * i + 4], y[8 * i + 5]), rope::pack2<T>(y[8 * i + 6], y[8 * i + 7]));
    };
    const int qpos = valid ? len - a.T + qj : -1, srow = kHalf * blk + brow;
    if (warp < kSoftWarps) {
      const float inv = whole ? (l_run == 0.f ? 0.f : 1.f / l_run) : 1.f;
      float* const slot = slot_of(blockIdx.x);
#pragma unroll 1
      for (int c = 0; c < kHeadDim / 16; ++c) {
        float y[16];
        __syncwarp();
        tmem_ld16(tmem + lane_off + 128 * blk + 16 * c, y);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          y[i] = l_run == 0.f ? 0.f : y[i] * inv;
          if (nan_from[16 * c + i] <= qpos) y[i] = CUDART_NAN_F;
        }
        if (whole) {
          if (valid) store16(c, y);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4*>(slot)[(4 * c + i) * kRows + srow] =
                make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
        }
      }
      if (!whole) {
        slot[kRows * kHeadDim + srow] = m_run;
        slot[kRows * kHeadDim + kRows + srow] = l_run;
      }
      fence_before_sync();
    }
    if (!whole) {
      const int frags = (int)(cl - cf + 1);
      __threadfence();
      __syncthreads();
      if (tid == 0) s_last = atomicAdd(a.cnt + cf, 1) == frags - 1;
      __syncthreads();
      if (s_last) {
        __threadfence();
        if (tid == 0) a.cnt[cf] = 0;  // as every launch finds it
        if (warp < kSoftWarps) {
          float top = kNone, sum = 0.f;
          for (int f = 0; f < frags; ++f) top = fmaxf(top, __ldcg(slot_of(cf + f) + kRows * kHeadDim + srow));
          for (int f = 0; f < frags; ++f) {
            const float* s = slot_of(cf + f) + kRows * kHeadDim + srow;
            sum = fmaf(__ldcg(s + kRows), ex2(__ldcg(s) - top), sum);
          }
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll 1
          for (int c = 0; c < kHeadDim / 16; ++c) {
            float y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = 0.f;
            for (int f = 0; f < frags; ++f) {
              const float* s = slot_of(cf + f);
              const float w = ex2(__ldcg(s + kRows * kHeadDim + srow) - top) * inv;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(s) + (4 * c + i) * kRows + srow);
                y[4 * i] = fmaf(v.x, w, y[4 * i]), y[4 * i + 1] = fmaf(v.y, w, y[4 * i + 1]);
                y[4 * i + 2] = fmaf(v.z, w, y[4 * i + 2]), y[4 * i + 3] = fmaf(v.w, w, y[4 * i + 3]);
              }
            }
            if (valid) store16(c, y);
          }
        }
      }
    }
    __syncthreads();
    if (tid < kHeadDim) nan_from[tid] = INT32_MAX;  // the next fragment's roles start behind a barrier
    x += n;
    if (x - at == (long long)tiles * g.num_kv_heads) {
      at = x;
      ++item;
    }
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

}  // namespace

size_t block_extend_workspace(int num_sms) { return 2 * (size_t)num_sms * kSlotFloats; }

cudaError_t block_extend_prepare() {
  cudaError_t e = cudaFuncSetAttribute(extend_kernel<__half>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(extend_kernel<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  return e;
}

cudaError_t launch_block_extend(const Geometry& g, AttnArgs a, int num_sms, cudaStream_t stream, cudaEvent_t ev_start,
                                cudaEvent_t ev_end) {
  if ((long long)a.B * ((a.rows + kRows - 1) / kRows) > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (ev_start) cudaEventRecord(ev_start, stream);
  if (g.bf16)
    extend_kernel<__nv_bfloat16><<<num_sms, kThreads, kSmem, stream>>>(g, a);
  else
    extend_kernel<__half><<<num_sms, kThreads, kSmem, stream>>>(g, a);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && ev_end) cudaEventRecord(ev_end, stream);
  return e;
}

}  // namespace rq
