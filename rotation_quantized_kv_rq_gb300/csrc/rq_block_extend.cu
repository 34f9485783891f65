// Extend (prefill) attention over the 8-bit block-scaled cache: T new tokens per sequence, each
// attending to the cached prefix and causally to the new tokens, on the 5th-generation tensor cores.
//
// The mathematics is rq_block_attention.cu's (value scales in the weights' exponents, a running
// maximum of score + EV that moves past a margin only).  What bounds it is the tensor cores' rate:
// 4 * 128 flops a (query row, token) against 257 cache bytes a token that 256 rows share.
//
// A CTA (one per SM) takes 256 query rows of one (sequence, kv head), two blocks of 128, and walks
// the cache in tiles of 128 tokens, its warps specialised and coupled through mbarriers:
//   softmax (warps 0-7, a thread per row): reads its row of S from tensor memory 64 columns at a
//     time, applies scales and mask, writes fp16 weights over S;
//   codes (warps 8-11): widen a tile's key and value codes (exact) into fp16 operands, keys in two
//     stages, values in one;
//   MMA (warp 12): for each block in turn O_b += W_b V(t) and behind it S_b(t + 1) = Q_b K(t + 1)^T, so
//     that one block is on the tensor cores while the other is in its softmax.  All of it in one warp
//     with uniform operands and an elected lane: an MMA takes 16 to 22 cycles to issue so, 50 in a
//     branch of one lane;
//   copies (warp 13): a block is one 4112-byte bulk copy into a ring of two tiles, page ids looked up
//     8 half tiles ahead.
// (Warps 14 and 15 only fill the warpgroup: 16 warps have 128 registers a thread.)
// Why these shapes: an MMA with N = 64 takes as long as one with N = 128 (64.5 and 65.5 cycles for M =
// 128, K = 16, A in tensor memory), so S is 128 columns wide.  That fills tensor memory (O 2 x 128
// columns, S 2 x 128 with W over it) and puts Q into shared memory.  A tile is 32 MMAs, 2064 cycles
// measured alone; 8 x 1,024 rows over 15K take 1.80 ms, 1,185 TFLOP/s, 63% of the burst rate of a
// large matrix product and 69% of its sustained rate.  What is left is the softmax between a block's S
// and its W: two passes over 128 scores a thread, beside which the tensor cores have one other block.
// Measured and slower: the two blocks' softmaxes kept in turns 3.0 ms (2.1 with turns of half a
// tile), 16 softmax warps of 80 registers 2.9, an MMA warp for each block 2.5, 32 columns at a time.
// The order of tokens inside a half tile of 64 is free as long as S's columns and V's rows agree.  It
// is the one in which the cache holds values: column 32 p + 8 t + 4 b + i is token {2t, 2t + 1, 2t + 8,
// 2t + 9}[i] of block 2 p + b, so that a thread's 16 bytes of two blocks' value codes become four
// whole 16-byte chunks of V^T, stored without bank conflicts, and no byte is ever shuffled.
//
// Work is cut evenly: tiles of all units (sequence, 256 rows, kv head) in order, one range per CTA.
// A unit that spans ranges is joined by the last of its CTAs to finish, in the ranges' order.
// Calls with little work (at most 2^23 rows x tokens of the block tables) go to the split-K kernel: a fragment
// opens and closes in some 10 us here.  Measured, split-K and this kernel: 3 x 77 rows of up to 2K (5.7 M)
// 28 and 46 us, 2 x 128 of 4K (8.4 M) 36 and 42, 4 x 128 of 2K (34 M) 110 and 58.
// Every wait is bounded: one that runs out sets RQ_STATUS_TIMEOUT and an abort flag every role polls.
#include <math_constants.h>

#include <cstddef>
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
constexpr int kMmaWarp = kSoftWarps + kCodeWarps, kCopyWarp = kMmaWarp + 1;
constexpr int kHalf = 128, kRows = 2 * kHalf;  // rows of a block (M of the MMAs), of a CTA
constexpr int kTok = 128, kPart = 64;          // tokens of a tile, of the half that softmax and V take at a time
constexpr int kKeyStages = 2, kRawStages = 4;  // K operands (tiles; V has one), raw codes (half tiles)
constexpr uint32_t kOperand = 32768, kRawBytes = 4 * kBlockBytes;
constexpr uint32_t kQBytes = 2 * 32768;
constexpr int kScaleSlots = 4;      // tiles whose scales are kept
constexpr float kLarge = 1048576.f; // |maximum| from which weights are formed in two roundings
constexpr int kMinTiles = 4;        // a CTA's least work, while there is enough
constexpr uint32_t kColS = 256;     // tensor memory: O_b at 128 b, S_b at 256 + 128 b
// floats of a fragment's slot: 256 rows x 128 (as [dim / 4][row][4]), then the rows' m and l
constexpr size_t kSlotFloats = (size_t)kRows * kHeadDim + 2 * kRows;

struct Frag {           // tiles r0 .. r0 + n - 1 of one unit
  int b, rb, h, r0, n, len;
  int whole, frags;     // the unit is all here; else its number of fragments
  long long range;      // its first range, and whether the fragment there is that range's last
  int range_last;
  int done;             // no more fragments
};
struct Misc {
  uint64_t raw_full[kRawStages], raw_empty[kRawStages];
  // K(t), V(t) are there; S(t), W V(t) of both blocks done: K(t), V(t) are read; [block] S(t); [block] W(t); [block] the
  // fragment's last W V; the fragment's queries; drained
  uint64_t k_full[kKeyStages], v_full, k_read[kKeyStages], v_read, s_full[2], p_full[2], o_done[2], q_full, drain;
  Frag f;
  uint32_t tmem;
  int abort, last, any_nan;
  alignas(16) float scales[kScaleSlots][2][3][4];  // [half][2^EK, EV, 2^-EV][block], read as float4
  int nan_from[kHeadDim];              // first position with a NaN value in a dim
};
// from a 1024-byte boundary on: Q, keys, values, raw codes, Misc
constexpr uint32_t kOffK = kQBytes, kOffV = kOffK + kKeyStages * kOperand, kOffRaw = kOffV + kOperand;
constexpr uint32_t kOffMisc = kOffRaw + kRawStages * kRawBytes;
constexpr int kSmem = (int)(kOffMisc + sizeof(Misc)) + 1024;
static_assert(kRawStages == 4, "two tiles' halves");
static_assert(kOffMisc % 16 == 0 && offsetof(Misc, scales) % 16 == 0, "float4 reads");
static_assert(kSmem + 64 <= 232448, "one CTA's shared memory");

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
// A warp's wait, bounded (about a second) like tc::role_wait, but asleep between its looks at the
// barrier.  All lanes look: one lane's loop beside 31 waiting ones took about 1000 cycles longer.
__device__ __forceinline__ bool warp_wait(const uint64_t& bar, uint32_t parity, volatile int* abort_flag) {
  bool ok = false;
  for (int i = 0; i < (1 << 16); ++i) {
    uint32_t done;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
                 : "=r"(done)
                 : "r"(smem_addr(&bar)), "r"(parity & 1), "r"(20000u)  // ns
                 : "memory");
    ok = done;
    if (done || *abort_flag) break;
  }
  if (!ok) *abort_flag = 1;
  return __all_sync(0xffffffffu, ok);
}
// A warp's arrival, by one lane (a predicate, no branch) behind all lanes' accesses.
__device__ __forceinline__ void warp_arrive(uint64_t& bar) {
  __syncwarp();
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n @e mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(
                   smem_addr(&bar))
               : "memory");
}
// The MMAs and commit of tc::, by one elected lane of a whole warp: with the operands uniform over the
// warp an MMA is issued in 16 to 22 cycles, against 50 in a branch that one lane takes.
__device__ __forceinline__ void elect_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate));
}
__device__ __forceinline__ void elect_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(accumulate));
}
__device__ __forceinline__ void elect_commit(uint32_t mbar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(mbar)
      : "memory");
}
// Place of column c of a half tile: the token's offset.
__host__ __device__ constexpr int token_of(int c) {
  const int i = c & 3, t = c >> 3 & 3;
  return 32 * (c >> 5) + 16 * (c >> 2 & 1) + 2 * t + (i & 1) + 8 * (i >> 1);
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
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
  const uint32_t base = smem_addr(smem_raw) + (1024 - (smem_addr(smem_raw) & 1023) & 1023);
  Misc& ms = *reinterpret_cast<Misc*>(smem_raw + (base - smem_addr(smem_raw)) + kOffMisc);
  const uint32_t q_ops = base, k_ring = base + kOffK, v_ring = base + kOffV, raw_ring = base + kOffRaw;
  volatile int* const abort_flag = &ms.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = a.max_pages * g.page_size, n_rb = (a.rows + kRows - 1) / kRows;

  // ---- the CTA's range of tiles: x .. end - 1 of `total`, kept by thread 0 ----
  long long total, parts, x = 0, end = 0, at = 0;
  long long item = 0;  // (sequence, rows): num_kv_heads units each, the first at tile `at`
  {
    long long* const scan = reinterpret_cast<long long*>(smem_raw + (base - smem_addr(smem_raw)));  // over Q
    __shared__ long long s_found[2];
    const long long n_items = (long long)a.B * n_rb, chunk = (n_items + kThreads - 1) / kThreads;
    long long mine = 0;
    for (long long i = tid * chunk; i < min(n_items, (tid + 1) * chunk); ++i)
      mine += unit_of(a, g.group, cap, (int)(i / n_rb), (int)(i % n_rb), blockIdx.x == 0).tiles;
    scan[tid] = mine;
    __syncthreads();
    for (int o = 1; o < kThreads; o <<= 1) {
      const long long v = tid >= o ? scan[tid - o] : 0;
      __syncthreads();
      scan[tid] += v;
      __syncthreads();
    }
    total = scan[kThreads - 1] * g.num_kv_heads;
    parts = min((long long)gridDim.x, max(1ll, total / kMinTiles));
    if ((long long)blockIdx.x >= parts) return;
    x = blockIdx.x * total / parts;
    end = (blockIdx.x + 1ll) * total / parts;
    const long long before = (scan[tid] - mine) * g.num_kv_heads;
    if (x >= before && x < scan[tid] * g.num_kv_heads) {
      long long p = before, i = tid * chunk;
      for (;; ++i) {
        const long long n =
            (long long)unit_of(a, g.group, cap, (int)(i / n_rb), (int)(i % n_rb), false).tiles * g.num_kv_heads;
        if (x < p + n) break;
        p += n;
      }
      s_found[0] = p;
      s_found[1] = i;
    }
    __syncthreads();
    at = s_found[0];
    item = s_found[1];
  }
  if (tid == 0) {
    for (int i = 0; i < kRawStages; ++i) {
      mbar_init(smem_addr(&ms.raw_full[i]), 1);
      mbar_init(smem_addr(&ms.raw_empty[i]), kCodeWarps);
    }
    for (int i = 0; i < kKeyStages; ++i) {
      mbar_init(smem_addr(&ms.k_full[i]), kCodeWarps);
      mbar_init(smem_addr(&ms.k_read[i]), 1);
    }
    mbar_init(smem_addr(&ms.v_full), kCodeWarps);
    mbar_init(smem_addr(&ms.v_read), 1);
    mbar_init(smem_addr(&ms.drain), 1);
    mbar_init(smem_addr(&ms.q_full), kSoftWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&ms.s_full[i]), 1);
      mbar_init(smem_addr(&ms.p_full[i]), kSoftWarps / 2);
      mbar_init(smem_addr(&ms.o_done[i]), 1);
    }
    ms.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  if (warp == 0) tmem_alloc(smem_addr(&ms.tmem), 512);

  uint32_t done_tiles = 0, done_frags = 0;  // tiles and fragments before: ring positions and parities
  uint32_t fills = 0;       // copy warp: half tiles asked for
  for (;;) {
    if (tid == 0) {  // the next fragment
      Frag& f = ms.f;
      f.done = x >= end;
      if (!f.done) {
        f.b = (int)(item / n_rb);
        f.rb = (int)(item % n_rb);
        const Unit un = unit_of(a, g.group, cap, f.b, f.rb, false);
        f.len = un.len;
        f.h = (int)((x - at) / un.tiles);
        f.r0 = (int)((x - at) % un.tiles);
        f.n = (int)min((long long)un.tiles - f.r0, end - x);
        f.whole = f.n == un.tiles;
        const long long u0 = x - f.r0, u1 = u0 + un.tiles - 1;
        f.range = ((u0 + 1) * parts - 1) / total;  // the range that holds tile u0
        f.range_last = f.range * total / parts != u0;
        f.frags = (int)(((u1 + 1) * parts - 1) / total - f.range) + 1;
        x += f.n;
        if (x - at == (long long)un.tiles * g.num_kv_heads) {
          at = x;
          ++item;
        }
      }
    }
    if (tid < kHeadDim) ms.nan_from[tid] = INT32_MAX;
    if (tid == 0) ms.any_nan = 0;
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (ms.f.done) break;
    const uint32_t tmem = *(volatile uint32_t*)&ms.tmem;
    const int b = ms.f.b, h = ms.f.h, r0 = ms.f.r0, n = ms.f.n, len = ms.f.len;
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    // softmax: row block, row in it (= lane of tensor memory), query row
    const int blk = warp >> 2 & 1, brow = 32 * (warp & 3) + lane, row = ms.f.rb * kRows + kHalf * blk + brow;
    const bool valid = row < a.rows;
    float q_scale = 0.f, m_run = kNone, l_run = 0.f;
    auto row_offset = [&]() {
      const int j = valid ? row / g.group : 0, head = h * g.group + (valid ? row % g.group : 0);
      return (((size_t)b * a.T + j) * g.num_q_heads + head) * kHeadDim;
    };

    // ---- Q of the row as an operand: fp16 as it is; a bf16 row by a power of two ----
    // (the keys' and values' roles start meanwhile; the MMAs wait for q_full)
    if (warp < kSoftWarps) {
      const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q) + row_offset());
      constexpr bool kBf16 = !std::is_same<T, __half>::value;
      float top = 0.f;
      if constexpr (kBf16) {
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const uint4 v = valid ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = rope::unpack2<T>(word(v, k));
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
      }
      const RowScale scale = row_scale<kBf16>(top, g.sm_scale * 1.44269504088896340736f);
      q_scale = scale.factor;
#pragma unroll 8
      for (int c = 0; c < 16; ++c) {
        const uint4 v = valid ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          w[k] = word(v, k);
          if constexpr (kBf16) {
            const float2 f = rope::unpack2<T>(w[k]);
            w[k] = rope::pack2<__half>(f.x * scale.down, f.y * scale.down);
          }
        }
        sts128(q_ops + 32768 * blk + 16384 * (c >> 3) + sw128(brow, c & 7), w[0], w[1], w[2], w[3]);
      }
      fence_async_smem();
      warp_arrive(ms.q_full);
    }

    bool ok = true;
    const uint32_t t_base = done_tiles;
    if (warp < kSoftWarps) {
      // ================= softmax: one thread per row =================
      const int qpos = valid ? len - a.T + row / g.group : -1;
      const uint32_t s_tile = tmem + lane_off + kColS + 128 * blk, o_cols = tmem + lane_off + 128 * blk;
      // weights are 2^(score + EV - from): `from` is the running maximum, or 0 (none yet)
      float from = 0.f;
      for (int t = 0; t < n && ok; ++t) {
        const uint32_t k = t_base + t;
        const int t0 = (r0 + t) * kTok;
        // S_b(t) complete: so is every MMA issued before it, W_b(t - 1) V included
        ok = warp_wait(ms.s_full[blk], k, abort_flag);
        if (!ok) break;
        fence_after_sync();
        const float4* sc = reinterpret_cast<const float4*>(ms.scales[k % kScaleSlots]);  // [half][2^EK, EV, 2^-EV]
        auto load = [&](float (&s)[kPart], int part) {
#pragma unroll
          for (int c = 0; c < kPart / 16; ++c) {
            float v[16];
            tmem_ld16(s_tile + kPart * part + 16 * c, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) s[16 * c + i] = v[i];
          }
          tmem_wait_ld();
          if (t0 + kPart * part + kPart - 1 > qpos) {  // mask what the row may not see
#pragma unroll
            for (int c = 0; c < kPart; ++c)
              if (t0 + kPart * part + token_of(c) > qpos) s[c] = -CUDART_INF_F;
          }
        };
        // the largest score + EV: the largest product of each block, then its scales
        float top = -CUDART_INF_F;
        auto highest = [&](const float (&s)[kPart], int part) {
          const float4 ks4 = sc[3 * part], ev4 = sc[3 * part + 1];
          const float ks[4] = {ks4.x, ks4.y, ks4.z, ks4.w}, ev[4] = {ev4.x, ev4.y, ev4.z, ev4.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {  // block q of the half: columns 32 (q / 2) + 4 (q % 2) + 8 t + i
            const int c = 32 * (q >> 1) + 4 * (q & 1);
            float m0 = max3(s[c], s[c + 1], s[c + 2]), m1 = max3(s[c + 3], s[c + 8], s[c + 9]);
            m0 = max3(m0, s[c + 10], s[c + 11]), m1 = max3(m1, s[c + 16], s[c + 17]);
            m0 = max3(m0, s[c + 18], s[c + 19]), m1 = max3(m1, s[c + 24], s[c + 25]);
            m0 = max3(m0, s[c + 26], s[c + 27]);
            top = fmaxf(top, fmaf(fmaxf(m0, m1), q_scale * ks[q], ev[q]));
          }
        };
        float s[kPart];
        load(s, 1);
        highest(s, 1);
        load(s, 0);
        highest(s, 0);
        const float above = top - (m_run == kNone ? -CUDART_INF_F : m_run);  // (NaN where nothing is seen: no move)
        if (__any_sync(0xffffffffu, above > kReach)) {
          float alpha = 1.f;
          if (above > kReach) {
            from = top - kLift;
            alpha = ex2(m_run - from);
            m_run = from;
            l_run *= alpha;
          }
          if (t > 0) {  // O *= alpha (the warp's rows)
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
        }
        const bool large = __any_sync(0xffffffffu, fabsf(from) > kLarge);  // the difference needs the rounded product
#pragma unroll 1  // (unrolled, the second half's registers spill: 1.84 -> 2.03 ms at 8 x 1,024 over 15K)
        for (int part = 0; part < 2; ++part) {
          if (part == 1) load(s, 1);
          const float4 ks4 = sc[3 * part], ev4 = sc[3 * part + 1], dn4 = sc[3 * part + 2];
          const float ks[4] = {ks4.x, ks4.y, ks4.z, ks4.w}, ev[4] = {ev4.x, ev4.y, ev4.z, ev4.w};
          const float dn[4] = {dn4.x, dn4.y, dn4.z, dn4.w};
          if (large) {
#pragma unroll
            for (int c = 0; c < kPart; ++c) {
              const int q = 2 * (c >> 5) + (c >> 2 & 1);
              s[c] = fmaf(s[c], q_scale * ks[q], ev[q]) - from;
            }
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint64_t f = pair(q_scale * ks[q], q_scale * ks[q]), d = pair(ev[q] - from, ev[q] - from);
#pragma unroll
              for (int t4 = 0; t4 < 4; ++t4) {
                const int c = 32 * (q >> 1) + 4 * (q & 1) + 8 * t4;
                fma2(s[c], s[c + 1], f, d);
                fma2(s[c + 2], s[c + 3], f, d);
              }
            }
          }
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
            tmem_st16u(s_tile + kPart * part + 16 * half, pw);
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              float lo, hi;
              unpair(sum[q], lo, hi);
              l_run = fmaf(lo + hi, dn[2 * half + q], l_run);
            }
          }
        }
        tmem_wait_st();
        fence_before_sync();
        warp_arrive(ms.p_full[blk]);
      }
      if (ok) ok = warp_wait(ms.o_done[blk], done_frags, abort_flag);
      fence_after_sync();
      if (!ok && lane == 0 && a.status) atomicOr(a.status, RQ_STATUS_TIMEOUT);
    } else if (warp < kSoftWarps + kCodeWarps) {
      // ================= codes =================
      // warp dw takes the keys of block dw of a half tile, and half of the dims of the values of blocks
      // p16 and p16 + 1
      const int dw = warp & 3, p16 = dw & 2, g8 = lane >> 2, t4 = lane & 3;
      const int kr = 32 * (dw >> 1) + 8 * (g8 >> 1) + 4 * (dw & 1) + (g8 & 1), vd = 64 * (dw & 1) + 4 * g8;
      const uint32_t k_off[2] = {sw128(kr, 2 * t4), sw128(kr + 2, 2 * t4)};  // + 16384 (u % 2); the next chunk: ^ 16
      uint32_t v_off[4];
#pragma unroll
      for (int k4 = 0; k4 < 4; ++k4) v_off[k4] = sw128(vd + k4, t4 + 4 * (dw >> 1));  // + 4096 i
      auto widen_keys = [&](int t) {  // K(t), once S(t - 2) is done
        const uint32_t k = t_base + t;
        const int t0 = (r0 + t) * kTok;
        if (k >= kKeyStages && !(ok = warp_wait(ms.k_read[k % kKeyStages], k / kKeyStages - 1, abort_flag))) return;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint32_t rs = (2 * k + part) % kRawStages, raw = raw_ring + rs * kRawBytes + dw * kBlockBytes;
          if (!(ok = warp_wait(ms.raw_full[rs], (2 * k + part) / kRawStages, abort_flag))) return;
          // unit u: token 8 (u / 2) + g8, dims 64 (u % 2) + 16 t4 ..; the token's row is its column of S
          const uint32_t dst = k_ring + k % kKeyStages * kOperand + part * (kPart * 128);
          const bool there = t0 + kPart * part + 16 * dw < len;  // else nothing was copied
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint4 c = make_uint4(0u, 0u, 0u, 0u);
            if (there) c = lds128(raw + 16 * (32 * u + lane));
            sts128(dst + k_off[u >> 1] + (u & 1) * 16384, widen2(c.x), widen2_hi(c.x), widen2(c.y), widen2_hi(c.y));
            sts128(dst + (k_off[u >> 1] ^ 16) + (u & 1) * 16384, widen2(c.z), widen2_hi(c.z), widen2(c.w), widen2_hi(c.w));
          }
          // (S(t - 2) came behind W V(t - 3): both softmaxes are past tile t - 3, t - 4's slot is free)
          if (lane == 0) {
            uint32_t exps = 0x7F7Fu;
            if (there) asm volatile("ld.shared.u16 %0, [%1];" : "=r"(exps) : "r"(raw + kExps));
            const int ev = exp_of_byte(exps >> 8);
            float(*sc)[4] = ms.scales[k % kScaleSlots][part];
            sc[0][dw] = pow2(exp_of_byte(exps & 0xFF));
            sc[1][dw] = (float)ev;
            sc[2][dw] = pow2(-ev);
          }
        }
        fence_async_smem();
        warp_arrive(ms.k_full[k % kKeyStages]);
      };
      widen_keys(0);
      for (int t = 0; t < n && ok; ++t) {
        const uint32_t k = t_base + t;
        const int t0 = (r0 + t) * kTok;
        uint4 vc[2][4];  // [part][2 i + b]: block p16 + b, dims 32 (2 (dw % 2) + i) + 4 g8 ..
        uint32_t bad = 0u;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4& c = vc[part][i];
            c = make_uint4(0u, 0u, 0u, 0u);
            if (t0 + kPart * part + 16 * (p16 + (i & 1)) < len)
              c = lds128(raw_ring + (2 * k + part) % kRawStages * kRawBytes + (p16 + (i & 1)) * kBlockBytes + kValues +
                         16 * (32 * (2 * (dw & 1) + (i >> 1)) + lane));
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4) bad |= (word(c, k4) & 0x7F7F7F7Fu) + 0x01010101u;  // bit 7 of a byte: NaN
          }
        }
        __syncwarp();
        if (lane < 2) mbar_arrive(smem_addr(&ms.raw_empty[(2 * k + lane) % kRawStages]));  // the warp has read its codes
        if (__any_sync(0xffffffffu, (bad & 0x80808080u) != 0u) || t0 + kTok > len) {
          // bytes past the sequence may be anything; a NaN value goes to the rows that see it at the end
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int part = j >> 2, i = j & 3;
            uint32_t w[4];
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4) {
              w[k4] = word(vc[part][i], k4);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int p = t0 + kPart * part + 16 * (p16 + (i & 1)) + 2 * t4 + (c & 1) + 8 * (c >> 1);
                const bool isnan = (w[k4] >> (8 * c) & 0x7Fu) == 0x7Fu;
                if (isnan && p < len) {
                  atomicMin(&ms.nan_from[32 * (2 * (dw & 1) + (i >> 1)) + 4 * g8 + k4], p);
                  ms.any_nan = 1;
                }
                if (isnan || p >= len) w[k4] &= ~(0xFFu << (8 * c));
              }
            }
            vc[part][i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        // the next keys while the values' stage is still read
        if (t + 1 < n) widen_keys(t + 1);
        // W V(t - 1) of both blocks is done, whose values stand here
        if (!ok || (k > 0 && !(ok = warp_wait(ms.v_read, k - 1, abort_flag)))) break;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const uint32_t dst = v_ring + part * (kOperand / 2);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4) {
              const uint32_t wa = word(vc[part][2 * i], k4), wb = word(vc[part][2 * i + 1], k4);
              sts128(dst + v_off[k4] + 4096 * i, widen2(wa), widen2_hi(wa), widen2(wb), widen2_hi(wb));
            }
          }
        }
        fence_async_smem();
        warp_arrive(ms.v_full);
      }
      if (!ok && lane == 0 && a.status) atomicOr(a.status, RQ_STATUS_TIMEOUT);
    } else if (warp == kMmaWarp) {
      // ================= MMA issue =================
      const uint32_t id = idesc_f16(kHalf, 128);  // S: N = 128 tokens; O: N = 128 dims
      bool issued = false;
      auto wait = [&](uint64_t& bar, uint32_t parity) { return ok = warp_wait(bar, parity, abort_flag); };
      auto s_mmas = [&](int bb, uint32_t k) {  // S_b of tile k
        const uint32_t q_at = q_ops + 32768 * bb, k_at = k_ring + k % kKeyStages * kOperand;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)
          elect_mma_ss(tmem + kColS + 128 * bb, sdesc(q_at + (ks >> 2) * 16384 + (ks & 3) * 32),
                       sdesc(k_at + (ks >> 2) * 16384 + (ks & 3) * 32), id, ks > 0);
        elect_commit(smem_addr(&ms.s_full[bb]));
        issued = true;
      };
      if (wait(ms.q_full, done_frags) && wait(ms.k_full[t_base % kKeyStages], t_base / kKeyStages)) {
        fence_after_sync();
        s_mmas(0, t_base);
        s_mmas(1, t_base);
        elect_commit(smem_addr(&ms.k_read[t_base % kKeyStages]));
      }
      for (int t = 0; t < n && ok; ++t) {
        const uint32_t k = t_base + t;
        const bool next = t + 1 < n;
        if (!wait(ms.v_full, k)) break;
        if (next && !wait(ms.k_full[(k + 1) % kKeyStages], (k + 1) / kKeyStages)) break;
#pragma unroll
        for (int bb = 0; bb < 2; ++bb) {
          if (!wait(ms.p_full[bb], k)) break;
          fence_after_sync();
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)  // tokens 16 ks ..: W 64 columns past S's for the second half
            elect_mma_ts(tmem + 128 * bb, tmem + kColS + 128 * bb + 64 * (ks >> 2) + 8 * (ks & 3),
                         sdesc(v_ring + (ks >> 2) * (kOperand / 2) + (ks & 3) * 32), id, t > 0 || ks > 0);
          if (bb == 1) elect_commit(smem_addr(&ms.v_read));
          if (next)
            s_mmas(bb, k + 1);  // over the same columns, behind the MMAs that read them
          else
            elect_commit(smem_addr(&ms.o_done[bb]));
        }
        if (ok && next) elect_commit(smem_addr(&ms.k_read[(k + 1) % kKeyStages]));
      }
      if (!ok) {
        if (issued) {  // nothing may be running when the tensor memory is freed
          elect_commit(smem_addr(&ms.drain));
          for (int i = 0; i < kWaitLimit; ++i)
            if (mbar_test(smem_addr(&ms.drain), 0u)) break;
        }
        if (lane == 0 && a.status) atomicOr(a.status, RQ_STATUS_TIMEOUT);
      }
    } else if (warp == kCopyWarp) {
      // ================= copies of the cache's blocks =================
      const int32_t* table = a.block_table + (size_t)b * a.max_pages;
      const int last = min(len, (r0 + n) * kTok);  // the fragment's tokens end here
      auto pages_of = [&](int batch) {  // pages of 32 blocks, a lane each
        const int p = r0 * kTok + 16 * (32 * batch + lane);
        if (p >= last) return 0;
        int page = __ldg(table + p / g.page_size);
        if (page < 0 || page >= g.num_pages) {
          if (a.status) atomicOr(a.status, RQ_STATUS_BAD_PAGE);
          page = 0;
        }
        return page;
      };
      int now = pages_of(0), later = pages_of(1);
      for (int t2 = 0; t2 < 2 * n && ok; ++t2) {
        const uint32_t k2 = 2 * t_base + t2, rs = k2 % kRawStages;
        if (t2 > 0 && (t2 & 7) == 0) {
          now = later;
          later = pages_of((t2 >> 3) + 1);
        }
        if (k2 >= kRawStages && !(ok = warp_wait(ms.raw_empty[rs], k2 / kRawStages - 1, abort_flag))) break;
        fills = k2 + 1;
        const uint32_t bar = smem_addr(&ms.raw_full[rs]);
        const int p = r0 * kTok + kPart * t2, count = min(4, max(0, (last - p + 15) / 16));
        const int page = __shfl_sync(0xffffffffu, now, 4 * (t2 & 7) + (lane & 3));
        if (lane == 0)
          asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(count * kBlockBytes) : "memory");
        __syncwarp();
        if (lane < count) {
          const int in_page = (p + 16 * lane) % g.page_size / 16;
          const uint8_t* src = a.pages + ((size_t)page * g.num_kv_heads + h) * g.page_bytes + (size_t)in_page * kBlockBytes;
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                  raw_ring + rs * kRawBytes + lane * kBlockBytes),
              "l"(src), "r"(kBlockBytes), "r"(bar)
              : "memory");
        }
      }
      if (!ok) {
        if (lane == 0 && a.status) atomicOr(a.status, RQ_STATUS_TIMEOUT);
      }
    }
    done_tiles += n;
    ++done_frags;
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (ms.abort) break;  // uniform: no role raises it between the barrier and here

    // ---- write the rows, or the fragment's part of them ----
    const bool whole = ms.f.whole;
    auto slot_of = [&](long long c) {  // range c's first fragment, or the last of the unit's first range
      return a.ws + (2 * c + (c == ms.f.range ? ms.f.range_last : 0)) * kSlotFloats;
    };
    auto store16 = [&](int c, const float (&y)[16]) {  // dims 16 c .. of the thread's row
      uint4* const dst = reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.out) + row_offset()) + 2 * c;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        dst[i] = make_uint4(rope::pack2<T>(y[8 * i], y[8 * i + 1]), rope::pack2<T>(y[8 * i + 2], y[8 * i + 3]),
                            rope::pack2<T>(y[8 * i + 4], y[8 * i + 5]), rope::pack2<T>(y[8 * i + 6], y[8 * i + 7]));
    };
    const int srow = kHalf * blk + brow;
    if (warp < kSoftWarps) {
      const int qpos = valid ? len - a.T + row / g.group : -1;
      const float inv = whole ? 1.f / l_run : 1.f;
      // a row that sees nothing, or only scores of minus infinity (their softmax is 0 / 0)
      const float empty = whole && qpos >= 0 ? CUDART_NAN_F : 0.f;
      float* const slot = slot_of(blockIdx.x);
#pragma unroll 2
      for (int c = 0; c < kHeadDim / 16; ++c) {
        float y[16];
        __syncwarp();
        tmem_ld16(tmem + lane_off + 128 * blk + 16 * c, y);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = l_run == 0.f ? empty : y[i] * inv;
        if (ms.any_nan) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (ms.nan_from[16 * c + i] <= qpos) y[i] = CUDART_NAN_F;
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
    }
    if (!whole) {
      const int frags = ms.f.frags;
      const long long cf = ms.f.range;
      __threadfence();
      __syncthreads();
      if (tid == 0) ms.last = atomicAdd(a.cnt + cf, 1) == frags - 1;
      __syncthreads();
      if (ms.last) {
        __threadfence();
        if (tid == 0) a.cnt[cf] = 0;  // as every launch finds it
        if (warp < kSoftWarps) {
          // a fragment's 64 dims and its m and l load together, the sums grow with the maximum
#pragma unroll 1
          for (int d = 0; d < 2; ++d) {
            float y[64], top = kNone, sum = 0.f;
#pragma unroll
            for (int i = 0; i < 64; ++i) y[i] = 0.f;
#pragma unroll 1
            for (int f = 0; f < frags; ++f) {
              const float* s = slot_of(cf + f);
              const float mf = __ldcg(s + kRows * kHeadDim + srow), lf = __ldcg(s + kRows * kHeadDim + kRows + srow);
              const float t = fmaxf(top, mf), wa = ex2(top - t), w = ex2(mf - t);
              top = t;
              sum = fmaf(sum, wa, lf * w);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(s) + (16 * d + i) * kRows + srow);
                y[4 * i] = fmaf(y[4 * i], wa, v.x * w), y[4 * i + 1] = fmaf(y[4 * i + 1], wa, v.y * w);
                y[4 * i + 2] = fmaf(y[4 * i + 2], wa, v.z * w), y[4 * i + 3] = fmaf(y[4 * i + 3], wa, v.w * w);
              }
            }
            const float inv = sum == 0.f ? (len - a.T + row / g.group >= 0 ? CUDART_NAN_F : 0.f) : 1.f / sum;
            if (valid) {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                float z[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) z[i] = y[16 * c + i] * inv;
                store16(4 * d + c, z);
              }
            }
          }
        }
      }
    }
    __syncthreads();  // ms.f and nan_from are written again
  }
  if (ms.abort && warp == kCopyWarp) {  // copies in flight land before the block ends
    for (uint32_t i = fills > kRawStages ? fills - kRawStages : 0; i < fills; ++i)
      for (int w = 0; w < kWaitLimit; ++w)
        if (mbar_test(smem_addr(&ms.raw_full[i % kRawStages]), (i / kRawStages) & 1)) break;
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(*(volatile uint32_t*)&ms.tmem, 512);
}

}  // namespace

size_t block_extend_workspace(int num_sms) { return 2 * (size_t)num_sms * kSlotFloats; }  // two slots a CTA

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
