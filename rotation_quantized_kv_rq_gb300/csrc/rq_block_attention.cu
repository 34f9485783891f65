// Attention over the 8-bit block-scaled cache: decode, chain verify and tree verify.
//
//   out = softmax(sm_scale q K^T) V,  K = code * 2^EK, V = code * 2^EV (a block's exponents)
//
// For a tile of 16 tokens (one block) and 8 query rows of a kv head, with e4m3 codes widened to
// fp16 (exact) as the A operands of m16n8k16 MMAs and f32 accumulators:
//   S^T = code_K q^T;   t = S 2^EK sm_scale log2(e) + EV - m;   w = 2^t
//   O^T += code_V^T w;   l += w 2^-EV;   out = O / l
// The value scale is part of the weight's exponent, so codes are never multiplied by it, and m follows
// the running maximum of score + EV: w, rounded to fp16 for the MMA (2^-11 of it), is then largest
// where a token weighs most in the output, whatever the scales (its range: rq_block.cuh).  Queries are
// fp16 as they are; a bf16 row is brought into fp16's range by a power of two.
//
// What bounds it: the cache is read once, 257 bytes a (token, kv head), against 4 MMAs' worth of
// work; so the design keeps copies in flight.  A block is one 4112-byte bulk copy into a ring of
// the warp's own, and no thread of the CTA waits for another inside a fragment; an SM has 48 tiles
// in flight.  With many units, four CTAs of four warps share an SM, so that one's opening and
// joining hide behind the others' copies; with fewer units than SMs one CTA of 16 warps does, which
// cuts a unit into a quarter of the parts to join (1 x 32K: 19 instead of 76).  Rows of a kv head beyond
// 8 (group > 8, verify) share the widened tile: up to three n-tiles of 8 rows a warp, with the
// registers for 12 and 8 warps an SM and the queries in shared memory.  Three n-tiles are bound by the
// chain wait - widen - MMA - softmax - MMA of two warps a quarter SM (0.36 instructions a cycle, the MMAs
// busy 31%).  8 x 16K, 6 rows x 4 heads: 71 us (3.8 TB/s).  Beside 69 us of the same kernel with an older
// partition: 72 with 12 warps (spills), 74 with the next tile's products before this one's softmax, 74 with the
// values loaded a quarter at a time.  Two n-tiles with 12 warps spill 26 to 32 bytes; 8 x 16K, 4 rows x 4
// heads: 55 us (4.9 TB/s).
//
// Work is cut evenly: a unit is (sequence, kv head, group of n-tiles) and costs one round per tile of
// each warp; the rounds of all units in order are cut into one range per CTA, on the device from
// seq_lens.  A unit that spans ranges is joined by the last of its CTAs to finish, in the order of
// the ranges (the result does not depend on which came last).  A CTA has at most two such
// fragments, its first and its last, so the workspace is two slots and one counter a CTA.  Where up to
// 32 sequences have no more units than CTAs, ranges that lie in one unit each are taken instead, if they
// are at most 6 rounds longer (us: 4 x 4K + 6 rows x 4 heads 23.9 -> 19.4, 1 x 16K + 8 x 8 28.4 -> 23.1,
// 8 x 4K decode 19.4 -> 16.8; 8 x 16K + 6, where they are 10 longer, 1 more for the search).  Short
// calls are chains of memory latencies (0.6 us each), so what can load together does: a fragment's
// page ids with its queries, the parts to join by bulk copies of a chunk at once.
#include <math_constants.h>

#include <type_traits>

#include "../../include/rq.h"
#include "rq_block.cuh"
#include "rq_rope.cuh"
#include "rq_tc.cuh"

namespace rq {
namespace {

using namespace block;

constexpr int kOpening = 6;         // rounds that a CTA's second fragment costs (opening, joining), about
constexpr int kRowStride = 132;     // floats per joined row (128 and padding)

constexpr int kRowBytes = kRowStride * 4;  // a joined row: 128 sums, the maximum, the weights' sum

// W warps a CTA; 16, 12 or 8 warps an SM for 1, 2 or 3 n-tiles
__host__ __device__ constexpr int warps_per_sm(int nt) { return nt == 1 ? 16 : nt == 2 ? 12 : 8; }
__host__ __device__ constexpr int stages(int nt) { return 48 / warps_per_sm(nt); }  // tiles of a warp's ring
constexpr int ring_bytes(int nt, int w) { return w * stages(nt) * kBlockBytes; }
constexpr int smem_bytes(int nt, int w) { return ring_bytes(nt, w) + (w * stages(nt) + 1) * 8; }

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool bounded_wait(uint32_t bar, uint32_t parity) {
  for (int i = 0; i < tc::kWaitLimit; ++i)
    if (tc::mbar_test(bar, parity)) return true;
  return false;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
// 1.0 in fp16 for each of the two codes that is NaN, else 0
__device__ __forceinline__ uint32_t nan2(uint32_t codes) {
  return ((codes & 0x7Fu) == 0x7Fu ? 0x3C00u : 0u) | ((codes & 0x7F00u) == 0x7F00u ? 0x3C000000u : 0u);
}
// the codes with NaNs replaced by 0
__device__ __forceinline__ uint32_t without_nan4(uint32_t codes) {
  const uint32_t is = __vcmpeq4(codes & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
  return codes & ~is;
}

// The partition: rounds of sequence b's units, and the sums over sequences.
struct Plan {
  int tiles, rounds;
};
template <int W>
__device__ __forceinline__ Plan plan_of(int len, int step = 1) {
  Plan p;
  p.tiles = (len + kBlockTokens - 1) / kBlockTokens;
  p.rounds = max(1, (p.tiles + W - 1) / W);  // an empty sequence's rows are written too
  if (step > 1) p.rounds = (p.rounds + step - 1) / step * step;
  return p;
}

template <int NT, int W, typename T>
__global__ void __launch_bounds__(32 * W, warps_per_sm(NT) / W) splitk_kernel(const Geometry g, const AttnArgs a) {
  constexpr int S = stages(NT), kRows = 8 * NT, kThreads = 32 * W;
  constexpr int kLens = 32 * W;  // sequences whose lengths are kept
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ long long s_sum[W], s_begin;  // rounds per warp's sequences; first sequence's rounds before it
  __shared__ int s_seq, s_last, s_len[kLens], s_parts;  // s_parts: ranges of the launch
  __shared__ float s_m[W][kRows], s_l[W][kRows];
  __shared__ uint4 s_q[NT > 1 ? NT * 4 * 32 : 1];  // query fragments [n][ks / 2][lane], the same in every warp
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gq = lane >> 2, tq = lane & 3;
  const int cap = a.max_pages * g.page_size, groups = (a.n_tiles_n + NT - 1) / NT;
  const int per_seq = g.num_kv_heads * groups;  // units of a sequence

  auto load_length = [&](int b, bool report) {
    int len = __ldg(a.seq_lens + b);
    if (len < 0 || len > cap || (len > 0 && len < a.T)) {
      if (report && a.status) atomicOr(a.status, RQ_STATUS_BAD_LEN);
      len = len < 0 ? 0 : min(len, cap);
    }
    return len;
  };
  auto length = [&](int b) { return a.B <= kLens ? s_len[b] : load_length(b, false); };

  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem) + warp * S * kBlockBytes;
  const uint32_t bars = (uint32_t)__cvta_generic_to_shared(smem) + W * S * kBlockBytes + warp * S * 8;
  const uint32_t join_bar = (uint32_t)__cvta_generic_to_shared(smem) + W * S * (kBlockBytes + 8);
  if (lane == 0) {
    for (int i = 0; i < S; ++i) tc::mbar_init(bars + 8 * i, 1);
    if (warp == 0) tc::mbar_init(join_bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }

  // ---- the CTA's range of rounds ----
  long long total, at;
  int b, step = 1;
  auto part_begin = [&](long long c) { return c * total / s_parts; };
  auto part_of = [&](long long x) { return ((x + 1) * s_parts - 1) / total; };  // the range that holds round x
  long long x;
  if (a.B <= 32) {  // a lane has a sequence, in every warp alike: no barrier before the first copies
    const int len = lane < a.B ? load_length(lane, blockIdx.x == 0 && warp == 0) : 0;
    s_len[lane] = len;  // (all warps write the same)
    int r = lane < a.B ? plan_of<W>(len).rounds : 0;
    total = (long long)__reduce_add_sync(0xffffffffu, r) * per_seq;
    // A range that crosses into a second unit opens and joins twice.  Ranges of `step` rounds, each in
    // one unit, if they are not longer by more than that costs (and there is not work for long).
    int parts = 0;
    if (a.B * per_seq <= (int)gridDim.x && total > gridDim.x && total < 1 << 18) {
      const uint32_t even = ((uint32_t)total + gridDim.x - 1) / gridDim.x;
      const uint32_t recip = 0xFFFFFFFFu / (even + (lane & 7)) + 1;  // n / d is exact so for n d < 2^32
#pragma unroll
      for (int k = kOpening; k >= 0; --k) {
        const uint32_t rec = __shfl_sync(0xffffffffu, recip, k), up = r + even + k - 1;
        const int pieces = __reduce_add_sync(0xffffffffu, even + k == 1 ? up : __umulhi(up, rec)) * per_seq;
        if (pieces <= (int)gridDim.x) step = even + k, parts = pieces;
      }
    }
    if (step > 1) {
      r = (r + step - 1) / step * step;
      total = (long long)parts * step;
      if ((int)blockIdx.x >= parts) return;
      x = (long long)blockIdx.x * step;
    } else {
      parts = (int)min((long long)gridDim.x, total);
      if ((int)blockIdx.x >= parts) return;
      x = blockIdx.x * total / parts;
    }
    s_parts = parts;
    __syncwarp();
    int upto = r;  // inclusive scan
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    b = __ffs(__ballot_sync(0xffffffffu, x < (long long)upto * per_seq)) - 1;
    at = (long long)__shfl_sync(0xffffffffu, upto - r, b) * per_seq;
  } else {
    const int chunk = (a.B + kThreads - 1) / kThreads;
    long long mine = 0;
    for (int i = tid * chunk; i < min(a.B, (tid + 1) * chunk); ++i) {
      const int len = load_length(i, blockIdx.x == 0);
      if (i < kLens) s_len[i] = len;
      mine += plan_of<W>(len).rounds;
    }
    long long upto = mine;  // inclusive scan over the threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) s_sum[warp] = upto;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w == warp) upto += total;
      total += s_sum[w];
    }
    total *= per_seq;
    const int parts = (int)min((long long)gridDim.x, total);
    if ((int)blockIdx.x >= parts) return;
    s_parts = parts;
    __syncwarp();
    x = part_begin(blockIdx.x);
    if (x >= (upto - mine) * per_seq && x < upto * per_seq) {
      long long begin = (upto - mine) * per_seq;
      int i = tid * chunk;
      for (; chunk > 1; ++i) {
        const long long r = (long long)plan_of<W>(length(i)).rounds * per_seq;
        if (x < begin + r) break;
        begin += r;
      }
      s_begin = begin;
      s_seq = i;
    }
    __syncthreads();
    at = s_begin;
    b = s_seq;
  }
  const long long end = step > 1 ? x + step : part_begin(blockIdx.x + 1ll);

  const uint32_t s_q_addr = (uint32_t)__cvta_generic_to_shared(s_q) + 16 * lane;
  uint32_t issued = 0, done = 0;  // tiles of this warp so far: ring positions and parities
  uint32_t joins = 0;
  bool failed = false;
  while (x < end) {
    // ---- the fragment: rounds r0 .. r1 - 1 of unit u of sequence b ----
    const int len = length(b);
    const Plan pl = plan_of<W>(len, step);
    const int u = (int)((x - at) / pl.rounds), r0 = (int)((x - at) % pl.rounds);
    const int r1 = (int)min((long long)pl.rounds, r0 + (end - x));
    const int h = u / groups, row0 = (u % groups) * kRows;
    const int first = r0 * W + warp;  // the warp's tiles: first, first + W, ...
    const int last = min(pl.tiles, r1 * W);
    const int count = first < last ? (last - first + W - 1) / W : 0;
    const int32_t* table = a.block_table + (size_t)b * a.max_pages;

    // the warp's queries, rows past the last one as that one (they are not written), and the pages of
    // its first 64 tiles: all loads in flight together
    uint4 raw[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = min(row0 + 8 * n + gq, a.rows - 1), j = row / g.group, head = h * g.group + row % g.group;
      const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q) +
                                                        (((size_t)b * a.T + j) * g.num_q_heads + head) * kHeadDim);
#pragma unroll
      for (int i = 0; i < 4; ++i) raw[n][i] = __ldg(src + 8 * (i >> 1) + 2 * tq + (i & 1));
    }
    // page of tile first + W * i, for i in the lane's place of the current and next 32
    auto page_at = [&](int i) { return i < count ? __ldg(table + (first + W * i) * kBlockTokens / g.page_size) : 0; };
    int pages_now = page_at(lane), pages_next = page_at(32 + lane);
    int batch = 0;
    auto issue = [&](int i) {  // tile i of the warp, by the whole warp
      if ((i >> 5) != batch) {
        batch = i >> 5;
        pages_now = pages_next;
        pages_next = page_at(32 * (batch + 1) + lane);
      }
      int page = __shfl_sync(0xffffffffu, pages_now, i & 31);
      if (lane == 0) {
        if (page < 0 || page >= g.num_pages) {
          if (a.status) atomicOr(a.status, RQ_STATUS_BAD_PAGE);
          page = 0;
        }
        const int in_page = (first + W * i) * kBlockTokens % g.page_size / kBlockTokens;
        const uint32_t s = issued % S;
        expect_bytes(bars + 8 * s, kBlockBytes);
        bulk_copy(ring + s * kBlockBytes,
                  a.pages + ((size_t)page * g.num_kv_heads + h) * g.page_bytes + (size_t)in_page * kBlockBytes, kBlockBytes,
                  bars + 8 * s);
      }
      ++issued;
    };
    if (!failed)
      for (int i = 0; i < min(S, count); ++i) issue(i);

    // ---- queries: B fragments, lane (row gq, dims 64 (ks / 4) + 16 tq + 4 (ks % 4) ..) ----
    uint32_t qf[NT][8][2];
    float qs[NT][2];  // factor of the scores of columns 2 tq, 2 tq + 1
    int lim[NT][2];   // last visible position of those columns' rows
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      constexpr bool kBf16 = !std::is_same<T, __half>::value;
      float top = 0.f;
      if constexpr (kBf16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 v = rope::unpack2<T>(word(raw[n][i >> 2], i & 3));
          top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      }
      const RowScale scale = row_scale<kBf16>(top, g.sm_scale * 1.44269504088896340736f);
      if constexpr (kBf16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 v = rope::unpack2<T>(word(raw[n][i >> 2], i & 3));
          qf[n][i >> 1][i & 1] = rope::pack2<__half>(v.x * scale.down, v.y * scale.down);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) qf[n][i >> 1][i & 1] = word(raw[n][i >> 2], i & 3);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        qs[n][c] = __shfl_sync(0xffffffffu, scale.factor, 4 * (2 * tq + c));
        lim[n][c] = len - a.T + (row0 + 8 * n + 2 * tq + c) / g.group;
      }
    }

    if constexpr (NT > 1) {  // the fragment's queries are the same in every warp: kept once
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if ((4 * n + k) % W == warp)
            s_q[(4 * n + k) * 32 + lane] = make_uint4(qf[n][2 * k][0], qf[n][2 * k][1], qf[n][2 * k + 1][0], qf[n][2 * k + 1][1]);
      }
      __syncthreads();
    }

    float o[NT][8][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = kNone;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
    }

    for (int i = 0; i < count; ++i) {
      const uint32_t st = done % S, tile = ring + st * kBlockBytes;
      if (failed || !__all_sync(0xffffffffu, bounded_wait(bars + 8 * st, (done / S) & 1))) {
        if (!failed && lane == 0 && a.status) atomicOr(a.status, RQ_STATUS_TIMEOUT);
        for (; done != issued; ++done) bounded_wait(bars + 8 * (done % S), (done / S) & 1);  // its own copies
        failed = true;
        break;
      }
      ++done;
      const int t0 = (first + W * i) * kBlockTokens;
      // rows see different parts of the tile: draft 0 is every chain row's, but a tree row's only by its bit
      const bool tail = t0 + kBlockTokens - 1 > len - a.T - (a.tree_mask ? 1 : 0);
      uint32_t exps;
      asm volatile("ld.shared.u16 %0, [%1];" : "=r"(exps) : "r"(tile + kExps));
      const float ks = pow2(exp_of_byte(exps & 0xFF));
      const int ev = exp_of_byte(exps >> 8);

      float s[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint4 lo = lds128(tile + 16 * (32 * half + lane)), hi = lds128(tile + 16 * (32 * (2 + half) + lane));
        uint4 qw[NT];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if constexpr (NT > 1) {
            if ((k & 1) == 0) {
#pragma unroll
              for (int n = 0; n < NT; ++n) qw[n] = lds128(s_q_addr + 512 * (4 * n + 2 * half + (k >> 1)));
            }
          }
          const uint32_t w0 = word(lo, k), w1 = word(hi, k);
          const uint32_t a0 = widen2(w0), a1 = widen2(w1), a2 = widen2_hi(w0), a3 = widen2_hi(w1);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if constexpr (NT > 1)
              mma(s[n], a0, a1, a2, a3, word(qw[n], 2 * (k & 1)), word(qw[n], 2 * (k & 1) + 1));
            else
              mma(s[n], a0, a1, a2, a3, qf[n][4 * half + k][0], qf[n][4 * half + k][1]);
          }
        }
      }
      if (tail) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int p = t0 + gq + 8 * (c >> 1), row = row0 + 8 * n + 2 * tq + (c & 1);
            bool seen = p <= lim[n][c & 1];
            if (a.tree_mask) {
              const int d = p - (len - a.T);
              seen = p < len && (d < 0 || (row < a.rows &&
                                           (__ldg(a.tree_mask + (size_t)b * a.T + row / g.group) >> d & 1)));
            }
            if (!seen) s[n][c] = -CUDART_INF_F;
          }
        }
      }
      const float fev = (float)ev, down = pow2(-ev);
      float t[NT][4];
      bool past = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          t[n][c] = fmaf(s[n][c], qs[n][c & 1] * ks, fev);  // rounded once: t - m <= 0 for the m it gives, at any size
          past = past || t[n][c] - m[n][c & 1] > kReach;
        }
      }
      if (__any_sync(0xffffffffu, past)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = fmaxf(t[n][c], t[n][c + 2]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float m_new = fmaxf(m[n][c], top - kLift), alpha = ex2(m[n][c] - m_new);
            m[n][c] = m_new;
            l[n][c] *= alpha;
#pragma unroll
            for (int d = 0; d < 8; ++d) o[n][d][c] *= alpha, o[n][d][c + 2] *= alpha;
          }
        }
      }
      uint32_t p[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float w0 = ex2(t[n][0] - m[n][0]), w1 = ex2(t[n][1] - m[n][1]);
        const float w2 = ex2(t[n][2] - m[n][0]), w3 = ex2(t[n][3] - m[n][1]);
        l[n][0] = fmaf(w0 + w2, down, l[n][0]);
        l[n][1] = fmaf(w1 + w3, down, l[n][1]);
        p[n][0] = transpose8x8(rope::pack2<__half>(w0, w1));
        p[n][1] = transpose8x8(rope::pack2<__half>(w2, w3));
      }
      uint4 v[4];
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4) v[q4] = lds128(tile + kValues + 16 * (32 * q4 + lane));
      if (tail) {
        // bytes past the sequence may be anything; a NaN value of a token that some rows see and
        // others do not reaches those that see it only
        uint32_t keep = 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (t0 + 2 * tq + (k & 1) + 8 * (k >> 1) < len) keep |= 0xFFu << (8 * k);
        bool any_nan = false;
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          v[q4].x &= keep, v[q4].y &= keep, v[q4].z &= keep, v[q4].w &= keep;
#pragma unroll
          for (int k = 0; k < 4; ++k) any_nan = any_nan || without_nan4(word(v[q4], k)) != word(v[q4], k);
        }
        if (__any_sync(0xffffffffu, any_nan)) {
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t w0 = word(v[q4], 2 * k), w1 = word(v[q4], 2 * k + 1);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                float hit[4] = {0.f, 0.f, 0.f, 0.f};
                mma(hit, nan2(w0), nan2(w1), nan2(w0 >> 16), nan2(w1 >> 16), p[n][0], p[n][1]);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  if (hit[c] > 0.f) o[n][2 * q4 + k][c] = CUDART_NAN_F;
              }
            }
            v[q4].x = without_nan4(v[q4].x), v[q4].y = without_nan4(v[q4].y);
            v[q4].z = without_nan4(v[q4].z), v[q4].w = without_nan4(v[q4].w);
          }
        }
      }
#pragma unroll
      for (int q4 = 0; q4 < 4; ++q4) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t w0 = word(v[q4], 2 * k), w1 = word(v[q4], 2 * k + 1);
          const uint32_t a0 = widen2(w0), a1 = widen2(w1), a2 = widen2_hi(w0), a3 = widen2_hi(w1);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma(o[n][2 * q4 + k], a0, a1, a2, a3, p[n][0], p[n][1]);
        }
      }
      __syncwarp();  // every lane has read the stage
      if (i + S < count) issue(i + S);
    }

    // ---- join the warps ----
    const int rows = min(kRows, a.rows - row0);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], d);
        if (gq == 0) {
          s_m[warp][8 * n + 2 * tq + c] = m[n][c];
          s_l[warp][8 * n + 2 * tq + c] = l[n][c];
        }
      }
    }
    __syncthreads();  // also: every warp is done with its ring
    float* const join = reinterpret_cast<float*>(smem);  // [warp][row][kRowStride]
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = 8 * n + 2 * tq + c;
        float top = s_m[0][r];
#pragma unroll
        for (int w = 1; w < W; ++w) top = fmaxf(top, s_m[w][r]);
        const float f = ex2(m[n][c] - top);
#pragma unroll
        for (int d = 0; d < 8; ++d)  // dims 32 (d / 2) + 4 gq + 2 (d % 2), and the next
          *reinterpret_cast<float2*>(join + (warp * kRows + r) * kRowStride + 32 * (d >> 1) + 4 * gq + 2 * (d & 1)) =
              make_float2(o[n][d][c] * f, o[n][d][c + 2] * f);
      }
    }
    __syncthreads();
    const long long u0 = at + (long long)u * pl.rounds;
    const bool whole = r0 == 0 && r1 == pl.rounds;
    const long long cf = part_of(u0), cl = part_of(u0 + pl.rounds - 1);
    auto slot_of = [&](long long c) {  // a unit's fragment in range c is c's first, or the last of the first range
      return a.ws + (2 * c + (c == cf && part_begin(c) != u0 ? 1 : 0)) * (kRows * kRowStride);
    };
    auto write_row = [&](int r, float4 v, float sum) {  // a lane's four dims of a row of the output
      const int row = row0 + r, j = row / g.group, head = h * g.group + row % g.group;
      T* dst = reinterpret_cast<T*>(a.out) + (((size_t)b * a.T + j) * g.num_q_heads + head) * kHeadDim;
      if (sum == 0.f) {  // the row sees nothing, or only scores of minus infinity: their softmax is 0 / 0
        const int lo = max(0, a.T - len);  // first of the T query tokens that the sequence holds
        const bool sees = a.tree_mask ? len > a.T || (lo < a.T && __ldg(a.tree_mask + (size_t)b * a.T + j) << (64 - a.T) >> (64 - a.T + lo))
                                      : len - a.T + j >= 0;
        const float x = sees ? CUDART_NAN_F : 0.f;
        v = make_float4(x, x, x, x);
        sum = 1.f;
      }
      const float inv = 1.f / sum;
      *(reinterpret_cast<uint2*>(dst) + lane) =
          make_uint2(rope::pack2<T>(v.x * inv, v.y * inv), rope::pack2<T>(v.z * inv, v.w * inv));
    };
    for (int r = warp; r < rows; r += W) {
      float top = s_m[0][r], sum = 0.f;
#pragma unroll
      for (int w = 1; w < W; ++w) top = fmaxf(top, s_m[w][r]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        sum += s_l[w][r] * ex2(s_m[w][r] - top);
        const float4 v = *(reinterpret_cast<const float4*>(join + (w * kRows + r) * kRowStride) + lane);
        acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
      }
      if (whole) {
        write_row(r, acc, sum);
      } else {
        float* const dst = slot_of(blockIdx.x) + r * kRowStride;
        *(reinterpret_cast<float4*>(dst) + lane) = acc;
        if (lane == 0) *reinterpret_cast<float2*>(dst + kHeadDim) = make_float2(top, sum);
      }
    }
    if (!whole) {
      const int frags = (int)(cl - cf + 1);
      __threadfence();
      __syncthreads();
      if (tid == 0) s_last = atomicAdd(a.cnt + cf, 1) == frags - 1;
      __syncthreads();
      if (s_last) {
        __threadfence();
        asm volatile("fence.proxy.async;" ::: "memory");  // the other CTAs' stores, before copies of them
        if (tid == 0) a.cnt[cf] = 0;  // as every launch finds it
        constexpr int kMine = (kRows + W - 1) / W;  // rows of a warp
        float4 acc[kMine];
        float top[kMine], sum[kMine];
#pragma unroll
        for (int i = 0; i < kMine; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f), top[i] = kNone, sum[i] = 0.f;
        const int bytes = rows * kRowBytes, at_once = min(32, W * S * kBlockBytes / bytes);
        for (int f0 = 0; f0 < frags; f0 += at_once) {
          const int nf = min(at_once, frags - f0);
          if (warp == 0) {
            if (lane == 0) expect_bytes(join_bar, nf * bytes);
            __syncwarp();
            if (lane < nf)
              bulk_copy((uint32_t)__cvta_generic_to_shared(smem) + lane * bytes, slot_of(cf + f0 + lane), bytes, join_bar);
          }
          if (!bounded_wait(join_bar, joins & 1) && lane == 0 && a.status) atomicOr(a.status, RQ_STATUS_TIMEOUT);
          ++joins;
#pragma unroll
          for (int i = 0; i < kMine; ++i) {
            const int r = warp + W * i;
            if (r >= rows) break;
            const float* src = join + r * kRowStride;
            for (int f = 0; f < nf; ++f, src += rows * kRowStride) {  // in the order of the ranges
              const float2 ml = *reinterpret_cast<const float2*>(src + kHeadDim);
              const float4 v = *(reinterpret_cast<const float4*>(src) + lane);
              const float t = fmaxf(top[i], ml.x), wa = ex2(top[i] - t), wv = ex2(ml.x - t);
              top[i] = t;
              sum[i] = sum[i] * wa + ml.y * wv;
              acc[i].x = acc[i].x * wa + v.x * wv, acc[i].y = acc[i].y * wa + v.y * wv;
              acc[i].z = acc[i].z * wa + v.z * wv, acc[i].w = acc[i].w * wa + v.w * wv;
            }
          }
          tc::fence_async_smem();
          __syncthreads();  // read, before the next chunk's copies
        }
#pragma unroll
        for (int i = 0; i < kMine; ++i)
          if (warp + W * i < rows) write_row(warp + W * i, acc[i], sum[i]);
      }
    }
    tc::fence_async_smem();  // the join's accesses to the ring, before the next fragment's copies
    __syncthreads();
    x += r1 - r0;
    if (x - at == (long long)pl.rounds * per_seq) {
      at = x;
      ++b;
    }
  }
}

template <int NT, int W>
cudaError_t launch(const Geometry& g, const AttnArgs& a, int num_sms, cudaStream_t stream) {
  const int grid = num_sms * (warps_per_sm(NT) / W);
  if (g.bf16)
    splitk_kernel<NT, W, __nv_bfloat16><<<grid, 32 * W, smem_bytes(NT, W), stream>>>(g, a);
  else
    splitk_kernel<NT, W, __half><<<grid, 32 * W, smem_bytes(NT, W), stream>>>(g, a);
  return cudaGetLastError();
}

template <int NT, int W>
cudaError_t prepare() {
  constexpr int bytes = smem_bytes(NT, W);
  cudaError_t e = cudaFuncSetAttribute(splitk_kernel<NT, W, __half>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(splitk_kernel<NT, W, __nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return e;
}

// n-tiles a unit carries: as few units as three n-tiles each allow, evenly filled
int unit_tiles(int n_tiles) {
  const int units = (n_tiles + 2) / 3;
  return (n_tiles + units - 1) / units;
}

}  // namespace

size_t block_attention_workspace(int num_sms, size_t* counters) {
  const size_t row = 8 * kRowStride;
  size_t most = 2 * (size_t)num_sms * 4 * row;  // two slots a CTA: four of 8 rows an SM, or one of 16 or 24
  *counters = (size_t)num_sms * 4;
  return most;
}

cudaError_t block_attention_prepare() {
  cudaError_t e = prepare<1, 4>();
  if (e == cudaSuccess) e = prepare<1, 16>();
  if (e == cudaSuccess) e = prepare<2, 12>();
  if (e == cudaSuccess) e = prepare<3, 8>();
  return e;
}

cudaError_t launch_block_attention(const Geometry& g, AttnArgs a, int num_sms, cudaStream_t stream, cudaEvent_t ev_start,
                                   cudaEvent_t ev_end) {
  a.n_tiles_n = (a.rows + 7) / 8;
  a.nt = unit_tiles(a.n_tiles_n);
  const long long units = (long long)a.B * g.num_kv_heads * ((a.n_tiles_n + a.nt - 1) / a.nt);
  if (ev_start) cudaEventRecord(ev_start, stream);
  cudaError_t e;
  if (a.nt == 1)
    e = units < num_sms ? launch<1, 16>(g, a, num_sms, stream) : launch<1, 4>(g, a, num_sms, stream);
  else
    e = a.nt == 2 ? launch<2, 12>(g, a, num_sms, stream) : launch<3, 8>(g, a, num_sms, stream);
  if (e == cudaSuccess && ev_end) cudaEventRecord(ev_end, stream);
  return e;
}

}  // namespace rq
