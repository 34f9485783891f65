// Attention in the absorbed form over the cache of latents: decode, chain and tree verify.
//
// score = sm_scale (q_c . c + q_pe . p), out = sum softmax(score) c: keys and values are one row a token, for all heads.
// The codes are operands of the tensor cores' 8-bit MMAs as they stand in the cache, for scores (K along dims) and for the
// weighted sum (N along dims) alike; what they are multiplied with is split instead.  A query row is 2^E times e4m3
// numbers: a bf16 value's 8 bits are exactly two of 4, an fp16 value's 11 three (what falls below e4m3's smallest step is off by
// 2^-10 where the row's largest is 224 to 448).  A weight times its token's scale is an e5m2 number, which brings the range, and
// one (bf16) or two (fp16) e4m3 numbers for the rest: 2^-8 or 2^-12 of it.  8-bit MMAs run at twice the 16-bit rate, so that two
// passes cost what one over widened codes would, without the widening.  Position parts are a 16-bit MMA into the same
// accumulators.
//
// What bounds it: 641 cache bytes a token against 2 * 1,088 flops a (token, row); from some 90 rows on the tensor cores.
//
// A pair of CTAs (two SMs) takes 128 query rows of one sequence (64 to a CTA) and walks the cache in tiles of 256 tokens; its
// MMAs span both (M = 128, N = 256: 64 to 66 cycles, the full rate; one CTA with M = 128 has no room: 512 f32 columns of
// output a row are all of its tensor memory).  A CTA holds 128 of a tile's tokens as keys, five slots of 16 KB (128 dims
// each, and the position parts), and 256 of the 512 dims of all its tokens as values, four slots (64 tokens each).  Roles:
//   softmax (warps 0-7 of both, four threads a row of 64 tokens each): scores from tensor memory, scales, mask, weights
//     to shared memory as the pieces above;
//   MMA (warp 8 of the leader): S(t + 1) before O += W(t) C(t), so that S is there a tile ahead;
//   copies (warp 9 of both): TMA boxes of the pages into a ring of slots, in the order of use;
//   scales (warp 10 of both): exponent bytes of a tile to floats;
//   tail (warp 11 of both): zeros over a last tile's rows behind the tokens that are seen, which may hold anything.
// Tensor memory: O at columns 0 to 255 (lanes 64 .. 127 hold the second half of the columns' dims), S(t) at 256 + 128 (t mod 2).
//
// Work is cut evenly: tiles of all units (sequence, 128 rows) in order and kOpen more for each unit, one range for each pair.  A unit that spans ranges
// leaves its parts (m, l, out) in the workspace, and a second kernel joins them.
// Every wait is bounded: one that runs out sets RQ_STATUS_TIMEOUT and an abort flag every role polls.  Warps that meet in a loop
// of such waits leave it together (rows_agree), and what the join reads is there whichever of them ran out.
//
// Device time: 64 x 16,384 x 128 heads bf16 217 us (1,344 TFLOP/s, 70% of the 16-bit rate), fp16 (three pieces) 287; 32 x 1K-32K x
// 16 heads bf16 81 us (3.6 TB/s: MMAs of M = 128 for 16 rows); verify 8 x 16K + 4 x 32 heads fp16 71; 1 x 1,024 x 16 heads fp16
// 14 us, a chain of latencies: lengths, queries, first copies, scores, weights, output, join.  A tile's 68 MMAs (bf16) take
// 4,433 cycles of 6,000 to 7,000: the softmax's tensor memory and shared memory accesses and the copies slow them.  Pages of 16
// tokens (boxes of 2 KB) take 20% more than of 64.
#include <math_constants.h>

#include <cfloat>
#include <cstddef>
#include <type_traits>

#include "../../include/rq.h"
#include "rq_block.cuh"
#include "rq_latent.cuh"
#include "rq_roles.cuh"
#include "rq_rope.cuh"
#include "rq_tma.h"

namespace rq {
namespace {

using namespace latent;
using namespace tc;

constexpr int kSoftWarps = 8, kMmaWarp = 8, kCopyWarp = 9, kScaleWarp = 10, kTailWarp = 11, kThreads = 384;
constexpr int kMmaRows = 128, kTok = 256;  // rows of a pair's MMAs, tokens of a tile
constexpr int kUnitRows = 128;             // the most rows of a unit
constexpr uint32_t kSlotBytes = 16384;
// Slots are filled and given back in units of two: a tile's keys are three units (dims 0 .. 255, 256 .. 511, and one slot of position
// parts), its values two (128 tokens each).  A wait or a commit costs the issuing warp about as much as three MMAs.  A ring of
// four slots (fp16, 64 rows) would hold two of them, too few to hide a load behind: there a unit is one slot (64 x 16K x 128
// heads fp16 309 -> 287 us).
constexpr int kUnits = 8;  // barriers for units: more than there can be in the ring
constexpr uint32_t kColS = 256;
// weights are 2^(score + E - m), m the running maximum of score + E less kLift, moved where a score is past it by more than
// kReach: below 2^12 an e5m2 number's remainder stays within e4m3's 448
constexpr float kLift = 10.f, kReach = 12.f;
constexpr float kNone = -3.402823466e38f;  // m before any visible token
// Opening a unit (its queries as pieces, the first scores) takes the time of some three tiles: in the cut of the work a unit counts
// for its tiles and kOpen more, so that a pair that opens a second one has as many tiles less.  Counted as 0 | 2 | 3 | 4, device us:
// 32 x 1K-32K x 16 heads 105 | 95 | 91 | 92, tree of 5 x 500-9K x 260 rows 40 | 37 | 34 | 34.
constexpr int kOpen = 3;
// floats of a fragment's slot: 128 rows x 512 (as [dim / 4][row][4]), then the rows' m and l
constexpr size_t kSlotFloats = (size_t)kUnitRows * kLatentDim + 2 * kUnitRows;

// A CTA has 64 rows of an MMA.  Where a unit has no more than 64 rows in all (RC = 32 to a CTA) operands are kept for 32: an MMA
// finds whatever follows in the place of the rest, rows whose results nobody reads, and the ring has 10 or 8 slots, more than
// a tile or nearly, instead of 7 or 4.
//
// Where it has no more than 32 (RV = 16 rows to a CTA, of RC = 32 kept), the queries' first two pieces are different rows of one
// operand, row r and r + 16, whose scores the softmax adds: half the MMAs for scores.  (Weights are pieces of two types, and
// one MMA's operand is of one.)  The lanes of the two rows then take 16 columns of 32 each, which halves the softmax, and the
// weights go to the first row's place.  32 x 1K-32K x 16 heads bf16 89 -> 81 us, fp16 113 -> 98,
// 1 x 1,024 15.9 -> 14.3.
template <typename T, int RC, int RV>
struct Shape {
  static constexpr int kPieces = std::is_same<T, __half>::value ? 3 : 2, kQueryPieces = RV < RC ? kPieces - 1 : kPieces;
  static constexpr uint32_t kRowsBytes = RC * 128;  // a chunk of 128 dims, or of 128 tokens' weights
  static constexpr uint32_t kPieceQ = 4 * kRowsBytes, kQBytes = kQueryPieces * kPieceQ + kRowsBytes;  // [piece][4 chunks][RC rows], position parts
  static constexpr uint32_t kPieceP = 2 * kRowsBytes, kTileP = kPieces * kPieceP;                // [piece][2 halves of 128 tokens][RC rows]
  static constexpr int kTilesP = RC < 64 ? 2 : 1;  // weights of two tiles, where there is room: one's are written while the other's are read
  static constexpr uint32_t kPBytes = kTilesP * kTileP;
  static constexpr uint32_t kOffMisc = 221184, kOffP = kQBytes, kOffRing = kOffP + kPBytes;
  static constexpr int kSlots = (kOffMisc - kOffRing) / kSlotBytes;
  static constexpr int kPer = kSlots < 5 ? 1 : 2, kKeys = 4 / kPer + 1, kValues = 4 / kPer;  // slots of a unit, units of a tile
};

struct Frag {           // tiles r0 .. r0 + n - 1 of one unit
  int b, rt, r0, n, len, end;  // end: tokens that the unit's rows see lie before it
  int whole;            // the unit is all here
  int range, range_last;  // its first range, and whether the fragment there is that range's last
  int done;             // no more fragments
};
struct Misc {
  // the leader's: a unit is full; the queries; W(t); a tail's zeros are written
  uint64_t full[kUnits], q_full, p_full[2], tail_done[kUnits];
  // both CTAs': a unit is read; S(t); O(t); drained; a unit of the tail is here; scales of a tile
  uint64_t empty[kUnits], s_full[2], o_done[2], drain, here[kUnits], sc_full[2], sc_empty[2];
  Frag f;
  uint32_t tmem;
  int abort;
  alignas(16) float ks[2][kTok], ev[2][kTok], dn[2][kTok];  // 2^E (or NaN), E, 2^-E of a tile's tokens
  float top[2][4][64];
  float q_scale[64];
};
constexpr int kSmem = (int)(Shape<__half, 64, 64>::kOffMisc + sizeof(Misc)) + 1024;
static_assert(kSmem + 128 <= 232448, "one CTA's shared memory");

struct Unit {
  int len, end, tiles;
};
__device__ __forceinline__ Unit unit_of(const LatentAttnArgs& a, int unit_rows, int cap, int b, int rt, bool report) {
  Unit u;
  u.len = __ldg(a.seq_lens + b);
  if (u.len < 0 || u.len > cap || (u.len > 0 && u.len < a.T)) {
    if (report && a.status) atomicOr(a.status, RQ_STATUS_BAD_LEN);
    u.len = u.len < 0 ? 0 : min(u.len, cap);
  }
  const long long rows = (long long)a.T * a.heads;
  const int last = (int)((uint32_t)(min(rows, (rt + 1ll) * unit_rows) - 1) / (uint32_t)a.heads);  // the last row's token (rows: below 2^30)
  u.end = a.tree_mask ? u.len : max(0, min(u.len, u.len - a.T + last + 1));
  u.tiles = max(1, (u.end + kTok - 1) / kTok);  // rows that see nothing are written too
  return u;
}

// Instruction descriptors: kind::f8f6f4 with A of e4m3 (0) or e5m2 (1), B of e4m3; bit 16: B with N along its rows.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, uint32_t a_type, uint32_t b_rows) {
  return idesc_f16(M, N) | a_type << 7 | b_rows << 16;
}
// An operand by the low word of its descriptor (address >> 4; the high word is the same for all: 1024 bytes from eight rows to the
// next, the 128-byte swizzle).  Few instructions an MMA: the issuing warp shares its scheduler with the softmax.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return saddr >> 4 | 1u << 16; }
__device__ __forceinline__ void pair_mma_f8(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 a, b;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n mov.b64 a, {%1, %5};\n"
      " mov.b64 b, {%2, %5};\n @e tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "r"(accumulate), "n"(0x40004040));
}
__device__ __forceinline__ void pair_mma_16(uint32_t d, uint32_t a, uint32_t b, uint32_t id) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 a, b;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, 1, 0;\n mov.b64 a, {%1, %4};\n"
      " mov.b64 b, {%2, %4};\n @e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(id), "n"(0x40004040));
}
// A box of the pool's planes ([page][plane][row][128 bytes]) for each lane whose turn it is; the bytes count at `bar`, a barrier of
// the leader (pair), or of this CTA.
__device__ __forceinline__ void load_pair(uint32_t dst, const CUtensorMap& map, int row, int plane, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(&map), "r"(0), "r"(row), "r"(plane), "r"(page), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void load_here(uint32_t dst, const CUtensorMap& map, int row, int plane, int page, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(&map), "r"(0), "r"(row), "r"(plane), "r"(page), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// The four warps that share 32 rows meet: whether all of them are ok.  One whose wait ran out comes here too, once, before it leaves,
// and the others leave behind it: this barrier has no limit of its own.
__device__ __forceinline__ bool rows_agree(int half, bool ok) {
  uint32_t all;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 q, %2, 0;\n bar.red.and.pred p, %1, 128, q;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(all)
               : "r"(2 + half), "r"((uint32_t)ok)
               : "memory");
  return all;
}

// Pieces of two weights (fp16, 0 to 2^12) in few operations of the integer and fp16 pipes (a conversion to 8 bits takes 14
// cycles of a scheduler, these two).  e5m2 is an fp16 number's upper byte: the first piece is the number rounded to that, its
// code the upper bytes.  What is left is within 2^8; times 2^-8 its fp16 pattern, moved up by a bit, is e4m3's in the upper
// byte (both have their smallest normal and their steps below it in the same place): rounded by half a step, the sign put back.
__device__ __forceinline__ uint32_t first_piece(uint32_t& h) {  // (ties go up: the next piece takes what is left either way)
  const uint32_t c = h + 0x00800080u & 0xFF00FF00u;
  asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h) : "r"(c));
  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h) : "r"(0x1C001C00u));  // 2^-8
  return c;
}
__device__ __forceinline__ uint32_t next_piece(uint32_t h) {  // h times 2^-8
  return (2u * h + 0x00800080u) & 0x7FFF7FFFu | h & 0x80008000u;
}
// What is left of h behind the piece of next_piece.
__device__ __forceinline__ uint32_t behind(uint32_t h, uint32_t code) {
  const uint32_t c = (code & 0x7F007F00u) >> 1 | h & 0x80008000u;
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h), "r"(c));
  return d;
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
__device__ __forceinline__ uint64_t plus2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// The smallest E of -126 and more with top_c <= 448 * 2^E and top_p <= 2^(15 + E), from their bits.  The largest bf16 number's is
// 120, and from -126 on even the smallest one, 2^-133, is a multiple of e4m3's smallest step: a row of any finite magnitude fits
// its pieces.
__device__ __forceinline__ int query_exp(uint32_t top_c, uint32_t top_p) {
  const int c = (int)(top_c >> 23) - 127 - 8 + ((top_c & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  const int p = (int)(top_p >> 23) - 127 - 15 + ((top_p & 0x7FFFFFu) != 0u ? 1 : 0);
  return max(max(c, p), -126);
}

template <typename T, int RC, int RV>
__global__ void __launch_bounds__(kThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap map, const LatentPool pool, const LatentAttnArgs a, int box, int4* info) {
  using S = Shape<T, RC, RV>;
  constexpr bool kTwice = RV < RC;  // a row stands in two places
  constexpr int kUR = 2 * RV;       // rows of a unit
  constexpr int NP = S::kPieces, NQ = S::kQueryPieces, kSlots = S::kSlots, kPer = S::kPer;
  constexpr bool kF16 = std::is_same<T, __half>::value;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = smem_addr(smem_raw) + (1024 - (smem_addr(smem_raw) & 1023) & 1023);
  Misc& ms = *reinterpret_cast<Misc*>(smem_raw + (base - smem_addr(smem_raw)) + S::kOffMisc);
  const uint32_t q_ops = base, p_ops = base + S::kOffP, ring = base + S::kOffRing;
  volatile int* const abort_flag = &ms.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int P = pool.page_size, cap = a.max_pages * P;
  const long long n_rows = (long long)a.T * a.heads;
  const int n_rt = (int)((n_rows + kUR - 1) / kUR);

  if (tid == 32 * kMmaWarp) {
    for (int i = 0; i < kUnits; ++i) {
      mbar_init(smem_addr(&ms.full[i]), 1);
      mbar_init(smem_addr(&ms.empty[i]), 1);
      mbar_init(smem_addr(&ms.here[i]), 1);
      mbar_init(smem_addr(&ms.tail_done[i]), 2);
    }
    mbar_init(smem_addr(&ms.q_full), 2 * kSoftWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&ms.p_full[i]), 2 * kSoftWarps);
      mbar_init(smem_addr(&ms.o_done[i]), 1);
      mbar_init(smem_addr(&ms.s_full[i]), 1);
      mbar_init(smem_addr(&ms.sc_full[i]), 1);
      mbar_init(smem_addr(&ms.sc_empty[i]), kSoftWarps);
    }
    mbar_init(smem_addr(&ms.drain), 1);
    ms.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncwarp();
  if (warp == kMmaWarp) pair_tmem_alloc(smem_addr(&ms.tmem), 512);  // (while the lengths come)
  fence_before_sync();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  // ---- the pair's range: x .. x_end - 1 of `total` (kOpen and the tiles of each unit), kept by thread 0 ----
  // range c starts at c * each + min(c, more)
  const uint32_t pairs = gridDim.x >> 1, me = blockIdx.x >> 1;
  uint32_t total, parts, each, more, x, x_end, at, item;  // at: where unit `item` begins
  Unit un;
  auto range_of = [&](uint32_t tile) {  // the range that holds a tile
    const uint32_t longer = more * (each + 1u);
    return tile < longer ? tile / (each + 1u) : more + (tile - longer) / each;
  };
  {
    __shared__ uint32_t s_sums[kThreads / 32], s_found[2];
    __shared__ Unit s_unit;
    // a thread's units; the first ones are the last warps', which have the least to do while a unit opens
    const uint32_t n_items = (uint32_t)a.B * n_rt, chunk = (n_items + kThreads - 1) / kThreads;
    const int order = kThreads / 32 - 1 - warp;
    const uint32_t owner = 32 * order + lane;
    uint32_t mine = 0;
    for (uint32_t i = owner * chunk; i < min(n_items, (owner + 1) * chunk); ++i)
      mine += kOpen + unit_of(a, kUR, cap, (int)(i / (uint32_t)n_rt), (int)(i % (uint32_t)n_rt), blockIdx.x == 0).tiles;
    uint32_t sum = mine;  // inclusive, over the warp, then over the warps before
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) s_sums[order] = sum;
    __syncthreads();
    uint32_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w == order) before = total;
      total += s_sums[w];
    }
    parts = min(pairs, total);
    each = total / parts, more = total - each * parts;
    x = me * each + min(me, more);
    x_end = me < parts ? x + each + (me < more ? 1u : 0u) : x;  // (a pair without a range: done at once)
    before += sum - mine;
    if (x < x_end && x >= before && x < before + mine) {
      uint32_t p = before, i = owner * chunk;
      for (;; ++i) {
        un = unit_of(a, kUR, cap, (int)(i / (uint32_t)n_rt), (int)(i % (uint32_t)n_rt), false);
        if (x < p + kOpen + un.tiles) break;
        p += kOpen + un.tiles;
      }
      s_found[0] = p;
      s_found[1] = i;
      s_unit = un;
    }
    __syncthreads();
    at = s_found[0];
    item = s_found[1];
    un = s_unit;
    // A note for each unit, for the join: its first range, its parts (0: it is whole), whether it is the last of its first range.  The
    // CTAs take the threads' units in turn and write their notes here, before any wait that can run out: the join finds every one.
    if (owner % gridDim.x == blockIdx.x)
      for (uint32_t i = owner * chunk, p = before; i < min(n_items, (owner + 1) * chunk); ++i) {
        const uint32_t end = p + (chunk == 1 ? mine : kOpen + unit_of(a, kUR, cap, (int)(i / (uint32_t)n_rt), (int)(i % (uint32_t)n_rt), false).tiles);
        const uint32_t first = range_of(p + kOpen), begins = first * each + min(first, more);
        const bool whole = end <= begins + each + (first < more ? 1u : 0u);
        info[i] = make_int4((int)first, whole ? 0 : (int)(range_of(end - 1) - first) + 1, begins < p, 0);
        p = end;
      }
  }
  bool first_frag = true;

  // softmax: row of the CTA (= lane of tensor memory, twice), the quarter of a tile's tokens and of the dims
  const int quad = warp & 3, col_half = warp >> 2 & 1, row = 32 * (quad & 1) + lane, tok_half = quad >> 1;
  const int quarter = 2 * tok_half + col_half;
  const uint32_t lane_off = (uint32_t)(32 * quad) << 16;
  uint32_t done_tiles = 0, done_frags = 0;  // with tokens: tiles and fragments before
  uint32_t tails = 0;                       // parity of the tail's use of each unit's barriers
  // copies: slots and units asked for, slots and units given back, which of the last 32 units are of two slots
  uint32_t asked = 0, asked_units = 0, freed = 0, freed_units = 0, twos = 0;
  for (;;) {
    if (tid == 0) {  // the next fragment
      Frag& f = ms.f;
      f.done = x >= x_end;
      if (!f.done) {
        f.b = (int)(item / (uint32_t)n_rt);
        f.rt = (int)(item % (uint32_t)n_rt);
        if (!first_frag) un = unit_of(a, kUR, cap, f.b, f.rt, false);
        f.len = un.len;
        f.end = un.end;
        f.r0 = max(0, (int)(x - at) - kOpen);
        f.n = min(un.tiles, (int)(x_end - at) - kOpen) - f.r0;
        f.done = f.n <= 0;  // the range ends before the unit's first tile
      }
      if (!f.done) {
        f.whole = f.n == un.tiles;
        const uint32_t first = range_of(at + kOpen);  // (this one, where r0 is 0)
        f.range = (int)first;
        f.range_last = first * each + min(first, more) < at;
        x = at + kOpen + f.r0 + f.n;
        if (f.r0 + f.n == un.tiles) {
          at = x;
          ++item;
        }
      }
    }
    fence_before_sync();
    __syncthreads();
    if (first_frag) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the peer's barriers are there
    first_frag = false;
    fence_after_sync();
    if (ms.f.done) break;
    const uint32_t tmem = *(volatile uint32_t*)&ms.tmem;
    const int b = ms.f.b, r0 = ms.f.r0, len = ms.f.len, end = ms.f.end;
    const int n = end > 0 ? ms.f.n : 0;  // tiles with tokens
    const long long urow = (long long)ms.f.rt * kUR + RV * (int)rank + (kTwice ? row % RV : row);  // the thread's query row
    const bool valid = row < RC && urow < n_rows;
    const int j = valid ? (int)((uint32_t)urow / (uint32_t)a.heads) : 0, head = valid ? (int)((uint32_t)urow % (uint32_t)a.heads) : 0;
    const uint32_t t_base = done_tiles;
    float m_run = kNone, l_run = 0.f;
    bool ok = true;

    if (warp < kSoftWarps) {
      float q_scale = 0.f;
      if (n > 0 && (!kTwice || 4 * warp < RV)) {
        // ---- queries as pieces: kRW rows to a warp, a lane 16 dims and an eighth of a position part of every fourth row ----
        constexpr int kRW = kTwice ? 4 : RC / kSoftWarps;
        // lane l: where row l % kRW of the warp's stands, -1 past the last row
        long long c_at = -1, pe_at = -1;
        {
          const long long u = (long long)ms.f.rt * kUR + RV * (int)rank + kRW * warp + lane % kRW;
          if (u < n_rows) {
            const uint32_t jj = (uint32_t)u / (uint32_t)a.heads, hh = (uint32_t)u - jj * (uint32_t)a.heads;
            const long long token = (long long)b * a.T + jj;
            c_at = token * a.q_c.stride + hh * a.q_c.head_stride;
            pe_at = token * a.q_pe.stride + hh * a.q_pe.head_stride;
          }
        }
        uint4 raw[kRW][2], pe2[kRW / 4];  // all loads in flight together
#pragma unroll
        for (int r = 0; r < kRW; ++r) {
          const long long from = __shfl_sync(0xffffffffu, c_at, r);
          const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q_c.x) + from) + 2 * lane;
#pragma unroll
          for (int i = 0; i < 2; ++i) raw[r][i] = from >= 0 ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int r = 0; r < kRW / 4; ++r) {
          const long long from = __shfl_sync(0xffffffffu, pe_at, 4 * r + (lane >> 3));
          pe2[r] = from >= 0 ? __ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(a.q_pe.x) + from) + (lane & 7)) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll 1
        for (int r4 = 0; r4 < kRW; r4 += 4) {
          const int row0 = kRW * warp + r4;
          const uint4 pe = pe2[0];
          // magnitudes order as their 16 bits do, NaN above infinity above the rest
          auto largest = [&](const uint4& v) {
            uint32_t m = v.x & 0x7FFF7FFFu;
            asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(v.y & 0x7FFF7FFFu));
            asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(v.z & 0x7FFF7FFFu));
            asm("max.u16x2 %0, %0, %1;" : "+r"(m) : "r"(v.w & 0x7FFF7FFFu));
            return max(m >> 16, m & 0xFFFFu);
          };
          uint32_t top_p = largest(pe);  // of row lane / 8
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) top_p = max(top_p, __shfl_xor_sync(0xffffffffu, top_p, o));
          float pe_down = 0.f;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t top_c = __reduce_max_sync(0xffffffffu, max(largest(raw[0][0]), largest(raw[0][1])));
            const uint32_t top_r = __shfl_sync(0xffffffffu, top_p, 8 * r);
            const bool odd = max(top_c, top_r) >= (kF16 ? 0x7C00u : 0x7F80u);  // a row that is not finite: all its scores are NaN
            const float2 tops = rope::unpack2<T>(top_c | top_r << 16);
            // (fp16: 2^(-e - 8) is a factor in fp16; what is below 2^-20 of 448 has few bits)
            const int e = odd ? 0 : max(query_exp(__float_as_uint(tops.x), __float_as_uint(tops.y)), kF16 ? -20 : -126);
            const float down = block::pow2(-e);
            if ((lane >> 3) == r) pe_down = odd ? 0.f : down;
            // (a factor past float32: the row's largest value times sm_scale is too)
            const float factor = a.sm_scale * (1.44269504088896340736f * block::pow2(e));
            if (lane == 0) ms.q_scale[row0 + r] = odd || factor > FLT_MAX ? CUDART_NAN_F : factor;
            uint32_t piece[NP][4];
            const float down8 = down * 0.00390625f;  // 2^-8: as next_piece wants it
            const uint32_t down8_2 = rope::pack2<__half>(down8, down8);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t code[2][NP];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                uint32_t h = word(raw[0][k >> 1], 2 * (k & 1) + i);  // times 2^(-e - 8): exact, but for what is below 2^-24
                if constexpr (kF16) {
                  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h) : "r"(down8_2));
                } else {
                  const float2 f = rope::unpack2<T>(h);
                  h = rope::pack2<__half>(f.x * down8, f.y * down8);
                }
                if (odd) h = 0u;
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                  code[i][p] = next_piece(h);
                  if (p + 1 < NP) h = behind(h, code[i][p]);
                }
              }
#pragma unroll
              for (int p = 0; p < NP; ++p) piece[p][k] = __byte_perm(code[0][p], code[1][p], 0x7531);
            }
#pragma unroll
            for (int p = 0; p < NP; ++p)
              sts128(q_ops + (kTwice ? p >> 1 : p) * S::kPieceQ + S::kRowsBytes * (lane >> 3) + sw128(row0 + r + (kTwice ? RV * (p & 1) : 0), lane & 7),
                     piece[p][0], piece[p][1], piece[p][2], piece[p][3]);
            if constexpr (kTwice && NP > 2)  // a third piece has no other beside it
              sts128(q_ops + S::kPieceQ + S::kRowsBytes * (lane >> 3) + sw128(row0 + r + RV, lane & 7), 0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i + 1 < kRW; ++i) raw[i][0] = raw[i + 1][0], raw[i][1] = raw[i + 1][1];  // (four rows' code, not eight)
          }
          if constexpr (kRW > 4) pe2[0] = pe2[1];
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = rope::unpack2<T>(word(pe, k));
            w[k] = pe_down == 0.f ? 0u : rope::pack2<T>(f.x * pe_down, f.y * pe_down);
          }
          sts128(q_ops + NQ * S::kPieceQ + sw128(row0 + (lane >> 3), lane & 7), w[0], w[1], w[2], w[3]);
          if constexpr (kTwice) sts128(q_ops + NQ * S::kPieceQ + sw128(row0 + (lane >> 3) + RV, lane & 7), 0u, 0u, 0u, 0u);
        }
        fence_async_smem();
      }
      if (n > 0) {
        warp_arrive_pair(peer_addr(smem_addr(&ms.q_full), 0));
        soft_sync();  // the rows' scales are there
        if (row < RC) q_scale = ms.q_scale[kTwice ? row % RV : row];
      }
      // ================= softmax =================
      // Scores 16 columns at a time, twice: loops over them and not 64 columns in a row, so that the roles' code fits the
      // instruction cache (unrolled, the warps spent more cycles without instructions than with them).
      // The row sees tokens before `all`, of the drafts behind them the ones up to its own or those of its mask.  A row past the
      // last one sees all: what becomes of it is not written.
      const int all = valid ? (a.tree_mask ? len - a.T : len - a.T + j + 1) : INT32_MAX - 1024;
      uint64_t mask = valid && a.tree_mask ? __ldg(a.tree_mask + (long long)b * a.T + j) : 0ull;
      if (a.T < 64) mask &= (1ull << a.T) - 1ull;
      const bool idle = !__any_sync(0xffffffffu, valid);  // (all four warps of the rows alike)
      const uint32_t s_cols = tmem + lane_off + kColS + 64 * col_half;
      constexpr int kStep = kTwice ? 32 : 16;
      const int own = kTwice ? lane & 16 : 0;  // the lane's 16 columns of a step
      constexpr int kBack = S::kTilesP;
      auto o_is_done = [&](uint32_t k) { return warp_wait(ms.o_done[k & 1], k >> 1, abort_flag); };  // O(k), counted over fragments
      for (int t = 0; t < n; ++t) {
        const uint32_t k = t_base + t, buf = k & 1;
        const uint32_t p_tile = p_ops + (kBack > 1 ? buf * S::kTileP : 0u);
        if (idle) {  // takes part in the counts; O(t - kTilesP) says that the last count is over, the scales that theirs is
          if (t >= kBack && !(ok = o_is_done(k - kBack))) break;
          if (!(ok = warp_wait(ms.sc_full[buf], k >> 1, abort_flag))) break;
          warp_arrive(ms.sc_empty[buf]);
          warp_arrive_pair(peer_addr(smem_addr(&ms.p_full[buf]), 0));
          continue;
        }
        const int t0 = (r0 + t) * kTok + 64 * quarter;
        ok = ok && warp_wait(ms.s_full[buf], k >> 1, abort_flag) && warp_wait(ms.sc_full[buf], k >> 1, abort_flag);
        if (!ok) {
          rows_agree(quad & 1, false);
          break;
        }
        fence_after_sync();
        float top = -CUDART_INF_F;
        {
          const uint64_t q2 = pair(q_scale, q_scale);
#pragma unroll 1
          for (int c = 0; c < 64; c += kStep) {  // score + E
            float v[16], other[16];
            tmem_ld16(s_cols + 128 * buf + c, v);
            if constexpr (kTwice) tmem_ld16(s_cols + 128 * buf + c + 16, other);
            const ulonglong2* const ks = reinterpret_cast<const ulonglong2*>(&ms.ks[buf][64 * quarter + c + own]);
            const ulonglong2* const ev = reinterpret_cast<const ulonglong2*>(&ms.ev[buf][64 * quarter + c + own]);
            ulonglong2 f[4], e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = ks[i], e[i] = ev[i];
            tmem_wait_ld();
            settle<16>(v);
            if constexpr (kTwice) {
              settle<16>(other);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float sent = __shfl_xor_sync(0xffffffffu, own ? v[i] : other[i], RV);
                v[i] = (own ? other[i] : v[i]) + sent;
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // the token's scale first: it takes no sum out of range, where the two factors' product may be
              unpair(fma2(mul2(pair(v[4 * i], v[4 * i + 1]), f[i].x), q2, e[i].x), v[4 * i], v[4 * i + 1]);
              unpair(fma2(mul2(pair(v[4 * i + 2], v[4 * i + 3]), f[i].y), q2, e[i].y), v[4 * i + 2], v[4 * i + 3]);
            }
            const int first = t0 + c + own - all;  // of the columns' tokens, counted from the first that the mask is for
            if (first > -16) {
              const uint32_t seen = first >= 64 ? 0u : first >= 0 ? (uint32_t)(mask >> first) : (1u << -first) - 1u | (uint32_t)mask << -first;
#pragma unroll
              for (int i = 0; i < 16; ++i)
                if (!(seen >> i & 1)) v[i] = -CUDART_INF_F;
            }
            float top1 = max3(v[0], v[1], v[2]);
#pragma unroll
            for (int i = 3; i < 15; i += 4) top = max3(top, v[i], v[i + 1]), top1 = max3(top1, v[i + 2], v[i + 3]);
            top = max3(top, top1, v[15]);
            tmem_st16(s_cols + 128 * buf + c, v);
          }
        }
        if constexpr (kTwice) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, RV));
        ms.top[buf][quarter][row] = top;
        tmem_wait_st();
        if (!(ok = rows_agree(quad & 1, true))) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, ms.top[buf][i][row]);
        const float above = top - (m_run == kNone ? -CUDART_INF_F : m_run);  // (NaN where nothing is seen: no move)
        float alpha = 1.f;
        const bool move = __any_sync(0xffffffffu, above > kReach);
        if (above > kReach) {
          float to = top - kLift;
          if (top - to > kReach) to = top;  // (float32's steps are 16 apart from 2^27 on: a lift of 16 would take the weight past fp16)
          alpha = ex2(m_run - to);
          m_run = to;
          l_run *= alpha;
        }
        const float from = m_run == kNone ? 0.f : m_run;
        // the weights' place is free behind O(t - kTilesP), and O may be scaled behind O(t - 1) (a wait that runs out: to the next meeting)
        if (kBack > 1 && t >= kBack && !(ok = o_is_done(k - kBack))) continue;
        if (t > 0 && (kBack == 1 || move)) {
          if (!(ok = o_is_done(k - 1))) continue;
          if (move) {
            fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              float v[16];
              const uint32_t cols = tmem + lane_off + 128 * col_half + 16 * c;
              tmem_ld16(cols, v);
              tmem_wait_ld();
              settle<16>(v);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] *= alpha;
              tmem_st16(cols, v);
            }
            tmem_wait_st();
          }
        }
        {
          uint64_t sum[2] = {0ull, 0ull};
          const uint64_t back = pair(-from, -from);
#pragma unroll 1
          for (int c = 0; c < 64; c += kStep) {
            float v[16];
            tmem_ld16(s_cols + 128 * buf + c, v);
            const ulonglong2* const dn = reinterpret_cast<const ulonglong2*>(&ms.dn[buf][64 * quarter + c + own]);
            ulonglong2 d[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = dn[i];
            tmem_wait_ld();
            settle<16>(v);
            uint32_t piece[NP][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float w[4];
              unpair(plus2(pair(v[4 * i], v[4 * i + 1]), back), w[0], w[1]);
              unpair(plus2(pair(v[4 * i + 2], v[4 * i + 3]), back), w[2], w[3]);
#pragma unroll
              for (int x = 0; x < 4; ++x) w[x] = ex2(w[x]);
              sum[0] = fma2(pair(w[0], w[1]), d[i].x, sum[0]);
              sum[1] = fma2(pair(w[2], w[3]), d[i].y, sum[1]);
              uint32_t h[2] = {rope::pack2<__half>(w[0], w[1]), rope::pack2<__half>(w[2], w[3])}, code[2];
#pragma unroll
              for (int x = 0; x < 2; ++x) code[x] = first_piece(h[x]);
              piece[0][i] = __byte_perm(code[0], code[1], 0x7531);
#pragma unroll
              for (int p = 1; p < NP; ++p) {
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  code[x] = next_piece(h[x]);
                  if (p + 1 < NP) h[x] = behind(h[x], code[x]);
                }
                piece[p][i] = __byte_perm(code[0], code[1], 0x7531);
              }
            }
#pragma unroll
            for (int p = 0; p < NP; ++p)
              sts128(p_tile + p * S::kPieceP + S::kRowsBytes * tok_half + sw128(kTwice ? row % RV : row, 4 * col_half + ((c + own) >> 4)), piece[p][0], piece[p][1], piece[p][2],
                     piece[p][3]);
          }
          float y[4];
          unpair(sum[0], y[0], y[1]);
          unpair(sum[1], y[2], y[3]);
          l_run += (y[0] + y[1]) + (y[2] + y[3]);
        }
        warp_arrive(ms.sc_empty[buf]);
        fence_async_smem();
        fence_before_sync();
        warp_arrive_pair(peer_addr(smem_addr(&ms.p_full[buf]), 0));
      }
      if (ok && n > 0) ok = o_is_done(t_base + n - 1);
      fence_after_sync();
    } else if (warp == kMmaWarp) {
      // ================= MMA issue: the leader's =================
      if (rank == 0 && n > 0) {
        constexpr uint32_t id_s = idesc_f8(kMmaRows, kTok, 0, 0), id_o5 = idesc_f8(kMmaRows, 256, 1, 1), id_o4 = idesc_f8(kMmaRows, 256, 0, 1);
        constexpr uint32_t type = std::is_same<T, __half>::value ? 0u : 1u;
        constexpr uint32_t id_p = idesc_f16(kMmaRows, kTok) | type << 7 | type << 10;
        bool issued = false;
        // units and slots in the order of use: K(0) | K(1) V(0) | K(2) V(1) | ...
        uint32_t u = (uint32_t)(S::kKeys + S::kValues) * t_base, sl = 9u * t_base;
        auto unit_full = [&](uint32_t v) -> uint64_t& { return ms.full[v % kUnits]; };
        uint32_t look = warp_look(unit_full(u), u / kUnits);
        auto take = [&]() { return ok = warp_wait_after(look, unit_full(u), u / kUnits, abort_flag); };  // unit u is full
        auto peek = [&]() { look = warp_look(unit_full(u + 1), (u + 1) / kUnits); };  // late in unit u, so that the look finds what there is
        uint32_t p_look = 0;
        auto give = [&]() {
          pair_commit(smem_addr(&ms.empty[u % kUnits]), 3);
          ++u;
          issued = true;
        };
        const uint32_t q_lo = desc_lo(q_ops), w_lo = desc_lo(p_ops), ring_lo = desc_lo(ring);
        auto slot = [&]() { return ring_lo + sl++ % kSlots * (kSlotBytes / 16); };
        auto s_mmas = [&](int t) {  // S(t)
          const uint32_t d = tmem + kColS + 128 * ((t_base + t) & 1);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            if (c % kPer == 0 && !take()) return;
            const uint32_t b_at = slot(), a_at = q_lo + S::kRowsBytes / 16 * c;
#pragma unroll
            for (int p = 0; p < NQ; ++p) {
              if (p + 1 == NQ && c % kPer == kPer - 1) peek();
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                pair_mma_f8(d, a_at + (p * S::kPieceQ + 32 * ks) / 16, b_at + 2 * ks, id_s, p > 0 || ks > 0 ? 1u : (uint32_t)c);
            }
            if (c % kPer == kPer - 1) give();
          }
          if (!take()) return;
          peek();
          if (t > 0) p_look = warp_look(ms.p_full[(t_base + t - 1) & 1], (t_base + t - 1) >> 1);
          const uint32_t b_at = slot();
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            pair_mma_16(d, q_lo + (NQ * S::kPieceQ + 32 * ks) / 16, b_at + 2 * ks, id_p);
          give();
          pair_commit(smem_addr(&ms.s_full[(t_base + t) & 1]), 3);
        };
        if (ok = warp_wait(ms.q_full, done_frags, abort_flag); ok) {
          fence_after_sync();
          s_mmas(0);
        }
        for (int t = 0; t < n && ok; ++t) {
          p_look = 0;
          if (t + 1 < n) s_mmas(t + 1);
          if (!ok || !(ok = warp_wait_after(p_look, ms.p_full[(t_base + t) & 1], (t_base + t) >> 1, abort_flag))) break;
          fence_after_sync();
          const uint32_t w_tile = S::kTilesP > 1 ? ((t_base + t) & 1) * (S::kTileP / 16) : 0u;
#pragma unroll 1
          for (int g = 0; g < 4; ++g) {  // 64 tokens
            if (g % kPer == 0) {
              if (!take()) break;
              if ((r0 + t) * kTok + 64 * (g + kPer) > end) {
                if (!(ok = warp_wait(ms.tail_done[u % kUnits], tails >> (u % kUnits) & 1, abort_flag))) break;
                tails ^= 1u << (u % kUnits);
              }
            }
            const uint32_t b_at = slot(), w_at = w_lo + w_tile + (g >> 1) * (S::kRowsBytes / 16) + (g & 1) * 4;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              if (ks == 1 && g % kPer == kPer - 1) peek();
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int p = 0; p < NP; ++p)
                  pair_mma_f8(tmem + 128 * h, w_at + (p * S::kPieceP + 32 * ks) / 16, b_at + (8192 * h + 4096 * ks) / 16,
                              p == 0 ? id_o5 : id_o4, ks > 0 || p > 0 ? 1u : (uint32_t)(t + g));
            }
            if (g % kPer == kPer - 1) give();
          }
          if (!ok) break;
          pair_commit(smem_addr(&ms.o_done[(t_base + t) & 1]), 3);
        }
        if (!ok && issued) {  // nothing may be running when the tensor memory is freed
          pair_commit(smem_addr(&ms.drain), 3);
          for (int i = 0; i < kWaitLimit; ++i)
            if (mbar_test(smem_addr(&ms.drain), 0u)) break;
        }
      }
    } else if (warp == kCopyWarp) {
      // ================= copies: this CTA's share =================
      const int32_t* table = a.block_table + (size_t)b * a.max_pages;
      const int per_half = 128 / box, per_slot = 64 / box;  // boxes
      // boxes 0 .. 256 / box - 1 of a tile, a lane each: page (or -1) and row in it
      auto place = [&](int t, int& page, int& in_page) {
        const int p = (r0 + t) * kTok + box * lane;
        page = -1, in_page = 0;
        if (t >= n || box * lane >= kTok || p >= end) return;
        page = __ldg(table + p / P);
        in_page = p % P;
        if (page < 0 || page >= pool.num_pages) {
          if (a.status) atomicOr(a.status, RQ_STATUS_BAD_PAGE);
          page = 0;
        }
      };
      // room for a unit of `count` slots: units are given back in order
      auto room = [&](uint32_t count) {
        while (asked + count - freed > (uint32_t)kSlots) {
          if (!(ok = warp_wait(ms.empty[freed_units % kUnits], freed_units / kUnits, abort_flag))) return false;
          freed += 1u + (twos >> (freed_units % 32) & 1u);
          ++freed_units;
        }
        twos = (twos & ~(1u << (asked_units % 32))) | (count - 1u) << (asked_units % 32);
        return true;
      };
      auto boxes = [&](int p, int count) { return min(max(0, (end - p + box - 1) / box), count); };  // from token p on
      auto keys = [&](int t, int page, int in_page) {
        const int p = (r0 + t) * kTok;
        const int both = boxes(p, per_half) + boxes(p + 128, per_half), mine = boxes(p + 128 * (int)rank, per_half);
        // lane: box lane % per_half of the unit's slot lane / per_half
        const int i = lane % per_half, c = lane / per_half;
        const int pg = __shfl_sync(0xffffffffu, page, per_half * (int)rank + i), ip = __shfl_sync(0xffffffffu, in_page, per_half * (int)rank + i);
        for (int k = 0; k < S::kKeys; ++k) {
          const int slots = k + 1 < S::kKeys ? kPer : 1;
          if (!room(slots)) return;
          const uint32_t u = asked_units % kUnits;
          if (rank == 0) elect_expect(smem_addr(&ms.full[u]), (uint32_t)(slots * both * box * 128));
          __syncwarp();
          if (c < slots && i < mine)
            load_pair(ring + (asked + c) % kSlots * kSlotBytes + i * box * 128, map, ip, kPer * k + c, pg, peer_addr(smem_addr(&ms.full[u]), 0));
          asked += slots;
          ++asked_units;
        }
      };
      auto values = [&](int t, int page, int in_page) {
        for (int g = 0; g < S::kValues; ++g) {  // slots of 64 tokens
          if (!room(kPer)) return;
          const uint32_t u = asked_units % kUnits;
          const int p = (r0 + t) * kTok + 64 * kPer * g, count = boxes(p, kPer * per_slot);
          const bool tail = p + 64 * kPer > end;
          // lane: box lane % (kPer per_slot) of dims 128 (2 rank + lane / (kPer per_slot)) ..
          const int i = lane % (kPer * per_slot), c = lane / (kPer * per_slot);
          const int pg = __shfl_sync(0xffffffffu, page, kPer * per_slot * g + i), ip = __shfl_sync(0xffffffffu, in_page, kPer * per_slot * g + i);
          const uint32_t dst = ring + (asked + i / per_slot) % kSlots * kSlotBytes + 8192 * c + i % per_slot * box * 128;
          const bool mine = c < 2 && i < count;
          if (!tail) {
            if (rank == 0) elect_expect(smem_addr(&ms.full[u]), 2 * kPer * kSlotBytes);
            __syncwarp();
            if (mine) load_pair(dst, map, ip, 2 * (int)rank + c, pg, peer_addr(smem_addr(&ms.full[u]), 0));
          } else {  // the tail's warp of this CTA first
            elect_expect(smem_addr(&ms.here[u]), (uint32_t)(2 * count * box * 128));
            __syncwarp();
            if (mine) load_here(dst, map, ip, 2 * (int)rank + c, pg, smem_addr(&ms.here[u]));
            if (rank == 0) warp_arrive(ms.full[u]);
          }
          asked += kPer;
          ++asked_units;
        }
      };
      int page[2], in_page[2];
      place(0, page[0], in_page[0]);
      place(1, page[1], in_page[1]);
      if (n > 0) keys(0, page[0], in_page[0]);
      for (int t = 0; t < n && ok; ++t) {
        int next_page, next_in;
        place(t + 2, next_page, next_in);
        if (t + 1 < n) keys(t + 1, page[1], in_page[1]);
        if (ok) values(t, page[0], in_page[0]);
        page[0] = page[1], in_page[0] = in_page[1];
        page[1] = next_page, in_page[1] = next_in;
      }
    } else if (warp == kScaleWarp) {
      // ================= scales =================
      const int32_t* table = a.block_table + (size_t)b * a.max_pages;
      auto bytes_of = [&](int t) {  // eight tokens of a tile to a lane
        const int p = (r0 + t) * kTok + 8 * lane;
        if (t >= n || p >= end) return make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        int page = __ldg(table + p / P);
        if (page < 0 || page >= pool.num_pages) page = 0;  // (reported by the copies)
        return __ldg(reinterpret_cast<const uint2*>(pool.pages + page_at(page, P) + 640 * P + p % P));
      };
      uint2 now = bytes_of(0);
      for (int t = 0; t < n; ++t) {
        const uint32_t k = t_base + t, buf = k & 1;
        const uint2 next = bytes_of(t + 1);
        if (k >= 2 && !(ok = warp_wait(ms.sc_empty[buf], (k >> 1) - 1, abort_flag))) break;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float f[3][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t byte = (i ? now.y : now.x) >> (8 * q) & 0xFFu;
            const int e = byte == kNanExp ? 0 : min(max((int)byte - 127, kMinExp), kMaxExp);
            f[0][q] = scale_of_byte(byte);
            f[1][q] = (float)e;
            f[2][q] = block::pow2(-e);
          }
          reinterpret_cast<float4*>(ms.ks[buf])[2 * lane + i] = make_float4(f[0][0], f[0][1], f[0][2], f[0][3]);
          reinterpret_cast<float4*>(ms.ev[buf])[2 * lane + i] = make_float4(f[1][0], f[1][1], f[1][2], f[1][3]);
          reinterpret_cast<float4*>(ms.dn[buf])[2 * lane + i] = make_float4(f[2][0], f[2][1], f[2][2], f[2][3]);
        }
        warp_arrive(ms.sc_full[buf]);
        now = next;
      }
    } else if (warp == kTailWarp) {
      // ================= the tail: zeros behind the last token that is seen =================
      if (n > 0) {
        const int t = n - 1, p0 = (r0 + t) * kTok;
        // the tile's values are the fragment's last kValues units, its last four slots
        for (int g = 0; g < S::kValues; ++g) {
          const int p = p0 + 64 * kPer * g;
          if (p + 64 * kPer <= end) continue;
          const uint32_t u = ((uint32_t)(S::kKeys + S::kValues) * (t_base + n) - S::kValues + g) % kUnits;
          if (!(ok = warp_wait(ms.here[u], tails >> u & 1, abort_flag))) break;
          tails ^= 1u << u;
          const int first = max(0, end - p);
          for (int i = first * 16 + lane; i < 64 * kPer * 16; i += 32) {  // row i / 16: eight chunks of either 128 dims
            const uint32_t sl = (9u * (t_base + n) - 4u + kPer * g + (i >> 10)) % kSlots;
            sts128(ring + sl * kSlotBytes + 8192 * (i >> 3 & 1) + (i >> 4 & 63) * 128 + (i & 7) * 16, 0u, 0u, 0u, 0u);
          }
          fence_async_smem();
          warp_arrive_pair(peer_addr(smem_addr(&ms.tail_done[u]), 0));
        }
      }
    }
    if (!ok && lane == 0 && a.status) atomicOr(a.status, RQ_STATUS_TIMEOUT);
    done_tiles += n;
    done_frags += n > 0;
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (ms.abort) break;  // uniform: no role raises it between the barrier and here

    // ---- write the rows, or the fragment's part of them ----
    if (warp < kSoftWarps) {
      ms.top[0][quarter][row] = l_run;
      soft_sync();
      float l = (ms.top[0][0][row] + ms.top[0][1][row]) + (ms.top[0][2][row] + ms.top[0][3][row]);
      if constexpr (kTwice) l += __shfl_xor_sync(0xffffffffu, l, RV);
      const bool whole = ms.f.whole;
      const int sees = valid ? (a.tree_mask ? len - a.T - 1 : len - a.T + j) : -1;
      // a row that sees nothing is zero; one whose scores are all minus infinity is NaN
      const float empty = whole && sees >= 0 ? CUDART_NAN_F : 0.f, inv = whole ? 1.f / l : 1.f;
      const bool writes = valid && (!kTwice || lane < RV);
      const int srow = RV * (int)rank + (kTwice ? row % RV : row), dim0 = 256 * tok_half + 128 * col_half;
      float* const slot = a.ws + (2ll * me + ((int)me == ms.f.range ? ms.f.range_last : 0)) * kSlotFloats;
      T* const out = reinterpret_cast<T*>(a.out) + (((size_t)b * a.T + j) * a.heads + head) * kLatentDim + dim0;
#pragma unroll 2
      for (int c = 0; c < 8; ++c) {
        float y[16];
        if (n > 0) {
          __syncwarp();
          tmem_ld16(tmem + lane_off + 128 * col_half + 16 * c, y);
          tmem_wait_ld();
          settle<16>(y);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = l == 0.f || n == 0 ? empty : y[i] * inv;
        if (!writes) continue;
        if (whole) {
          uint4* const dst = reinterpret_cast<uint4*>(out) + 2 * c;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            dst[i] = make_uint4(rope::pack2<T>(y[8 * i], y[8 * i + 1]), rope::pack2<T>(y[8 * i + 2], y[8 * i + 3]),
                                rope::pack2<T>(y[8 * i + 4], y[8 * i + 5]), rope::pack2<T>(y[8 * i + 6], y[8 * i + 7]));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4*>(slot)[(dim0 / 4 + 4 * c + i) * kUR + srow] =
                make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
        }
      }
      if (!whole && quarter == 0 && writes) {
        slot[kUR * kLatentDim + srow] = m_run;
        slot[kUR * kLatentDim + kUR + srow] = l;
      }
    }
    fence_before_sync();
    __syncthreads();  // ms.f and the rows' sums are written again
    fence_after_sync();
  }
  if (ms.abort) {  // copies in flight land before the block ends: a millisecond is many times what one takes
    const long long start = clock64();
    while (clock64() - start < 2000000) __nanosleep(1000);
  }
  fence_before_sync();
  __syncthreads();
  cluster_sync();  // the peer is done with this CTA's operands and barriers
  fence_after_sync();
  if (warp == kMmaWarp) pair_tmem_dealloc(*(volatile uint32_t*)&ms.tmem, 512);
}

// Joins the parts of units that span ranges.  A CTA takes 8 rows and 32 / G groups of 4 dims of a unit, its parts in G shares.
template <typename T, int G>
__global__ void __launch_bounds__(256) latent_join_kernel(const LatentAttnArgs a, const int4* info, int row_groups, int unit_rows) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float part[G][32 / G][8][6];
  const int tid = threadIdx.x, r8 = tid & 7, d = (tid >> 3) % (32 / G), share = (tid >> 3) / (32 / G);
  const long long unit = blockIdx.x / row_groups;
  const int4 u = __ldcg(info + unit);
  if (u.y == 0) return;
  const long long n_rows = (long long)a.T * a.heads;
  const int n_rt = (int)((n_rows + unit_rows - 1) / unit_rows), b = (int)(unit / n_rt), rt = (int)(unit % n_rt);
  const int srow = 8 * (int)(blockIdx.x % row_groups) + r8, d4 = blockIdx.y * (32 / G) + d;
  const long long urow = (long long)rt * unit_rows + srow;
  const bool valid = urow < n_rows;
  float m = kNone, l = 0.f;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  if (valid) {
#pragma unroll 4
    for (int f = share; f < u.y; f += G) {
      const float* s = a.ws + (2ll * (u.x + f) + (f == 0 ? u.z : 0)) * kSlotFloats;
      const float mf = __ldcg(s + unit_rows * kLatentDim + srow), lf = __ldcg(s + unit_rows * kLatentDim + unit_rows + srow);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(s) + d4 * unit_rows + srow);
      const float to = fmaxf(m, mf), wa = ex2(m - to), w = ex2(mf - to);
      m = to;
      l = fmaf(l, wa, lf * w);
      y.x = fmaf(y.x, wa, v.x * w), y.y = fmaf(y.y, wa, v.y * w), y.z = fmaf(y.z, wa, v.z * w), y.w = fmaf(y.w, wa, v.w * w);
    }
  }
  if (G > 1) {
    float* p = part[share][d][r8];
    p[0] = m, p[1] = l, p[2] = y.x, p[3] = y.y, p[4] = y.z, p[5] = y.w;
    __syncthreads();
    if (share > 0) return;
#pragma unroll
    for (int g = 1; g < G; ++g) {
      const float* p = part[g][d][r8];
      const float to = fmaxf(m, p[0]), wa = ex2(m - to), w = ex2(p[0] - to);
      m = to;
      l = fmaf(l, wa, p[1] * w);
      y.x = fmaf(y.x, wa, p[2] * w), y.y = fmaf(y.y, wa, p[3] * w), y.z = fmaf(y.z, wa, p[4] * w), y.w = fmaf(y.w, wa, p[5] * w);
    }
  }
  if (!valid) return;
  const int j = (int)(urow / a.heads), head = (int)(urow % a.heads), len = __ldg(a.seq_lens + b);
  const float none = (a.tree_mask ? len - a.T - 1 : len - a.T + j) >= 0 ? CUDART_NAN_F : 0.f, inv = 1.f / l;
  y = l == 0.f ? make_float4(none, none, none, none) : make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
  T* const out = reinterpret_cast<T*>(a.out) + (((size_t)b * a.T + j) * a.heads + head) * kLatentDim + 4 * d4;
  *reinterpret_cast<uint2*>(out) = make_uint2(rope::pack2<T>(y.x, y.y), rope::pack2<T>(y.z, y.w));
}

template <typename T, int RC, int RV = RC>
cudaError_t launch(const CUtensorMap& map, const LatentPool& pool, const LatentAttnArgs& a, int box, int num_sms, int4* info, long long units,
                   cudaStream_t stream) {
  const int pairs = num_sms / 2;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, latent_kernel<T, RC, RV>, map, pool, a, box, info);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)a.T * a.heads;
  const int row_groups = (int)((rows < 2 * RV ? rows : 2 * RV) + 7) / 8;
  if (units * row_groups > 0x7fffffffLL) return cudaErrorInvalidValue;
  const bool many = units * 8 <= pairs;  // eight parts a unit or more
  cudaLaunchAttribute behind[1];
  behind[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  behind[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t join = {};
  join.gridDim = dim3((unsigned)(units * row_groups), many ? 32u : 4u);
  join.blockDim = dim3(256);
  join.stream = stream;
  join.attrs = behind;
  join.numAttrs = 1;
  return many ? cudaLaunchKernelEx(&join, latent_join_kernel<T, 8>, a, (const int4*)info, row_groups, 2 * RV)
              : cudaLaunchKernelEx(&join, latent_join_kernel<T, 1>, a, (const int4*)info, row_groups, 2 * RV);
}

}  // namespace

size_t latent_attention_workspace(int num_sms, long long rows, int max_batch) {
  const size_t parts = 2 * (size_t)(num_sms / 2) * kSlotFloats;  // two slots a pair
  return parts + 4 * (size_t)((rows + kUnitRows - 1) / kUnitRows) * (size_t)max_batch;  // and a note for each unit
}

template <typename T>
static cudaError_t prepare() {
  cudaError_t e = cudaFuncSetAttribute(latent_kernel<T, 32, 16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(latent_kernel<T, 32, 32>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(latent_kernel<T, 64, 64>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  return e;
}

cudaError_t latent_attention_prepare() {
  const cudaError_t e = prepare<__half>();
  return e == cudaSuccess ? prepare<__nv_bfloat16>() : e;
}

cudaError_t launch_latent_attention(const LatentPool& pool, const LatentAttnArgs& a, int num_sms, cudaStream_t stream) {
  if (!tensor_map_encoder()) return cudaErrorNotSupported;
  const long long units = (long long)a.B * (((long long)a.T * a.heads + kUnitRows - 1) / kUnitRows);
  const cuuint64_t P = (cuuint64_t)pool.page_size;
  const int box = pool.page_size % 64 == 0 ? 64 : pool.page_size % 32 == 0 ? 32 : 16;  // rows that stand together in a page
  CUtensorMap map;
  const cuuint64_t sizes[4] = {128, P, 5, (cuuint64_t)pool.num_pages}, strides[3] = {128, 128 * P, kLatentTokenBytes * P};
  const cuuint32_t boxes[4] = {128u, (cuuint32_t)box, 1u, 1u}, steps[4] = {1u, 1u, 1u, 1u};
  if (tensor_map_encoder()(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(pool.pages), sizes, strides, boxes, steps,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  int4* const info = reinterpret_cast<int4*>(a.ws + 2 * (size_t)(num_sms / 2) * kSlotFloats);
  const long long rows = (long long)a.T * a.heads;
  const auto of_type = [&](auto t) {
    using T = decltype(t);
    return rows <= 32   ? launch<T, 32, 16>(map, pool, a, box, num_sms, info, units, stream)
           : rows <= 64 ? launch<T, 32>(map, pool, a, box, num_sms, info, units, stream)
                        : launch<T, 64>(map, pool, a, box, num_sms, info, units, stream);
  };
  return pool.bf16 ? of_type(__nv_bfloat16()) : of_type(__half());
}

}  // namespace rq
