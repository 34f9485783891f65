// Causal attention of new tokens in the expanded form of latent attention, sequences packed one after the other: heads of
// 192 (128 of their own and 64 that all heads share) against values of 128, on the 5th-generation tensor cores.
//
// score = scale (q[:128] . k + q[128:] . k_pe), out = sum softmax(score) v, in one pass over the keys with a running maximum
// and sum.  What bounds it is the tensor cores' rate: 640 flops a visible (row, key) of a head.
//
// A pair of CTAs (two SMs) takes 512 query rows of one (sequence, head), two blocks of 256, 128 rows of each block to a
// CTA, and walks the keys in tiles of 128.  Its MMAs span both (M = 256): each CTA holds half of a tile's keys and half of its
// values' dims, 40 KB a tile instead of 80, so that three tiles stand beside the 96 KB of queries.  (One CTA alone, with
// 1.6 tiles, waited for its loads: 4,950 cycles a tile, 1 x 16,384 x 16 heads 1,134 us.)  Warps are specialised and
// coupled through mbarriers:
//   softmax (warps 0-7 of both, a thread per row): takes its row of S from tensor memory into registers, masks, writes
//     16-bit weights over S (their MMA's operands have the values' type, so bf16 outputs are up to 1.4 times as far from the 64-bit
//     result as with f32 weights; two pieces a weight would double the MMAs over the values; the sum takes them unrounded);
//   MMA (warp 8 of the leader): for each block in turn O_b += W_b V(t) and behind it S_b(t + 1) = Q_b K(t + 1)^T, so that one block
//     is on the tensor cores while the other is in its softmax;
//   copies (warp 9 of both): TMA tiles straight from the caller's tensors, whatever their strides;
//   values (warps 10, 11 of both): in tiles that some row of the pair sees in part, values that are not finite are taken
//     out before the weights, zeros among them, are multiplied with them, and given to the rows that see them at the end.
// Tensor memory: O_b at columns 128 b, S_b at 256 + 128 b with W_b over its first half.
// The units with the most keys go first, and neighbouring pairs take neighbouring heads, whose rows share DRAM pages.  (Tiles of
// all units cut into one even range a pair, pairs at unrelated places: 1 x 16,384 x 16 heads 846 -> 1,419 us.)  Where units
// are few, or the last ones leave pairs idle, they are cut into parts, whose (m, l, out) a second kernel joins.
// Every wait is bounded: one that runs out sets RQ_STATUS_TIMEOUT and an abort flag every role polls.
//
// Device time, bf16: 1 x 16,384 x 16 heads 836 to 863 us (1,640 to 1,590 TFLOP/s, 85 to 83% of the burst rate; 892 under the power cap),
// 4 x 512 over 7,680 x 64 heads 450 to 460 us (1,450, 75%), 8,192 x 8 heads 120 us; six prompts of 1 to 400 x 5 heads fp16 24 to 28 us: one
// unit's opening, four tiles and closing, one after the other (not cut: a part has at least four tiles).
#include <math_constants.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>
#include <type_traits>

#include "../../include/rq.h"
#include "rq_roles.cuh"
#include "rq_rope.cuh"
#include "rq_tma.h"

namespace rq {
namespace {

using namespace tc;

constexpr int kSoftWarps = 8, kFixWarps = 2, kMmaWarp = 8, kCopyWarp = 9, kFixWarp = 10, kThreads = 384;
constexpr int kHalf = 128, kRows = 256, kUnitRows = 512;  // rows of a block in a CTA, of a CTA, of a pair
constexpr int kTok = 128, kDim = 128;
constexpr int kStages = 3;                               // tiles of keys, and of values
constexpr uint32_t kChunk = 16384;                       // 128 rows of 64 dims
constexpr uint32_t kQBytes = 6 * kChunk, kKBytes = 3 * kChunk / 2, kVBytes = kChunk;  // a CTA's
constexpr uint32_t kColS = 256;
constexpr float kLift = 7.f, kReach = 15.f;      // weights are 2^(score - m), m between maximum - kReach and maximum - kLift
constexpr float kNone = -3.402823466e38f;        // m before any visible key
// |maximum| from which weights are formed in two roundings: m comes from the rounded product, and a weight from an exact one would be
// off by half of a step there, a factor of 2^(2^-4) at 2^20, past fp16's range from 2^24 on
constexpr float kLarge = 1048576.f;

struct Misc {
  // the leader's: K(t), V(t), the queries are there; [block] W(t); the values' warps are through with a tile
  uint64_t k_full[kStages], v_full[kStages], q_full, p_full[2], fix_done[kStages];
  // both CTAs': K(t), V(t) are read; [block] S(t); [block] the last W V; drained; a CTA's values of a tile seen in part
  uint64_t k_empty[kStages], v_empty[kStages], s_full[2], o_done[2], drain, v_here[kStages];
  uint32_t tmem;
  int abort, any;
  int from[3][kDim / 2];   // first key with +inf, -inf, NaN among the values of a dim of the CTA's half
};
constexpr uint32_t kOffK = kQBytes, kOffV = kOffK + kStages * kKBytes, kOffMisc = kOffV + kStages * kVBytes;
constexpr int kSmem = (int)(kOffMisc + sizeof(Misc)) + 1024;
static_assert(kSmem <= 232448, "one CTA's shared memory");
// floats of a part's slot: 512 rows x 128 (as [dim / 4][row][4]), then the rows' m and l
constexpr size_t kSlotFloats = (size_t)kUnitRows * kDim + 2 * kUnitRows;
constexpr int kSlotsPerPair = 4;

// Instruction descriptor of kind::f16 for T (fp16 0, bf16 1 at bits 7 and 10); bit 16: B with N along its rows.
template <typename T>
__host__ __device__ constexpr uint32_t idesc(int M, int N, int b_rows) {
  const uint32_t type = std::is_same<T, __half>::value ? 0u : 1u;
  return idesc_f16(M, N) | type << 7 | type << 10 | (uint32_t)b_rows << 16;
}
// A box of the tensor to this CTA's shared memory; the bytes count at a barrier of the leader (pair_bar), or of this CTA.
__device__ __forceinline__ void load_pair(uint32_t dst, const CUtensorMap& map, int x, int y, int z, uint32_t pair_bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];\n}"
      ::"r"(dst), "l"(&map), "r"(x), "r"(y), "r"(z), "r"(pair_bar)
      : "memory");
}
__device__ __forceinline__ void load_here(uint32_t dst, const CUtensorMap& map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n}" ::"r"(dst),
      "l"(&map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
      "%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]),
        "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
struct Maps {
  CUtensorMap q, k, pe, v;
};

// Units in order: rows r0 .. r0 + 511 of a sequence, the ones with the most keys first, each for all heads.  The last ones may be
// cut: units from `whole` on have `splits` parts each.
struct Cut {
  int n_rb, whole, splits;
};

// dual: calls of no more than 256 queries a sequence.  They fill one block only: both blocks take them, one the even tiles and
// one the odd, so that here too one is on the tensor cores while the other is in its softmax; joined at the end.  2 x 100
// rows over 4,000 x 128 heads 250 -> 177 us.  (As a choice of each unit's in one kernel it cost the others 3 to 4%.)
template <typename T, bool dual>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ Maps maps, const PromptArgs a, const Cut cut) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = smem_addr(smem_raw) + (1024 - (smem_addr(smem_raw) & 1023) & 1023);
  Misc& ms = *reinterpret_cast<Misc*>(smem_raw + (base - smem_addr(smem_raw)) + kOffMisc);
  const uint32_t q_ops = base, k_ring = base + kOffK, v_ring = base + kOffV;
  volatile int* const abort_flag = &ms.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank(), pair_id = blockIdx.x >> 1, heads = (uint32_t)a.q.heads;

  // ---- the pair's unit, or part of one ----
  const bool is_part = pair_id >= (uint32_t)cut.whole;
  const uint32_t part_id = is_part ? pair_id - (uint32_t)cut.whole : 0u, splits = is_part ? (uint32_t)cut.splits : 1u;
  const uint32_t unit = is_part ? (uint32_t)cut.whole + part_id / splits : pair_id, part = part_id % splits;
  const int h = (int)(unit % heads), b = (int)(unit / heads % (uint32_t)a.B), turn = (int)(unit / heads / (uint32_t)a.B);
  const int q0 = __ldg(a.q_offsets + b), q1 = __ldg(a.q_offsets + b + 1), k0 = __ldg(a.k_offsets + b), k1 = __ldg(a.k_offsets + b + 1);
  if (q0 < 0 || q1 < q0 || q1 > a.nq || k0 < 0 || k1 < k0 || k1 > a.nk || q1 - q0 > a.max_new) {
    if (tid == 0 && a.status) atomicOr(a.status, RQ_STATUS_BAD_LEN);
    return;
  }
  const int nq = q1 - q0, nk = k1 - k0, ahead = nk - nq, n_rb = (nq + kUnitRows - 1) / kUnitRows;
  if (turn >= n_rb) return;  // (both CTAs of the pair)
  const int r0 = (n_rb - 1 - turn) * kUnitRows;
  // tiles that a block's rows see, and this part's range of them
  auto tiles_to = [&](int row) { return max(0, (ahead + min(nq, row) + kTok - 1) / kTok); };
  const int all0 = tiles_to(r0 + kRows), all1 = r0 + kRows < nq ? tiles_to(r0 + kUnitRows) : 0, all = max(all0, all1);
  const int t_first = (int)((long long)part * all / splits), t_end = (int)((long long)(part + 1) * all / splits);
  const int n = t_end - t_first;
  const int n_b[2] = {dual ? (n + 1) / 2 : min(max(all0 - t_first, 0), n), dual ? n / 2 : min(max(all1 - t_first, 0), n)};
  // from this tile on, rows of the pair see tiles in part
  const int t_fix = max(0, max(0, ahead + r0 + 1) / kTok - t_first);

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_addr(&ms.k_full[i]), 1);
      mbar_init(smem_addr(&ms.v_full[i]), 1);
      mbar_init(smem_addr(&ms.k_empty[i]), 1);
      mbar_init(smem_addr(&ms.v_empty[i]), 1);
      mbar_init(smem_addr(&ms.v_here[i]), 1);
      mbar_init(smem_addr(&ms.fix_done[i]), 2 * kFixWarps);
    }
    mbar_init(smem_addr(&ms.q_full), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&ms.s_full[i]), 1);
      mbar_init(smem_addr(&ms.p_full[i]), kSoftWarps);  // four warps of either CTA
      mbar_init(smem_addr(&ms.o_done[i]), 1);
    }
    mbar_init(smem_addr(&ms.drain), 1);
    ms.abort = 0;
    ms.any = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int i = tid; i < 3 * kDim / 2; i += kThreads) (&ms.from[0][0])[i] = INT32_MAX;
  __syncwarp();
  if (warp == kMmaWarp) pair_tmem_alloc(smem_addr(&ms.tmem), 512);
  fence_before_sync();
  __syncthreads();
  cluster_sync();  // the peer's barriers are there
  fence_after_sync();
  const uint32_t tmem = *(volatile uint32_t*)&ms.tmem;
  const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
  const int blk = warp >> 2 & 1, brow = 32 * (warp & 3) + lane, row = r0 + (dual ? 0 : kRows * blk) + kHalf * (int)rank + brow;
  const bool valid = row < nq;
  const int qpos = valid ? ahead + row : -1;  // the last key that the row sees
  float m_run = kNone, l_run = 0.f;
  bool ok = true;

  if (warp < kSoftWarps) {
    // ================= softmax: one thread per row =================
    const float scale = a.sm_scale * 1.44269504088896340736f;
    const uint32_t s_tile = tmem + lane_off + kColS + 128 * blk, o_cols = tmem + lane_off + 128 * blk;
    float from = 0.f;
    for (int t = 0; t < n_b[blk]; ++t) {
      const int t0 = (t_first + (dual ? 2 * t + blk : t)) * kTok;
      ok = warp_wait(ms.s_full[blk], t, abort_flag);  // S_b(t), and W_b(t - 1) V before it
      if (!ok) break;
      fence_after_sync();
      float s[kTok];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(s_tile + 32 * c, s + 32 * c);
      tmem_wait_ld();
      settle<kTok>(s);
      if (t0 + kTok - 1 > qpos) {
#pragma unroll
        for (int c = 0; c < kTok; ++c)
          if (t0 + c > qpos) s[c] = -CUDART_INF_F;
      }
      float top[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
      for (int c = 4; c < kTok; c += 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = c + 4 + i < kTok ? max3(top[i], s[c + i], s[c + 4 + i]) : fmaxf(top[i], s[c + i]);
      }
      const float most = __fmul_rn(fmaxf(max3(top[0], top[1], top[2]), top[3]), scale);
      const float above = most - (m_run == kNone ? -CUDART_INF_F : m_run);  // (NaN where nothing is seen: no move)
      if (__any_sync(0xffffffffu, above > kReach)) {
        float alpha = 1.f;
        if (above > kReach) {
          from = most - kLift;
          alpha = ex2(m_run - from);
          m_run = from;
          l_run *= alpha;
        }
        if (t > 0) {  // O *= alpha (the warp's rows)
#pragma unroll 1
          for (int c = 0; c < kDim / 16; ++c) {
            float v[16];
            tmem_ld16(o_cols + 16 * c, v);
            tmem_wait_ld();
            settle<16>(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= alpha;
            tmem_st16(o_cols + 16 * c, v);
          }
        }
      }
      {
        uint64_t f = pair(scale, scale);
        const uint64_t d = pair(-from, -from);
        if (__any_sync(0xffffffffu, fabsf(from) > kLarge)) {  // products rounded as the maximum's, not in one operation with the difference
          const uint64_t none = pair(-0.f, -0.f);
#pragma unroll
          for (int c = 0; c < kTok; c += 2) fma2(s[c], s[c + 1], f, none);
          f = pair(1.f, 1.f);
        }
#pragma unroll
        for (int c = 0; c < kTok; c += 2) fma2(s[c], s[c + 1], f, d);
      }
      uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
      for (int c = 0; c < kTok; c += 32) {
        uint32_t pw[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float w0 = ex2(s[c + i]), w1 = ex2(s[c + i + 1]);
          add2(sum[i >> 1 & 1], w0, w1);
          pw[i >> 1] = rope::pack2<T>(w0, w1);
        }
        tmem_st16u(s_tile + c / 2, pw);
      }
      float x[4];
      unpair(sum[0], x[0], x[1]);
      unpair(sum[1], x[2], x[3]);
      l_run += (x[0] + x[1]) + (x[2] + x[3]);
      tmem_wait_st();
      fence_before_sync();
      warp_arrive_pair(peer_addr(smem_addr(&ms.p_full[blk]), 0));
    }
    if (ok && n_b[blk] > 0) ok = warp_wait(ms.o_done[blk], 0, abort_flag);
    fence_after_sync();
  } else if (warp == kMmaWarp) {
    // ================= MMA issue: the leader's =================
    if (rank == 0 && n > 0) {
      constexpr uint32_t id_s = idesc<T>(kRows, kTok, 0), id_o = idesc<T>(kRows, kDim, 1);
      const int last_b = !dual && n_b[1] > 0 ? 1 : 0;  // the block that uses a tile last (dual: the one that uses it)
      bool issued = false;
      auto wait = [&](uint64_t& bar, uint32_t parity) { return ok = warp_wait(bar, parity, abort_flag); };
      auto s_mmas = [&](int bb, int t) {  // S_b(t)
        const int st = t % kStages;
        if (!wait(ms.k_full[st], t / kStages)) return;
        const uint32_t q_at = q_ops + 3 * bb * kChunk, k_at = k_ring + st * kKBytes;
#pragma unroll
        for (int ks = 0; ks < 12; ++ks)
          pair_mma_ss(tmem + kColS + 128 * bb, sdesc(q_at + (ks >> 2) * kChunk + 32 * (ks & 3)),
                      sdesc(k_at + (ks >> 2) * (kChunk / 2) + 32 * (ks & 3)), id_s, ks > 0);
        issued = true;
        if ((dual || bb == last_b) && t + kStages < n) pair_commit(smem_addr(&ms.k_empty[st]), 3);
        pair_commit(smem_addr(&ms.s_full[bb]), 3);
      };
      wait(ms.q_full, 0);
#pragma unroll
      for (int bb = 0; bb < 2; ++bb)
        if (ok && n_b[bb] > 0) s_mmas(bb, dual ? bb : 0);
      for (int t = 0; t < n && ok; ++t) {
        const int st = t % kStages;
        if (!wait(ms.v_full[st], t / kStages)) break;
        if (t >= t_fix && !wait(ms.fix_done[st], (t - t_fix) / kStages)) break;
#pragma unroll
        for (int bb = 0; bb < 2; ++bb) {
          const int i = dual ? t >> 1 : t;  // the block's tile
          if (!ok || (dual ? bb != (t & 1) : t >= n_b[bb])) continue;
          if (!wait(ms.p_full[bb], i)) break;
          fence_after_sync();
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)  // keys 16 ks ..
            pair_mma_ts(tmem + 128 * bb, tmem + kColS + 128 * bb + 8 * ks, sdesc(v_ring + st * kVBytes + 2048 * ks), id_o, i > 0 || ks > 0);
          if ((dual || bb == last_b) && t + kStages < n) pair_commit(smem_addr(&ms.v_empty[st]), 3);
          if (i + 1 < n_b[bb])
            s_mmas(bb, dual ? t + 2 : t + 1);  // over the same columns, behind the MMAs that read them
          else
            pair_commit(smem_addr(&ms.o_done[bb]), 3);
        }
      }
      if (!ok && issued) {  // nothing may be running when the tensor memory is freed
        pair_commit(smem_addr(&ms.drain), 3);
        for (int i = 0; i < kWaitLimit; ++i)
          if (mbar_test(smem_addr(&ms.drain), 0u)) break;
      }
    }
  } else if (warp == kCopyWarp) {
    // ================= copies: this CTA's share =================
    if (n > 0) {
      if (rank == 0) elect_expect(smem_addr(&ms.q_full), 2 * kQBytes);
      const uint32_t bar = peer_addr(smem_addr(&ms.q_full), 0);
#pragma unroll
      for (int i = 0; i < 6; ++i)
        load_pair(q_ops + i * kChunk, maps.q, 64 * (i % 3), h, q0 + r0 + (dual ? 0 : kRows * (i / 3)) + kHalf * (int)rank, bar);
    }
    for (int t = 0; t < n && ok; ++t) {
      const int st = t % kStages, z = k0 + (t_first + t) * kTok;
      if (t >= kStages && !(ok = warp_wait(ms.k_empty[st], t / kStages - 1, abort_flag))) break;
      if (rank == 0) elect_expect(smem_addr(&ms.k_full[st]), 2 * kKBytes);
      const uint32_t kbar = peer_addr(smem_addr(&ms.k_full[st]), 0), dst = k_ring + st * kKBytes;
      const int zk = z + kTok / 2 * (int)rank;  // this CTA's 64 keys
      load_pair(dst, maps.k, 0, h, zk, kbar);
      load_pair(dst + kChunk / 2, maps.k, 64, h, zk, kbar);
      load_pair(dst + kChunk, maps.pe, 0, 0, zk, kbar);
      if (t >= kStages && !(ok = warp_wait(ms.v_empty[st], t / kStages - 1, abort_flag))) break;
      if (t < t_fix) {
        if (rank == 0) elect_expect(smem_addr(&ms.v_full[st]), 2 * kVBytes);
        load_pair(v_ring + st * kVBytes, maps.v, 64 * (int)rank, h, z, peer_addr(smem_addr(&ms.v_full[st]), 0));
      } else {  // seen in part: the values' warps of this CTA first
        elect_expect(smem_addr(&ms.v_here[st]), kVBytes);
        load_here(v_ring + st * kVBytes, maps.v, 64 * (int)rank, h, z, smem_addr(&ms.v_here[st]));
        if (rank == 0) warp_arrive(ms.v_full[st]);
      }
    }
  } else if (warp < kFixWarp + kFixWarps) {
    // ================= values that are not finite, in tiles seen in part =================
    // 16-bit halves whose exponent is all ones, two to a word
    constexpr bool kF16 = std::is_same<T, __half>::value;
    constexpr uint32_t kExp = kF16 ? 0x7C007C00u : 0x7F807F80u, kOne = kF16 ? 0x04000400u : 0x00800080u;
    for (int t = t_fix; t < n; ++t) {
      const int st = t % kStages;
      if (!(ok = warp_wait(ms.v_here[st], (t - t_fix) / kStages, abort_flag))) break;
      bool any = false;
      for (int r8 = warp - kFixWarp; r8 < kTok / 4; r8 += kFixWarps) {  // a row (key) is eight chunks
        const int r = 4 * r8 + (lane >> 3), chunk = lane & 7;
        const uint32_t addr = v_ring + st * kVBytes + sw128(r, chunk);
        const uint4 v = lds128(addr);
        const uint32_t odd = ((v.x & kExp) + kOne) | ((v.y & kExp) + kOne) | ((v.z & kExp) + kOne) | ((v.w & kExp) + kOne);
        if (!(odd & 0x80008000u)) continue;
        const int key = (t_first + t) * kTok + r;
        uint32_t w[4];
        for (int k = 0; k < 4; ++k) {
          w[k] = word(v, k);
          for (int s = 0; s < 2; ++s) {
            const uint32_t x = w[k] >> (16 * s) & 0xFFFFu, e = kExp & 0xFFFFu;
            if ((x & e) != e) continue;
            const int kind = (x & 0x7FFFu) != e ? 2 : x >> 15 ? 1 : 0;
            if (key < nk) {
              atomicMin(&ms.from[kind][8 * chunk + 2 * k + s], key);
              ms.any = 1;
            }
            w[k] &= s ? 0x0000FFFFu : 0xFFFF0000u;
          }
        }
        sts128(addr, w[0], w[1], w[2], w[3]);
        any = true;
      }
      if (any) fence_async_smem();
      warp_arrive_pair(peer_addr(smem_addr(&ms.fix_done[st]), 0));
    }
  }
  if (!ok && lane == 0 && a.status) atomicOr(a.status, RQ_STATUS_TIMEOUT);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const bool aborted = ms.abort != 0;
  if (aborted) {  // copies in flight land before the block ends: a millisecond is many times what one takes
    const long long start = clock64();
    while (clock64() - start < 2000000) __nanosleep(1000);
  }
  cluster_sync();  // the peer is done with this CTA's operands, and its values' warps have left what they found

  // ---- write the rows, or the part of them ----
  float* const other = reinterpret_cast<float*>(smem_raw + (base - smem_addr(smem_raw)));  // over the operands: [dim / 4][row][4], m, l
  if (dual) {
    if (blk == 1 && warp < kSoftWarps && !aborted) {
#pragma unroll 1
      for (int c = 0; c < kDim / 16; ++c) {
        float y[16];
        if (n_b[1] > 0) {
          tmem_ld16(tmem + lane_off + 128 + 16 * c, y);
          tmem_wait_ld();
          settle<16>(y);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          reinterpret_cast<float4*>(other)[(4 * c + i) * kHalf + brow] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
      }
      other[kHalf * kDim + brow] = m_run;
      other[kHalf * kDim + kHalf + brow] = l_run;
    }
    __syncthreads();
  }
  if (warp < kSoftWarps && !aborted && !(dual && blk == 1)) {
    float w0 = 1.f, w1 = 0.f;  // dual: the factors of the two blocks' rows
    if (dual) {
      const float m1 = other[kHalf * kDim + brow], l1 = other[kHalf * kDim + kHalf + brow], to = fmaxf(m_run, m1);
      w0 = ex2(m_run - to), w1 = ex2(m1 - to);
      l_run = fmaf(l_run, w0, l1 * w1);
      m_run = to;
    }
    // a row whose scores are all minus infinity; one that sees nothing
    const float empty = !is_part && qpos >= 0 ? CUDART_NAN_F : 0.f, inv = is_part ? 1.f : 1.f / l_run;
    // what the values' warps found: dims 64 r .. of the pair's CTA r
    int odd[2];
    for (int r = 0; r < 2; ++r) odd[r] = __float_as_int(peer_ld(peer_addr(smem_addr(&ms.any), r)));
    auto first_of = [&](int kind, int d) { return __float_as_int(peer_ld(peer_addr(smem_addr(&ms.from[kind][d & 63]), d >> 6))); };
    float* const slot = a.ws + (size_t)part_id * kSlotFloats;
    T* const out = reinterpret_cast<T*>(a.out) + (((size_t)q0 + row) * heads + h) * kDim;
#pragma unroll 2
    for (int c = 0; c < kDim / 16; ++c) {
      float y[16];
      if (n_b[blk] > 0) {
        __syncwarp();
        tmem_ld16(tmem + lane_off + 128 * blk + 16 * c, y);
        tmem_wait_ld();
        settle<16>(y);
        if (dual) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 v = reinterpret_cast<const float4*>(other)[(4 * c + i) * kHalf + brow];
            y[4 * i] = fmaf(y[4 * i], w0, v.x * w1), y[4 * i + 1] = fmaf(y[4 * i + 1], w0, v.y * w1);
            y[4 * i + 2] = fmaf(y[4 * i + 2], w0, v.z * w1), y[4 * i + 3] = fmaf(y[4 * i + 3], w0, v.w * w1);
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = l_run == 0.f ? empty : y[i] * inv;
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = empty;
      }
      if (!valid) continue;
      if (odd[c >> 2]) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (first_of(0, 16 * c + i) <= qpos) y[i] += CUDART_INF_F;
          if (first_of(1, 16 * c + i) <= qpos) y[i] -= CUDART_INF_F;
          if (first_of(2, 16 * c + i) <= qpos) y[i] = CUDART_NAN_F;
        }
      }
      if (!is_part) {
        uint4* const dst = reinterpret_cast<uint4*>(out) + 2 * c;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          dst[i] = make_uint4(rope::pack2<T>(y[8 * i], y[8 * i + 1]), rope::pack2<T>(y[8 * i + 2], y[8 * i + 3]),
                              rope::pack2<T>(y[8 * i + 4], y[8 * i + 5]), rope::pack2<T>(y[8 * i + 6], y[8 * i + 7]));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          reinterpret_cast<float4*>(slot)[(4 * c + i) * kUnitRows + (row - r0)] =
              make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
      }
    }
    if (is_part && valid) {
      slot[kUnitRows * kDim + (row - r0)] = m_run;
      slot[kUnitRows * kDim + kUnitRows + (row - r0)] = l_run;
    }
  }
  fence_before_sync();
  __syncthreads();
  cluster_sync();  // a peer's shared memory is read until here
  fence_after_sync();
  if (warp == kMmaWarp) pair_tmem_dealloc(tmem, 512);
}

// Joins a unit's parts.  A CTA takes 8 rows, a thread 4 dims of one.
template <typename T>
__global__ void __launch_bounds__(256) prompt_join_kernel(const PromptArgs a, const Cut cut) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t unit = (uint32_t)cut.whole + blockIdx.x, heads = (uint32_t)a.q.heads;
  const int h = (int)(unit % heads), b = (int)(unit / heads % (uint32_t)a.B), turn = (int)(unit / heads / (uint32_t)a.B);
  const int q0 = __ldg(a.q_offsets + b), q1 = __ldg(a.q_offsets + b + 1), k0 = __ldg(a.k_offsets + b), k1 = __ldg(a.k_offsets + b + 1);
  if (q0 < 0 || q1 < q0 || q1 > a.nq || k0 < 0 || k1 < k0 || k1 > a.nk || q1 - q0 > a.max_new) return;
  const int nq = q1 - q0, n_rb = (nq + kUnitRows - 1) / kUnitRows;
  if (turn >= n_rb) return;
  const int srow = 8 * (int)blockIdx.y + (threadIdx.x & 7), d4 = threadIdx.x >> 3, row = (n_rb - 1 - turn) * kUnitRows + srow;
  if (row >= nq) return;
  const float* s = a.ws + (size_t)blockIdx.x * cut.splits * kSlotFloats;
  float m = kNone, l = 0.f;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int f = 0; f < cut.splits; ++f, s += kSlotFloats) {
    const float mf = __ldcg(s + kUnitRows * kDim + srow), lf = __ldcg(s + kUnitRows * kDim + kUnitRows + srow);
    const float4 v = __ldcg(reinterpret_cast<const float4*>(s) + d4 * kUnitRows + srow);
    const float to = fmaxf(m, mf), wa = ex2(m - to), w = ex2(mf - to);
    m = to;
    l = fmaf(l, wa, lf * w);
    y.x = fmaf(y.x, wa, v.x * w), y.y = fmaf(y.y, wa, v.y * w), y.z = fmaf(y.z, wa, v.z * w), y.w = fmaf(y.w, wa, v.w * w);
  }
  const float none = k1 - k0 - nq + row >= 0 ? CUDART_NAN_F : 0.f, inv = 1.f / l;
  y = l == 0.f ? make_float4(none, none, none, none) : make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
  *reinterpret_cast<uint2*>(reinterpret_cast<T*>(a.out) + (((size_t)q0 + row) * heads + h) * kDim + 4 * d4) =
      make_uint2(rope::pack2<T>(y.x, y.y), rope::pack2<T>(y.z, y.w));
}

// Boxes of 64 dims and `box` rows of one head of x [n][heads][dims].
bool encode(CUtensorMap* map, bool bf16, const HeadsDev& x, int dims, int n, int box) {
  const cuuint64_t sizes[3] = {(cuuint64_t)dims, (cuuint64_t)x.heads, (cuuint64_t)n};
  // a stride that is not used (one head, one row) may be anything
  const cuuint64_t strides[2] = {(cuuint64_t)(x.heads > 1 ? x.head_stride : dims) * 2, (cuuint64_t)(n > 1 ? x.stride : dims) * 2};
  const cuuint32_t boxes[3] = {64u, 1u, (cuuint32_t)box}, steps[3] = {1u, 1u, 1u};
  return tensor_map_encoder()(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(x.x), sizes, strides,
                   boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Which units are cut, at the batch's mean lengths.  Units of one size (no more than 512 queries a sequence): the ones that would
// have the last round of pairs to themselves, so that their parts fill it.  Units of several sizes (causal over more rows): all,
// where the longest would outlast an even share of the work.  A part opens and closes in the time of some 4 tiles, so it has
// at least that many; and there is a slot for each.
// Device time, us, without and with: 4 x 512 of 8K x 64 heads (256 units on 76 pairs) 490 | 449; 8,192 x 8 heads (128 units of 4 to
// 64 tiles, share 57) 127 | 174, not cut; 8,192 x 2 heads 118 | 65; 2 x 1,024 over 7K x 4 heads 117 | 67; 64 over 16K x 2 heads 232 | 31.
Cut cut_of(const PromptArgs& a, long long units, int n_rb) {
  const int pairs = a.num_sms / 2;
  const double rows = (double)a.nq / a.B, keys = (double)a.nk / a.B, longest = keys / kTok + 1.0;
  Cut c{n_rb, (int)units, 1};
  if (units >= 6ll * pairs) return c;
  long long cut = units % pairs, splits = cut > 0 ? pairs / cut : 1;
  if (n_rb > 1) {
    // (at least a tile: rows of no sequence, or sequences with fewer keys than queries, would make it nothing)
    const double share = fmax(1.0, (keys - 0.5 * rows + kUnitRows / 2) / kTok * (rows / kUnitRows) * a.B * a.q.heads / pairs);
    cut = units;
    splits = longest > 1.25 * share ? (long long)(longest / share) + 1 : 1;
  }
  if (cut > 0) splits = std::min({splits, (long long)(longest / 4), (long long)kSlotsPerPair * pairs / cut});
  if (splits > 1) c.whole = (int)(units - cut), c.splits = (int)splits;
  return c;
}

template <typename T>
cudaError_t launch(const Maps& maps, const PromptArgs& a, int n_rb, cudaStream_t stream) {
  static_assert(sizeof(Maps) + sizeof(PromptArgs) + 32 <= 4096, "kernel parameters");
  // the kernel's shared-memory limit, once a device (at every call on those past the 64th)
  static std::atomic<unsigned long long> set{0};
  const bool dual = a.max_new <= kRows;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (!(set.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(prompt_kernel<T, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(prompt_kernel<T, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  const long long units = (long long)a.B * n_rb * a.q.heads;
  const Cut cut = cut_of(a, units, n_rb);
  const long long n_cut = units - cut.whole, n_pairs = cut.whole + n_cut * cut.splits;
  if (n_pairs > 0x3fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2u * (unsigned)n_pairs);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = dual ? cudaLaunchKernelEx(&cfg, prompt_kernel<T, true>, maps, a, cut) : cudaLaunchKernelEx(&cfg, prompt_kernel<T, false>, maps, a, cut);
  if (e != cudaSuccess || n_cut == 0) return e;
  cudaLaunchAttribute behind[1];
  behind[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  behind[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t join = {};
  join.gridDim = dim3((unsigned)n_cut, (unsigned)((a.max_new < kUnitRows ? a.max_new : kUnitRows) + 7) / 8);
  join.blockDim = dim3(256);
  join.stream = stream;
  join.attrs = behind;
  join.numAttrs = 1;
  return cudaLaunchKernelEx(&join, prompt_join_kernel<T>, a, cut);
}

}  // namespace

size_t prompt_workspace(int num_sms) { return (size_t)kSlotsPerPair * (num_sms / 2) * kSlotFloats * sizeof(float); }

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t stream) {
  if (!tensor_map_encoder()) return cudaErrorNotSupported;
  const int n_rb = (a.max_new + kUnitRows - 1) / kUnitRows;
  Maps maps{};
  HeadsDev k = a.k, v = a.v, pe{a.k_pe, a.k_pe_stride, 0, 1};
  if (a.nk == 0) k = v = pe = a.q;  // no key is ever read
  const int nk = a.nk > 0 ? a.nk : 1;
  if (!encode(&maps.q, a.bf16, a.q, kPromptDim, a.nq, kHalf) || !encode(&maps.k, a.bf16, k, kDim, nk, kTok / 2) ||
      !encode(&maps.pe, a.bf16, pe, kPositionDim, nk, kTok / 2) || !encode(&maps.v, a.bf16, v, kDim, nk, kTok))
    return cudaErrorInvalidValue;
  return a.bf16 ? launch<__nv_bfloat16>(maps, a, n_rb, stream) : launch<__half>(maps, a, n_rb, stream);
}

}  // namespace rq
