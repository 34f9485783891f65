// Helpers of the tcgen05 kernels whose warps are specialised: waits and arrivals of whole warps, MMAs by an elected
// lane, and two f32 operations in one instruction.
#pragma once

#include "rq_tc.cuh"

namespace rq {
namespace tc {

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
// A warp's wait, bounded (about a second) like role_wait, but asleep between its looks at the
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
// A look at a barrier whose result is wanted later: a wait that finds it ready takes some 200 cycles, which a look ahead
// spends beside other work.  warp_wait_after: the wait, unless the look found it ready.
__device__ __forceinline__ uint32_t warp_look(const uint64_t& bar, uint32_t parity) {
  uint32_t done;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(done)
               : "r"(smem_addr(&bar)), "r"(parity & 1)
               : "memory");
  return done;
}
__device__ __forceinline__ bool warp_wait_after(uint32_t look, const uint64_t& bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, look) || warp_wait(bar, parity, abort_flag);
}
// A warp's arrival, by one lane (a predicate, no branch) behind all lanes' accesses.
__device__ __forceinline__ void warp_arrive(uint64_t& bar) {
  __syncwarp();
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n @e mbarrier.arrive.shared::cta.b64 _, [%0];\n}" ::"r"(
                   smem_addr(&bar))
               : "memory");
}
// The MMAs and commit of rq_tc.cuh, by one elected lane of a whole warp: with the operands uniform over the
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
// ---- pairs of CTAs (cta_group::2): the even CTA of a cluster leads and issues the MMAs of both ----

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
// The address of a CTA's shared memory in the cluster's window, and loads from there.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ float peer_ld(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
// A warp's arrival at a barrier of the pair's leader (its address in the cluster's window).  What it announces is in tensor
// memory, or in shared memory behind a proxy fence, and is complete before (the waits for stores, the fence), so the arrival
// has no writes to bring along: released at the cluster's scope it took some 1,400 cycles.
__device__ __forceinline__ void warp_arrive_pair(uint32_t bar) {
  __syncwarp();
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n @e mbarrier.arrive.shared::cluster.b64 _, [%0];\n}" ::"r"(bar)
               : "memory");
}
// An arrival that expects bytes of copies, by an elected lane.
__device__ __forceinline__ void elect_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n}" ::"r"(bar),
               "r"(bytes)
               : "memory");
}
// MMAs over the pair's operands and accumulators, and a commit that arrives at this barrier of both.
__device__ __forceinline__ void pair_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate));
}
__device__ __forceinline__ void pair_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, e;\n elect.sync _|e, 0xffffffff;\n setp.ne.b32 p, %4, 0;\n"
      " @e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(accumulate));
}
// cta_mask: the pair's two CTAs of the cluster.
__device__ __forceinline__ void pair_commit(uint32_t mbar, uint32_t cta_mask) {
  asm volatile(
      "{\n .reg .pred e;\n .reg .b16 m;\n cvt.u16.u32 m, %1;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}" ::"r"(mbar),
      "r"(cta_mask)
      : "memory");
}
__device__ __forceinline__ void pair_tmem_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}

// Loaded registers, not to be used before this point: behind the wait for the loads (no instruction).
template <int N>
__device__ __forceinline__ void settle(float* v) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

}  // namespace tc
}  // namespace rq
