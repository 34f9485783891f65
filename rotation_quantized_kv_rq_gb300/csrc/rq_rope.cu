// Norms of queries and keys per head with the position rotation, in one pass over the rows.
//
// What bounds it: every row is read once and written once, 512 bytes, against some 10 f32 operations a
// value.  16,384 tokens x 72 heads with three axes: 102 us, 604 MB at 5.9 TB/s, 87% of the copy rate;
// there the SMs issue in 58% of the cycles.  A few tokens (16 x 40 heads: 3.4 us) are one chain of
// latencies: the position, the cosine, the row, the norm's sum.
#include "rq_rope.cuh"

namespace rq {
namespace {

using namespace rope;

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // rows that a half-warp has in flight

// A half-warp takes `per` rows of one token (rows part, part + parts, ...: neighbouring half-warps
// read neighbouring rows), so that the token's cosines and sines, in registers, serve all of them.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeArgs a, int parts) {
  const int j = threadIdx.x & 15;
  const long long hw = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 4;
  const long long t = hw / parts;
  if (t >= a.n) return;  // whole half-warps; the shuffles pair lanes of one half-warp
  const int part = (int)(hw % parts);
  const Lane l = lane_of<INTERLEAVED>(j, a.rope.rotary_dim);
  Angles cs;
  if (l.pair >= 0) {
    float4 c, si;
    cos_sin4(c, si, a.rope, l.pair, a.positions, a.n, t);
    cs = angles_of(c, si);
  }
  turn_rows<T, INTERLEAVED>(reinterpret_cast<const T*>(a.q.x) + t * a.q.stride, reinterpret_cast<T*>(a.q.out) + t * a.q.out_stride,
                            part, parts, a.q.heads, a.q.weight, a.eps, cs, l);
  // the keys go on where the queries end: row heads + h of the token
  const int k0 = part >= a.q.heads ? part - a.q.heads : (parts - (a.q.heads - part) % parts) % parts;
  turn_rows<T, INTERLEAVED>(reinterpret_cast<const T*>(a.k.x) + t * a.k.stride, reinterpret_cast<T*>(a.k.out) + t * a.k.out_stride,
                            k0, parts, a.k.heads, a.k.weight, a.eps, cs, l);
}

template <typename T>
cudaError_t launch(const NormRopeArgs& a, int parts, unsigned ctas, cudaStream_t stream) {
  if (a.rope.interleaved)
    norm_rope_kernel<T, true><<<ctas, kThreads, 0, stream>>>(a, parts);
  else
    norm_rope_kernel<T, false><<<ctas, kThreads, 0, stream>>>(a, parts);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int num_sms, cudaStream_t stream) {
  const int rows = a.q.heads + a.k.heads;
  // the fewest parts per token (the most rows behind one set of cosines) that still give every SM
  // eight CTAs' half-warps
  const long long want = (long long)num_sms * 8 * (kThreads / 16);
  int parts = (int)((want + a.n - 1) / a.n);
  const int most = (rows + kBatch - 1) / kBatch;
  parts = parts > rows ? rows : (parts < 1 ? 1 : parts);
  if (parts > most && a.n * (long long)most >= num_sms * 16) parts = most;
  const long long ctas = (a.n * (long long)parts * 16 + kThreads - 1) / kThreads;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
  return a.bf16 ? launch<__nv_bfloat16>(a, parts, (unsigned)ctas, stream)
                : launch<__half>(a, parts, (unsigned)ctas, stream);
}

}  // namespace rq
