// Extend (prefill) attention over the 8-bit block-scaled cache.
#include <math_constants.h>

#include "../../include/rq.h"
#include "rq_block.cuh"
#include "rq_rope.cuh"

namespace rq {
namespace {

using namespace block;

constexpr int kWarps = 4;

// One CTA per (sequence, query row): its warps take every fourth block of 16 tokens, each with a
// running maximum and sum, and are joined at the end.  Scores: lane (half, token) sums 64 dims.
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) rows_kernel(const Geometry g, const AttnArgs a) {
  __shared__ float q[kHeadDim], part[kWarps][kHeadDim], ms[kWarps], ls[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long row = blockIdx.x;  // (b, j, head)
  const int head = (int)(row % g.num_q_heads), b = (int)(row / g.num_q_heads / a.T);
  const int j = (int)(row / g.num_q_heads % a.T), h = head / g.group;
  const int cap = a.max_pages * g.page_size;
  int len = a.seq_lens[b];
  if (len < 0 || len > cap || (len > 0 && len < a.T)) {
    if (tid == 0 && a.status) atomicOr(a.status, RQ_STATUS_BAD_LEN);
    len = len < 0 ? 0 : min(len, cap);
  }
  const T* src = reinterpret_cast<const T*>(a.q) + row * kHeadDim;
  q[tid] = (float)src[tid] * (g.sm_scale * 1.44269504088896340736f);
  __syncthreads();
  const int prefix = len - a.T;  // position of draft 0
  const uint64_t mask = a.tree_mask ? a.tree_mask[(size_t)b * a.T + j] : 0;
  const int end = a.tree_mask ? len : min(len, prefix + j + 1);
  const int r = lane & 15, half = lane >> 4;
  float m = -CUDART_INF_F, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int t0 = kBlockTokens * warp; t0 < end; t0 += kBlockTokens * kWarps) {
    int page = a.block_table[(size_t)b * a.max_pages + t0 / g.page_size];
    if (page < 0 || page >= g.num_pages) {
      if (lane == 0 && a.status) atomicOr(a.status, RQ_STATUS_BAD_PAGE);
      page = 0;
    }
    const uint8_t* blk = a.pages + ((size_t)page * g.num_kv_heads + h) * g.page_bytes +
                         (size_t)(t0 % g.page_size / kBlockTokens) * kBlockBytes;
    const float ek = pow2(exp_of_byte(blk[kExps])), ev = pow2(exp_of_byte(blk[kExps + 1]));
    float s = 0.f;
    for (int u = 0; u < 4; ++u) {
      const uint4 c = reinterpret_cast<const uint4*>(blk)[(2 * (r >> 3) + half) * 32 + (r & 7) * 4 + u];
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
      for (int k = 0; k < 4; ++k) {
        const float2 x = rope::unpack2<__half>(widen2(w[k])), y = rope::unpack2<__half>(widen2_hi(w[k]));
        const float* qq = q + 64 * half + 16 * u + 4 * k;
        s += x.x * qq[0] + x.y * qq[1] + y.x * qq[2] + y.y * qq[3];
      }
    }
    s += __shfl_xor_sync(0xffffffffu, s, 16);
    const int p = t0 + r;
    bool seen = p < end;
    if (a.tree_mask && p >= prefix) seen = seen && (mask >> (p - prefix) & 1);
    s = seen ? s * ek : -CUDART_INF_F;
    float top = s;
    for (int x = 8; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float m_new = fmaxf(m, top), base = m_new == -CUDART_INF_F ? 0.f : m_new;
    const float alpha = exp2f(m - base), w = exp2f(s - base);
    m = m_new;
    float sum = w;
    for (int x = 8; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    l = l * alpha + sum;
    for (int d = 0; d < 4; ++d) o[d] *= alpha;
    for (int t = 0; t < 4; ++t) {
      const uint4 c = reinterpret_cast<const uint4*>(blk + kValues)[4 * lane + t];
      const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
      const int rows[4] = {2 * t, 2 * t + 1, 2 * t + 8, 2 * t + 9};
      for (int k = 0; k < 4; ++k) {
        const float wr = __shfl_sync(0xffffffffu, w, rows[k]) * ev;
        if (wr == 0.f) continue;  // a masked token's bytes may be anything
        for (int d = 0; d < 4; ++d) o[d] += wr * rope::unpack2<__half>(widen2(cw[d] >> (8 * k) & 0xFF)).x;
      }
    }
  }
  if (lane == 0) ms[warp] = m, ls[warp] = l;
  for (int d = 0; d < 4; ++d) part[warp][4 * lane + d] = o[d];
  __syncthreads();
  float top = -CUDART_INF_F, sum = 0.f, out = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ms[w]);
  for (int w = 0; w < kWarps; ++w) {
    const float f = ms[w] == -CUDART_INF_F ? 0.f : exp2f(ms[w] - top);
    sum += ls[w] * f;
    out += part[w][tid] * f;
  }
  out = sum > 0.f || sum != sum ? out / sum : 0.f;  // a row that sees nothing gives zeros
  reinterpret_cast<T*>(a.out)[row * kHeadDim + tid] = (T)out;
}

}  // namespace

cudaError_t launch_block_extend(const Geometry& g, const AttnArgs& a, cudaStream_t stream, cudaEvent_t ev_start,
                                   cudaEvent_t ev_end) {
  const long long rows = (long long)a.B * a.T * g.num_q_heads;
  if (rows > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (ev_start) cudaEventRecord(ev_start, stream);
  if (g.bf16)
    rows_kernel<__nv_bfloat16><<<(unsigned)rows, 32 * kWarps, 0, stream>>>(g, a);
  else
    rows_kernel<__half><<<(unsigned)rows, 32 * kWarps, 0, stream>>>(g, a);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && ev_end) cudaEventRecord(ev_end, stream);
  return e;
}

}  // namespace rq
