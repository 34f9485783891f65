// Attention in the absorbed form over the cache of latents: decode, chain and tree verify.
#include <math_constants.h>

#include "../../include/rq.h"
#include "rq_block.cuh"
#include "rq_latent.cuh"
#include "rq_rope.cuh"

namespace rq {
namespace {

using namespace latent;

constexpr int kThreads = 128;

// One query row a CTA: a thread a token for the scores, then a thread four dims for the sum.
template <typename T>
__global__ void __launch_bounds__(kThreads) latent_rows_kernel(const LatentPool pool, const LatentAttnArgs a) {
  __shared__ float q[kLatentDim + kPositionDim], w[kThreads], red[kThreads / 32];
  __shared__ const uint8_t* at[kThreads];
  __shared__ int off[kThreads];
  const int tid = threadIdx.x, P = pool.page_size;
  const long long token = blockIdx.x / a.heads;
  const int h = blockIdx.x % a.heads, b = (int)(token / a.T), j = (int)(token % a.T);
  const int cap = a.max_pages * P;
  int len = __ldg(a.seq_lens + b);
  if (len < 0 || len > cap || (len > 0 && len < a.T)) {
    if (tid == 0 && a.status) atomicOr(a.status, RQ_STATUS_BAD_LEN);
    len = len < 0 ? 0 : min(len, cap);
  }
  const float up = a.sm_scale * 1.44269504088896340736f;
  const T* qc = reinterpret_cast<const T*>(a.q_c.x) + token * a.q_c.stride + h * a.q_c.head_stride;
  const T* qp = reinterpret_cast<const T*>(a.q_pe.x) + token * a.q_pe.stride + h * a.q_pe.head_stride;
  for (int i = tid; i < kLatentDim; i += kThreads) q[i] = (float)qc[i];
  for (int i = tid; i < kPositionDim; i += kThreads) q[kLatentDim + i] = (float)qp[i];
  const uint64_t mask = a.tree_mask ? __ldg(a.tree_mask + token) : 0ull;
  float m = -CUDART_INF_F, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int t0 = 0; t0 < len; t0 += kThreads) {
    const int p = t0 + tid, draft = p - (len - a.T);
    const bool see = p < len && (draft < 0 || (a.tree_mask ? (mask >> draft & 1) != 0 : draft <= j));
    float s = -CUDART_INF_F, scale = 0.f;
    __syncthreads();
    if (see) {
      int page = __ldg(a.block_table + (size_t)b * a.max_pages + p / P);
      if (page < 0 || page >= pool.num_pages) {
        if (a.status) atomicOr(a.status, RQ_STATUS_BAD_PAGE);
        page = 0;
      }
      const uint8_t* base = pool.pages + page_at(page, P);
      const int r = p % P;
      at[tid] = base;
      off[tid] = r;
      scale = scale_of_byte(base[640 * P + r]);
      float sum = 0.f;
      for (int c = 0; c < 32; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(base + (c >> 3) * 128 * P + chunk_at(r, c & 7));
        const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
        for (int k = 0; k < 4; ++k) {
          const float2 lo = rope::unpack2<__half>(block::widen2(w4[k])), hi = rope::unpack2<__half>(block::widen2_hi(w4[k]));
          const float* qq = q + 16 * c + 4 * k;
          sum += lo.x * qq[0] + lo.y * qq[1] + hi.x * qq[2] + hi.y * qq[3];
        }
      }
      for (int c = 0; c < 8; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(base + 512 * P + chunk_at(r, c));
        const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
        for (int k = 0; k < 4; ++k) {
          const float2 f = rope::unpack2<T>(w4[k]);
          sum += f.x * q[kLatentDim + 8 * c + 2 * k] + f.y * q[kLatentDim + 8 * c + 2 * k + 1];
        }
      }
      s = sum * scale * up;
    }
    float top = s;
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 31) == 0) red[tid >> 5] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float m_new = fmaxf(m, top), from = m_new == -CUDART_INF_F ? 0.f : m_new;
    const float alpha = m == -CUDART_INF_F ? 0.f : exp2f(m - from);
    m = m_new;
    const float e = see ? exp2f(s - from) : 0.f;
    w[tid] = e * scale;
    float sum = e;
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    l = l * alpha + (red[0] + red[1] + red[2] + red[3]);
    for (int i = 0; i < 4; ++i) acc[i] *= alpha;
    for (int k = 0; k < min(kThreads, len - t0); ++k) {
      if (w[k] == 0.f) continue;
      const int d = 4 * tid;
      const uint32_t v = *reinterpret_cast<const uint32_t*>(at[k] + (d >> 7) * 128 * P + chunk_at(off[k], (d & 127) >> 4) + (d & 15));
      const float2 lo = rope::unpack2<__half>(block::widen2(v)), hi = rope::unpack2<__half>(block::widen2_hi(v));
      acc[0] = fmaf(w[k], lo.x, acc[0]), acc[1] = fmaf(w[k], lo.y, acc[1]);
      acc[2] = fmaf(w[k], hi.x, acc[2]), acc[3] = fmaf(w[k], hi.y, acc[3]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* out = reinterpret_cast<T*>(a.out) + ((size_t)token * a.heads + h) * kLatentDim + 4 * tid;
  *reinterpret_cast<uint2*>(out) =
      make_uint2(rope::pack2<T>(acc[0] * inv, acc[1] * inv), rope::pack2<T>(acc[2] * inv, acc[3] * inv));
}

}  // namespace

size_t latent_attention_workspace(int num_sms) { return (size_t)num_sms; }
cudaError_t latent_attention_prepare() { return cudaSuccess; }

cudaError_t launch_latent_attention(const LatentPool& pool, const LatentAttnArgs& a, int num_sms, cudaStream_t stream) {
  (void)num_sms;
  const long long rows = (long long)a.B * a.T * a.heads;
  if (rows > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (pool.bf16)
    latent_rows_kernel<__nv_bfloat16><<<(unsigned)rows, kThreads, 0, stream>>>(pool, a);
  else
    latent_rows_kernel<__half><<<(unsigned)rows, kThreads, 0, stream>>>(pool, a);
  return cudaGetLastError();
}

}  // namespace rq
