// Causal attention of new tokens in the expanded form of latent attention: heads of 192 (128 of their own and 64 that
// all heads share) against values of 128, sequences packed one after the other.
#include <math_constants.h>

#include "../../include/rq.h"
#include "rq_rope.cuh"

namespace rq {
namespace {

constexpr int kThreads = 128;

// One row of one head a CTA: a thread a key for the scores, then a thread a dim for the sum.
template <typename T>
__global__ void __launch_bounds__(kThreads) prompt_rows_kernel(const PromptArgs a) {
  __shared__ float q[kPromptDim], w[kThreads], red[kThreads / 32];
  const int tid = threadIdx.x, j = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int q0 = __ldg(a.q_offsets + b), q1 = __ldg(a.q_offsets + b + 1);
  const int k0 = __ldg(a.k_offsets + b), k1 = __ldg(a.k_offsets + b + 1);
  if (q0 < 0 || q1 < q0 || q1 > a.nq || k0 < 0 || k1 < k0 || k1 > a.nk || q1 - q0 > a.max_new) {
    if (tid == 0 && a.status) atomicOr(a.status, RQ_STATUS_BAD_LEN);
    return;
  }
  if (j >= q1 - q0) return;
  const T* row = reinterpret_cast<const T*>(a.q.x) + (q0 + (long long)j) * a.q.stride + h * a.q.head_stride;
  for (int i = tid; i < kPromptDim; i += kThreads) q[i] = (float)row[i] * (a.sm_scale * 1.44269504088896340736f);
  const int end = (k1 - k0) - (q1 - q0) + j + 1;
  float m = -CUDART_INF_F, l = 0.f, acc = 0.f;
  for (int t0 = 0; t0 < end; t0 += kThreads) {
    const int p = t0 + tid;
    __syncthreads();
    float s = -CUDART_INF_F;
    if (p < end) {
      const T* k = reinterpret_cast<const T*>(a.k.x) + (k0 + (long long)p) * a.k.stride + h * a.k.head_stride;
      const T* pe = reinterpret_cast<const T*>(a.k_pe) + (k0 + (long long)p) * a.k_pe_stride;
      s = 0.f;
      for (int i = 0; i < 128; ++i) s = fmaf(q[i], (float)k[i], s);
      for (int i = 0; i < 64; ++i) s = fmaf(q[128 + i], (float)pe[i], s);
    }
    float top = s;
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 31) == 0) red[tid >> 5] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float m_new = fmaxf(m, top), from = m_new == -CUDART_INF_F ? 0.f : m_new;
    const float alpha = m == -CUDART_INF_F ? 0.f : exp2f(m - from);
    m = m_new;
    const float e = p < end ? exp2f(s - from) : 0.f;
    w[tid] = e;
    float sum = e;
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    l = l * alpha + (red[0] + red[1] + red[2] + red[3]);
    acc *= alpha;
    const T* v = reinterpret_cast<const T*>(a.v.x) + (k0 + (long long)t0) * a.v.stride + h * a.v.head_stride + tid;
    for (int k = 0; k < min(kThreads, end - t0); ++k) acc = fmaf(w[k], (float)v[k * a.v.stride], acc);
  }
  const float y = end <= 0 ? 0.f : acc / l;
  reinterpret_cast<T*>(a.out)[((q0 + (size_t)j) * a.q.heads + h) * 128 + tid] = (T)y;
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t stream) {
  const dim3 grid((unsigned)a.max_new, (unsigned)a.q.heads, (unsigned)a.B);
  if (a.bf16)
    prompt_rows_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a);
  else
    prompt_rows_kernel<__half><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace rq
