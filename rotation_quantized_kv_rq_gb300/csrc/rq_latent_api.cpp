// Host side of latent attention in the C ABI (include/rq.h): argument validation and the context of a cache of latents.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <new>

#include "../../include/rq.h"
#include "rq_host.h"
#include "rq_internal.h"

using rq::DeviceScope;
using rq::misaligned16;
using rq::to_status;

struct rq_latent {
  rq_latent_config cfg;
  int device, num_sms;
  float* d_ws;
};

namespace {

constexpr long long kMostStride = 1ll << 40;  // elements

bool bad_stride(long long s, long long least) { return s < least || s % 8 != 0 || s > kMostStride; }

// Rows of n tokens whose heads have `dims` elements.
bool bad_rows(const rq_heads* r, int dims, long long n) {
  if (!r->x || misaligned16(r->x) || r->heads <= 0 || r->heads > 65535) return true;
  if (r->heads > 1 && bad_stride(r->head_stride, dims)) return true;
  return n > 1 && bad_stride(r->stride, dims);
}
rq::HeadsDev heads_dev(const rq_heads* r) {
  return r ? rq::HeadsDev{r->x, r->stride, r->heads > 1 ? r->head_stride : 0, r->heads} : rq::HeadsDev{};
}

// The bytes of n rows, for overlaps.  Rows interleaved in one buffer (one stride, apart within it) do not overlap.
struct Span {
  uintptr_t at, stride, row, end;
};
Span span(const void* x, long long stride, long long row, long long n) {
  Span s;
  s.at = (uintptr_t)x;
  s.row = (uintptr_t)row * 2;
  s.stride = n > 1 ? (uintptr_t)stride * 2 : s.row;
  s.end = s.at + (uintptr_t)(n - 1) * s.stride + s.row;
  return s;
}
Span span(const rq_heads* r, int dims, long long n) {
  const long long heads = (r->heads > 1 ? r->head_stride : 0) * (r->heads - 1);
  if (n > 1 && r->stride < heads + dims) {  // head after head: one span over all
    Span s = span(r->x, 0, heads + (n - 1) * r->stride + dims, 1);
    return s;
  }
  return span(r->x, r->stride, heads + dims, n);
}
bool overlap(const Span& a, const Span& b) {
  if (a.end <= b.at || b.end <= a.at) return false;
  if (a.stride != b.stride) return true;
  const uintptr_t d = a.at <= b.at ? (b.at - a.at) % b.stride : (a.stride - (a.at - b.at) % a.stride) % a.stride;
  return d < a.row || d + b.row > a.stride;
}

// Whether two of the n tokens' rows of `dims` elements share some (strides at least dims, bad_rows says).
bool rows_meet(const rq_heads* r, int dims, long long n) {
  if (r->heads == 1 || n == 1) return false;
  const long long s = r->stride, h = r->head_stride;
  if ((s - dims) / h >= r->heads - 1 || (h - dims) / s >= n - 1) return false;  // all heads before the next token, or all tokens before the next head
  for (long long d = 1; d < r->heads; ++d) {  // d heads on, k tokens back
    const long long at = d * h, k = at / s;
    if ((k >= 1 && k < n && at - k * s < dims) || (k + 1 < n && (k + 1) * s - at < dims)) return true;
  }
  return false;
}

rq::LatentPool pool_of(const rq_latent* ctx, const void* pages) {
  return rq::LatentPool{(const uint8_t*)pages, ctx->cfg.page_size, ctx->cfg.num_pages, ctx->cfg.io_type == RQ_BF16};
}

}  // namespace

extern "C" {

int rq_latent_create(rq_latent** out, const rq_latent_config* cfg) {
  if (!out) return RQ_ERR_INVALID;
  *out = nullptr;
  if (!cfg) return RQ_ERR_INVALID;
  if (cfg->num_heads <= 0 || cfg->latent_dim <= 0 || cfg->position_dim <= 0 || cfg->page_size <= 0 || cfg->num_pages <= 0 ||
      cfg->max_batch <= 0 || cfg->max_query_tokens <= 0 || cfg->max_pages_per_seq <= 0 ||
      (cfg->io_type != RQ_F16 && cfg->io_type != RQ_BF16) || !(cfg->sm_scale >= 0.f) || std::isinf(cfg->sm_scale))
    return RQ_ERR_INVALID;
  if (cfg->latent_dim != rq::kLatentDim || cfg->position_dim != rq::kPositionDim || cfg->num_heads > 1024 ||
      cfg->page_size % 16 != 0 || cfg->page_size > 256 || cfg->max_batch > rq::kMaxBatch ||
      (long long)cfg->num_pages * cfg->page_size > INT32_MAX ||
      (long long)cfg->max_pages_per_seq * cfg->page_size > INT32_MAX - 4096 ||
      (long long)cfg->max_query_tokens * cfg->num_heads > INT32_MAX / 2)
    return RQ_ERR_UNSUPPORTED;
  int dev = cfg->device;
  if (dev < 0 && cudaGetDevice(&dev) != cudaSuccess) return RQ_ERR_CUDA;
  DeviceScope scope(dev);
  if (!scope.ok()) return RQ_ERR_CUDA;
  rq_latent* ctx = new (std::nothrow) rq_latent();
  if (!ctx) return RQ_ERR_CUDA;
  ctx->cfg = *cfg;
  if (cfg->sm_scale == 0.f) ctx->cfg.sm_scale = (float)(1.0 / std::sqrt((double)rq::kPromptDim));
  ctx->device = dev;
  cudaError_t e = cudaDeviceGetAttribute(&ctx->num_sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaMalloc(&ctx->d_ws, rq::latent_attention_workspace(ctx->num_sms, (long long)cfg->max_query_tokens * cfg->num_heads, cfg->max_batch) * sizeof(float));
  if (e == cudaSuccess) e = rq::latent_attention_prepare();
  if (e != cudaSuccess) {
    cudaFree(ctx->d_ws);
    delete ctx;
    return RQ_ERR_CUDA;
  }
  *out = ctx;
  return RQ_OK;
}

void rq_latent_free(rq_latent* ctx) {
  if (!ctx) return;
  {
    DeviceScope scope(ctx->device);
    cudaFree(ctx->d_ws);
  }
  delete ctx;
}

size_t rq_latent_page_bytes(const rq_latent* ctx) {
  return ctx ? (size_t)ctx->cfg.page_size * rq::kLatentTokenBytes : 0;
}

int rq_latent_append(rq_latent* ctx, const rq_rope* rope, const void* c, long long c_stride, const float* weight, float eps,
                     const void* k_pe, long long k_pe_stride, const rq_heads* q_pe, const rq_heads* q_pe_out,
                     const int32_t* positions, const int32_t* slot_mapping, int n, void* pages, int32_t* d_status,
                     void* stream) {
  constexpr int kPe = rq::kPositionDim;
  if (!ctx || n < 0 || !(eps >= 0.f) || std::isinf(eps) || !q_pe != !q_pe_out) return RQ_ERR_INVALID;
  if (n == 0) return RQ_OK;
  if (!c || !k_pe || !slot_mapping || !pages || misaligned16(c) || misaligned16(k_pe) || misaligned16(pages) ||
      misaligned16(weight))
    return RQ_ERR_INVALID;
  if (n > 1 && (bad_stride(c_stride, rq::kLatentDim) || bad_stride(k_pe_stride, kPe))) return RQ_ERR_INVALID;
  if (rope && (rope->table.rotary_dim > kPe || rope->device != ctx->device || (rope->table.rotary_dim > 0 && !positions)))
    return RQ_ERR_INVALID;
  if (q_pe) {
    if (bad_rows(q_pe, kPe, n) || bad_rows(q_pe_out, kPe, n) || q_pe->heads != q_pe_out->heads || rows_meet(q_pe_out, kPe, n))
      return RQ_ERR_INVALID;
    const Span o = span(q_pe_out, kPe, n);
    const bool in_place = q_pe->x == q_pe_out->x && (n == 1 || q_pe->stride == q_pe_out->stride) &&
                          (q_pe->heads == 1 || q_pe->head_stride == q_pe_out->head_stride);
    if ((overlap(o, span(q_pe, kPe, n)) && !in_place) || overlap(o, span(c, c_stride, rq::kLatentDim, n)) ||
        overlap(o, span(k_pe, k_pe_stride, kPe, n)))
      return RQ_ERR_INVALID;
  }
  DeviceScope scope(ctx->device);
  if (!scope.ok()) return RQ_ERR_CUDA;
  rq::LatentAppendArgs a{};
  a.c = c;
  a.k_pe = k_pe;
  a.c_stride = c_stride;
  a.k_pe_stride = k_pe_stride;
  a.weight = weight;
  a.eps = eps;
  a.q = heads_dev(q_pe);
  a.q_out = heads_dev(q_pe_out);
  if (rope) a.rope = rope->table;
  a.positions = positions;
  a.slots = slot_mapping;
  a.n = n;
  a.status = d_status;
  return to_status(rq::launch_latent_append(pool_of(ctx, pages), a, ctx->num_sms, (cudaStream_t)stream));
}

int rq_latent_attention(rq_latent* ctx, const rq_heads* q_c, const rq_heads* q_pe, int T, const uint64_t* tree_mask,
                        const void* pages, const int32_t* block_table, int max_pages, const int32_t* seq_lens, int B, void* out,
                        int32_t* d_status, void* stream) {
  if (!ctx || B < 0 || T < 1 || max_pages < 1 || (tree_mask && T > 64)) return RQ_ERR_INVALID;
  if (B == 0) return RQ_OK;
  if (!q_c || !q_pe || !pages || !block_table || !seq_lens || !out || misaligned16(pages) || misaligned16(out))
    return RQ_ERR_INVALID;
  const long long n = (long long)B * T;
  if (bad_rows(q_c, rq::kLatentDim, n) || bad_rows(q_pe, rq::kPositionDim, n) || q_c->heads != ctx->cfg.num_heads ||
      q_pe->heads != ctx->cfg.num_heads)
    return RQ_ERR_INVALID;
  {  // a unit's rows are written when its queries have been read, by the CTAs that read them or behind all
    const long long H = ctx->cfg.num_heads;
    const Span o = span(out, H * rq::kLatentDim, H * rq::kLatentDim, n);
    const bool in_place = q_c->x == out && (H == 1 || q_c->head_stride == rq::kLatentDim) && (n == 1 || q_c->stride == H * rq::kLatentDim);
    if ((overlap(o, span(q_c, rq::kLatentDim, n)) && !in_place) || overlap(o, span(q_pe, rq::kPositionDim, n))) return RQ_ERR_INVALID;
  }
  if (B > ctx->cfg.max_batch || T > ctx->cfg.max_query_tokens || max_pages > ctx->cfg.max_pages_per_seq)
    return RQ_ERR_CAPACITY;
  // tiles of 256 tokens, and three more for each group, over all sequences and groups of 128 rows are counted in 31 bits
  const long long groups = (long long)B * (((long long)T * ctx->cfg.num_heads + 127) / 128);
  if (groups > INT32_MAX / (((long long)max_pages * ctx->cfg.page_size + 255) / 256 + 3)) return RQ_ERR_CAPACITY;
  DeviceScope scope(ctx->device);
  if (!scope.ok()) return RQ_ERR_CUDA;
  rq::LatentAttnArgs a{};
  a.q_c = heads_dev(q_c);
  a.q_pe = heads_dev(q_pe);
  a.T = T;
  a.tree_mask = tree_mask;
  a.block_table = block_table;
  a.max_pages = max_pages;
  a.seq_lens = seq_lens;
  a.B = B;
  a.heads = ctx->cfg.num_heads;
  a.out = out;
  a.sm_scale = ctx->cfg.sm_scale;
  a.status = d_status;
  a.ws = ctx->d_ws;
  return to_status(rq::launch_latent_attention(pool_of(ctx, pages), a, ctx->num_sms, (cudaStream_t)stream));
}

int rq_latent_read(rq_latent* ctx, const void* pages, const int32_t* block_table, int max_pages, const int32_t* starts,
                   const int32_t* offsets, int B, int n, void* c, void* k_pe, int32_t* d_status, void* stream) {
  if (!ctx || B < 0 || n < 0 || max_pages < 1) return RQ_ERR_INVALID;
  if (B == 0 || n == 0) return RQ_OK;
  if (!pages || !block_table || !offsets || !c || !k_pe || misaligned16(pages) || misaligned16(c) || misaligned16(k_pe))
    return RQ_ERR_INVALID;
  if (overlap(span(c, rq::kLatentDim, rq::kLatentDim, n), span(k_pe, rq::kPositionDim, rq::kPositionDim, n))) return RQ_ERR_INVALID;
  DeviceScope scope(ctx->device);
  if (!scope.ok()) return RQ_ERR_CUDA;
  rq::LatentReadArgs a{};
  a.block_table = block_table;
  a.max_pages = max_pages;
  a.starts = starts;
  a.offsets = offsets;
  a.B = B;
  a.n = n;
  a.c = c;
  a.k_pe = k_pe;
  a.status = d_status;
  return to_status(rq::launch_latent_read(pool_of(ctx, pages), a, (cudaStream_t)stream));
}

size_t rq_prompt_workspace(int device) {
  int dev = device, sms = 0;
  if (dev < 0 && cudaGetDevice(&dev) != cudaSuccess) return 0;
  return cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess ? rq::prompt_workspace(sms) : 0;
}

int rq_prompt_attention(const rq_prompt* p, int32_t* d_status, void* stream) {
  if (!p || p->B < 0 || p->B > 65535 || p->nq < 0 || p->nk < 0 || p->max_new < 0 || !(p->sm_scale >= 0.f) ||
      std::isinf(p->sm_scale) || (p->io_type != RQ_F16 && p->io_type != RQ_BF16))
    return RQ_ERR_INVALID;
  if (p->B == 0 || p->nq == 0 || p->max_new == 0) return RQ_OK;
  const int H = p->q.heads;
  if (bad_rows(&p->q, rq::kPromptDim, p->nq) || !p->out || misaligned16(p->out) || !p->q_offsets || !p->k_offsets ||
      !p->workspace || misaligned16(p->workspace))
    return RQ_ERR_INVALID;
  if (p->nk > 0 && (bad_rows(&p->k, 128, p->nk) || bad_rows(&p->v, 128, p->nk) || p->k.heads != H || p->v.heads != H ||
                    !p->k_pe || misaligned16(p->k_pe) || (p->nk > 1 && bad_stride(p->k_pe_stride, rq::kPositionDim))))
    return RQ_ERR_INVALID;
  const Span o = span(p->out, (long long)H * 128, (long long)H * 128, p->nq);
  if (overlap(o, span(&p->q, rq::kPromptDim, p->nq)) ||
      (p->nk > 0 && (overlap(o, span(&p->k, 128, p->nk)) || overlap(o, span(&p->v, 128, p->nk)) ||
                     overlap(o, span(p->k_pe, p->k_pe_stride, rq::kPositionDim, p->nk)))))
    return RQ_ERR_INVALID;
  // units (512 rows of a sequence and head) are counted in 30 bits
  const int max_new = p->max_new < p->nq ? p->max_new : p->nq;
  if (((long long)max_new + 511) / 512 * p->B * H > (1 << 30) - 1) return RQ_ERR_CAPACITY;
  rq::PromptArgs a{};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&a.num_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return RQ_ERR_CUDA;
  if (p->workspace_bytes < rq::prompt_workspace(a.num_sms)) return RQ_ERR_CAPACITY;
  a.ws = (float*)p->workspace;
  a.q = heads_dev(&p->q);
  if (p->nk > 0) {
    a.k = heads_dev(&p->k);
    a.v = heads_dev(&p->v);
    a.k_pe = p->k_pe;
    a.k_pe_stride = p->k_pe_stride;
  }
  a.out = p->out;
  a.q_offsets = p->q_offsets;
  a.k_offsets = p->k_offsets;
  a.B = p->B;
  a.nq = p->nq;
  a.nk = p->nk;
  a.max_new = max_new;
  a.sm_scale = p->sm_scale > 0.f ? p->sm_scale : (float)(1.0 / std::sqrt((double)rq::kPromptDim));
  a.bf16 = p->io_type == RQ_BF16;
  a.status = d_status;
  return to_status(rq::launch_prompt_attention(a, (cudaStream_t)stream));
}

}  // extern "C"
