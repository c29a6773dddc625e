// C-ABI entry points of the paged key/value cache: argument checks and
// parameter blocks for the kernels in paged.cu.
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/dllm.h"
#include "kernels.cuh"

using namespace dllm;

namespace {

constexpr int kMaxSeqs = 1024;
constexpr long long kMaxRows = 1ll << 24;
constexpr long long kMaxPositions = 1ll << 24;

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool aligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

dllm_status check_shape(const dllm_kv_pages* kv, PagedPool* o) {
  if (!kv) return DLLM_ERR_INVALID;
  if (kv->n_pages < 1 || kv->page_size < 1 || kv->n_kv_heads < 1 || kv->head_dim < 1)
    return DLLM_ERR_INVALID;
  if (kv->type != DLLM_KV_BF16 && kv->type != DLLM_KV_F16) return DLLM_ERR_INVALID;
  if (kv->head_dim != 32 && kv->head_dim != 64 && kv->head_dim != 128) return DLLM_ERR_UNSUPPORTED;
  if (kv->page_size & (kv->page_size - 1) || kv->page_size < 8 || kv->page_size > 65536)
    return DLLM_ERR_UNSUPPORTED;
  if (kv->n_kv_heads > 1024) return DLLM_ERR_UNSUPPORTED;
  int shift = 0;
  while ((1 << shift) < kv->page_size) ++shift;
  *o = PagedPool{kv->k, kv->v, kv->page_stride, kv->head_stride, kv->slot_stride, kv->n_pages,
                 shift, kv->n_kv_heads, kv->head_dim, kv->type == DLLM_KV_F16};
  return DLLM_OK;
}

// A stride counts only where its axis has more than one element; the tensor
// maps take strides below 2^40 bytes.
bool stride_ok(long long stride, long long extent, long long least) {
  return extent == 1 || (stride >= least && stride % 8 == 0 && stride < (1ll << 39));
}

dllm_status check_pool(const dllm_kv_pages* kv, PagedPool* o) {
  const dllm_status e = check_shape(kv, o);
  if (e != DLLM_OK) return e;
  if (!kv->k || !kv->v || !aligned16(kv->k) || !aligned16(kv->v)) return DLLM_ERR_INVALID;
  if (!stride_ok(kv->page_stride, kv->n_pages, kv->head_dim) ||
      !stride_ok(kv->head_stride, kv->n_kv_heads, kv->head_dim) ||
      !stride_ok(kv->slot_stride, kv->page_size, kv->head_dim))
    return DLLM_ERR_INVALID;
  return DLLM_OK;
}

dllm_status check_batch(const dllm_paged_batch* b, const PagedPool& kv, PagedBatch* o) {
  if (!b || !b->row_start || !b->page_table || !aligned4(b->row_start) || !aligned4(b->page_table))
    return DLLM_ERR_INVALID;
  if (b->n_seqs < 1 || b->n_rows < 1 || b->max_pages < 1 || b->table_stride < b->max_pages)
    return DLLM_ERR_INVALID;
  if (b->n_seqs > kMaxSeqs || b->n_rows >= kMaxRows ||
      ((long long)b->max_pages << kv.page_shift) > kMaxPositions)
    return DLLM_ERR_UNSUPPORTED;
  *o = PagedBatch{b->n_seqs, b->n_rows, b->max_pages, b->table_stride, b->row_start,
                  b->page_table};
  return DLLM_OK;
}

bool rows_ok(const dllm_rows* r, long long n_rows, int heads, int D, PagedRows* o) {
  if (!r || !r->data || !aligned16(r->data)) return false;
  if (!stride_ok(r->row_stride, n_rows, D) || !stride_ok(r->head_stride, heads, D)) return false;
  *o = PagedRows{r->data, r->row_stride, r->head_stride};
  return true;
}

dllm_status check_heads(int n_q_heads, const PagedPool& kv) {
  if (n_q_heads < 1 || n_q_heads % kv.Hkv) return DLLM_ERR_INVALID;
  if (n_q_heads / kv.Hkv > 128) return DLLM_ERR_UNSUPPORTED;
  return DLLM_OK;
}

size_t workspace_bytes() { return 256; }

dllm_status run_attn(const dllm_kv_pages* kv, const dllm_paged_batch* batch,
                     const dllm_prefix_groups* groups, int32_t n_q_heads, const int32_t* segs,
                     const int32_t* row_limit, float scale, const dllm_rows* q,
                     const dllm_rows* out, float* lse, void* ws, size_t ws_bytes,
                     dllm_stream stream) {
  PagedAttnParams p{};
  dllm_status e = check_pool(kv, &p.kv);
  if (e == DLLM_OK) e = check_batch(batch, p.kv, &p.bt);
  if (e == DLLM_OK) e = check_heads(n_q_heads, p.kv);
  if (e != DLLM_OK) return e;
  if (!segs || !aligned4(segs) || !aligned4(row_limit) || !aligned4(lse)) return DLLM_ERR_INVALID;
  if (!(scale >= 0.f && scale <= FLT_MAX)) return DLLM_ERR_INVALID;  // NaN, inf, negative
  if (!rows_ok(q, p.bt.n_rows, n_q_heads, p.kv.D, &p.q) ||
      !rows_ok(out, p.bt.n_rows, n_q_heads, p.kv.D, &p.out) || q->data == out->data)
    return DLLM_ERR_INVALID;
  if (groups) {
    if (groups->n_groups < 1 || groups->max_pages < 1 || groups->table_stride < groups->max_pages)
      return DLLM_ERR_INVALID;
    if (!groups->seq_start || !groups->page_table || !groups->len ||
        !aligned4(groups->seq_start) || !aligned4(groups->page_table) || !aligned4(groups->len))
      return DLLM_ERR_INVALID;
    if (groups->n_groups > kMaxSeqs ||
        ((long long)groups->max_pages << p.kv.page_shift) > kMaxPositions)
      return DLLM_ERR_UNSUPPORTED;
    p.n_groups = groups->n_groups;
    p.pmax_pages = groups->max_pages;
    p.ptable_stride = groups->table_stride;
    p.gseq = groups->seq_start;
    p.ptable = groups->page_table;
    p.plen = groups->len;
  }
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256) return DLLM_ERR_INVALID;
  if (ws_bytes < workspace_bytes()) return DLLM_ERR_WORKSPACE;
  p.Hq = n_q_heads;
  p.segs = segs;
  p.row_limit = row_limit;
  p.scale_log2 = 1.4426950408889634f * (scale > 0.f ? scale : 1.f / sqrtf((float)p.kv.D));
  p.lse = lse;
  p.status = static_cast<int*>(ws);
  return launch_paged_attn(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? DLLM_OK
             : DLLM_ERR_CUDA;
}

}  // namespace

extern "C" {

dllm_status dllm_paged_append(const dllm_kv_pages* kv, const dllm_paged_batch* batch,
                              int32_t n_q_heads, const dllm_rows* q, const dllm_rows* k,
                              const dllm_rows* v, const dllm_rows* q_out, const int32_t* pos,
                              const int32_t* rope_shift, float rope_theta, int32_t* status,
                              dllm_stream stream) {
  PagedAppendParams p{};
  dllm_status e = check_pool(kv, &p.kv);
  if (e == DLLM_OK) e = check_batch(batch, p.kv, &p.bt);
  if (e == DLLM_OK && q) e = check_heads(n_q_heads, p.kv);
  if (e != DLLM_OK) return e;
  if (!pos || !aligned4(pos) || !aligned4(rope_shift) || !aligned4(status)) return DLLM_ERR_INVALID;
  if (!(rope_theta >= 0.f && rope_theta <= FLT_MAX)) return DLLM_ERR_INVALID;  // NaN, inf
  const int D = p.kv.D;
  if (!rows_ok(k, p.bt.n_rows, p.kv.Hkv, D, &p.k) || !rows_ok(v, p.bt.n_rows, p.kv.Hkv, D, &p.v))
    return DLLM_ERR_INVALID;
  if (q) {
    if (!rows_ok(q, p.bt.n_rows, n_q_heads, D, &p.q) ||
        !rows_ok(q_out, p.bt.n_rows, n_q_heads, D, &p.q_out))
      return DLLM_ERR_INVALID;
    if (q->data == q_out->data &&
        (q->row_stride != q_out->row_stride || q->head_stride != q_out->head_stride))
      return DLLM_ERR_INVALID;
    p.Hq = n_q_heads;
  }
  p.pos = pos;
  p.shift = rope_shift;
  p.status = status;
  p.rope = rope_theta > 0.f;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  for (int i = 0; p.rope && i < D / 2; ++i)
    p.turns[i] = pow((double)rope_theta, -2.0 * i / D) / kTwoPi;
  return launch_paged_append(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? DLLM_OK
             : DLLM_ERR_CUDA;
}

dllm_status dllm_paged_workspace_size(const dllm_kv_pages* kv, int32_t n_q_heads,
                                      int32_t max_rows, int32_t max_groups, size_t* bytes) {
  PagedPool pool;
  dllm_status e = check_shape(kv, &pool);
  if (e == DLLM_OK) e = check_heads(n_q_heads, pool);
  if (e != DLLM_OK) return e;
  if (!bytes || max_rows < 1 || max_groups < 0) return DLLM_ERR_INVALID;
  if (max_rows >= kMaxRows || max_groups > kMaxSeqs) return DLLM_ERR_UNSUPPORTED;
  *bytes = workspace_bytes();
  return DLLM_OK;
}

dllm_status dllm_paged_workspace_init(void* ws, size_t ws_bytes, dllm_stream stream) {
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256) return DLLM_ERR_INVALID;
  if (ws_bytes < 256) return DLLM_ERR_WORKSPACE;
  return cudaMemsetAsync(ws, 0, 256, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? DLLM_OK
             : DLLM_ERR_CUDA;
}

dllm_status dllm_paged_attn(const dllm_kv_pages* kv, const dllm_paged_batch* batch,
                            int32_t n_q_heads, const int32_t* segs, const int32_t* row_limit,
                            float scale, const dllm_rows* q, const dllm_rows* out, float* lse,
                            void* ws, size_t ws_bytes, dllm_stream stream) {
  return run_attn(kv, batch, nullptr, n_q_heads, segs, row_limit, scale, q, out, lse, ws,
                  ws_bytes, stream);
}

dllm_status dllm_shared_prefix_attn(const dllm_kv_pages* kv, const dllm_paged_batch* batch,
                                    const dllm_prefix_groups* groups, int32_t n_q_heads,
                                    const int32_t* segs, const int32_t* row_limit, float scale,
                                    const dllm_rows* q, const dllm_rows* out, float* lse,
                                    void* ws, size_t ws_bytes, dllm_stream stream) {
  if (!groups) return DLLM_ERR_INVALID;
  return run_attn(kv, batch, groups, n_q_heads, segs, row_limit, scale, q, out, lse, ws, ws_bytes,
                  stream);
}

}  // extern "C"
