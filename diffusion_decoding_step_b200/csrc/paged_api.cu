// C-ABI entry points of the paged key/value cache: argument checks and
// parameter blocks for the kernels in paged.cu.
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "../../include/dllm.h"
#include "kernels.cuh"
#include "ptx.cuh"

namespace dllm {
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();
}

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

// Query tiles by the average query rows of an item (a group, or a sequence
// without one), rounded down since a padded batch has a few rows too many: up to
// 32 rows the 32-row tiles, whose softmax is spread over all warps, else the
// 128-row ones.  16 sequences of 1024 keys, 8 kv heads: 16 rows 24.2 us the first way
// and 29.3 the second, 32 rows 24.3 and 26.1; 40 rows, two tiles the first way, 31.9
// and 27.1.
int query_tiles(int n_rows, int items, int G) {
  const long long rows = (long long)std::max(n_rows / items, 1) * G;
  return rows <= 32 ? kPagedQuad : kPagedSplit;
}

// Workspace: status word (cleared once), a record per CTA, the parts of cut query
// tiles.
constexpr size_t kWsCut = 256, kWsParts = 4096;
static_assert(kWsCut + sizeof(int4) * kNumSMs <= kWsParts, "the records fit before the parts");

int slot_rows(long long n_rows, int G) {
  return (int)std::min((n_rows * G + 7) / 8 * 8, 128ll);
}
size_t workspace_bytes(const PagedPool& kv, int slot) {
  return kWsParts + (size_t)2 * kNumSMs * slot * (kv.D * sizeof(float) + sizeof(float2));
}

// One-time per-device setup that must not run inside a stream capture.
dllm_status prepare_device() {
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DLLM_ERR_CUDA;
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev]) return DLLM_OK;
  if (!tensor_map_encoder() || paged_attn_prepare() != cudaSuccess) return DLLM_ERR_CUDA;
  done[dev] = true;
  return DLLM_OK;
}

// Tensor map of 16-bit elements (any 16-bit type copies alike): extents d, byte
// strides of axes 1.. where the extent is above one.
bool make_map(CUtensorMap* m, const void* ptr, int rank, const cuuint64_t* d,
              const long long* stride, const cuuint32_t* box, int head_dim) {
  cuuint64_t st[3];
  for (int i = 0; i + 1 < rank; ++i) st[i] = d[i + 1] > 1 ? 2 * (cuuint64_t)stride[i] : 256;
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return tensor_map_encoder()(
             m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(ptr), d, st, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE,
             head_dim >= 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

dllm_status run_attn(const dllm_kv_pages* kv, const dllm_paged_batch* batch,
                     const dllm_prefix_groups* groups, int32_t n_q_heads, const int32_t* segs,
                     const int32_t* row_limit, float scale, const dllm_rows* q,
                     const dllm_rows* out, float* lse, void* ws, size_t ws_bytes,
                     dllm_stream stream, int stall = kStallNone,
                     unsigned long long wait_ns = kWaitLimitNs) {
  PagedAttnParams p{};
  p.stall = stall;
  p.wait_ns = wait_ns;
  dllm_status e = check_pool(kv, &p.kv);
  if (e == DLLM_OK) e = check_batch(batch, p.kv, &p.bt);
  if (e == DLLM_OK) e = check_heads(n_q_heads, p.kv);
  if (e != DLLM_OK) return e;
  if (!segs || !aligned4(segs) || !aligned4(row_limit) || !aligned4(lse)) return DLLM_ERR_INVALID;
  // NaN, inf, negative; in log2 units it has to be finite as well
  if (!(scale >= 0.f && scale <= 0x1p127f)) return DLLM_ERR_INVALID;
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
  p.Hq = n_q_heads;
  p.G = n_q_heads / p.kv.Hkv;
  p.slot_rows = slot_rows(p.bt.n_rows, p.G);
  if (ws_bytes < workspace_bytes(p.kv, p.slot_rows)) return DLLM_ERR_WORKSPACE;
  const int mode = query_tiles(p.bt.n_rows, groups ? p.n_groups : p.bt.n_seqs, p.G);
  if (mode == kPagedQuad) p.slot_rows = std::min(p.slot_rows, 32);
  const int D = p.kv.D;
  uint8_t* w = static_cast<uint8_t*>(ws);
  p.rows_per_tile = (mode == kPagedQuad ? 32 : 128) / p.G;
  // The line of work units (key tiles, and a cost per query tile) has 32-bit
  // coordinates: its length at the tables' full width has to fit.
  const long long own_tiles = (((long long)p.bt.max_pages << p.kv.page_shift) + 127) / 128;
  const long long pre_tiles = (((long long)p.pmax_pages << p.kv.page_shift) + 127) / 128;
  const long long q_tiles = p.bt.n_rows / p.rows_per_tile + p.bt.n_seqs;
  if (q_tiles * p.kv.Hkv * (2 * own_tiles + pre_tiles + 8) >= (1ll << 31))
    return DLLM_ERR_UNSUPPORTED;
  p.segs = segs;
  p.row_limit = row_limit;
  p.scale_log2 = 1.4426950408889634f * (scale > 0.f ? scale : 1.f / sqrtf((float)D));
  p.lse = lse;
  p.status = static_cast<int*>(ws);
  p.cut = reinterpret_cast<int4*>(w + kWsCut);
  p.part = reinterpret_cast<float*>(w + kWsParts);
  p.part_ml = reinterpret_cast<float2*>(p.part + (size_t)2 * kNumSMs * p.slot_rows * D);
  e = prepare_device();
  if (e != DLLM_OK) return e;
  const cuuint32_t bd = D >= 64 ? 64 : D;
  const cuuint64_t qd[3] = {(cuuint64_t)D, (cuuint64_t)n_q_heads, (cuuint64_t)p.bt.n_rows};
  const long long qs[2] = {p.q.head_stride, p.q.row_stride};
  const cuuint32_t qb[3] = {bd, (cuuint32_t)p.G, (cuuint32_t)p.rows_per_tile};
  const cuuint64_t kd[4] = {(cuuint64_t)D, (cuuint64_t)kv->page_size, (cuuint64_t)p.kv.Hkv,
                            (cuuint64_t)p.kv.n_pages};
  const long long ks[3] = {p.kv.slot_stride, p.kv.head_stride, p.kv.page_stride};
  const cuuint32_t kb[4] = {bd, (cuuint32_t)std::min(kv->page_size, 128), 1, 1};
  CUtensorMap qm, km, vm;
  if (!make_map(&qm, p.q.data, 3, qd, qs, qb, D) || !make_map(&km, p.kv.k, 4, kd, ks, kb, D) ||
      !make_map(&vm, p.kv.v, 4, kd, ks, kb, D))
    return DLLM_ERR_CUDA;
  return launch_paged_attn(qm, km, vm, p, mode, reinterpret_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
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
                                      int32_t max_rows, size_t* bytes) {
  PagedPool pool;
  dllm_status e = check_shape(kv, &pool);
  if (e == DLLM_OK) e = check_heads(n_q_heads, pool);
  if (e != DLLM_OK) return e;
  if (!bytes || max_rows < 1) return DLLM_ERR_INVALID;
  if (max_rows >= kMaxRows) return DLLM_ERR_UNSUPPORTED;
  *bytes = workspace_bytes(pool, slot_rows(max_rows, n_q_heads / pool.Hkv));
  return DLLM_OK;
}

dllm_status dllm_paged_workspace_init(void* ws, size_t ws_bytes, dllm_stream stream) {
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256) return DLLM_ERR_INVALID;
  if (ws_bytes < kWsParts) return DLLM_ERR_WORKSPACE;
  const dllm_status e = prepare_device();  // so that the first attention may be a captured one
  if (e != DLLM_OK) return e;
  return cudaMemsetAsync(ws, 0, kWsCut, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
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

dllm_status dllm_selftest_paged_timeout(const dllm_kv_pages* kv, const dllm_paged_batch* batch,
                                        int32_t n_q_heads, const int32_t* segs,
                                        const dllm_rows* q, const dllm_rows* out, void* ws,
                                        size_t ws_bytes, int32_t where, int32_t limit_us,
                                        dllm_stream stream) {
  if (where < 0 || where > 2 || limit_us < 1 || limit_us > 1000000) return DLLM_ERR_INVALID;
  return run_attn(kv, batch, nullptr, n_q_heads, segs, nullptr, 0.f, q, out, nullptr, ws, ws_bytes,
                  stream, kStallPiece + where, 1000ull * limit_us);
}

}  // extern "C"
