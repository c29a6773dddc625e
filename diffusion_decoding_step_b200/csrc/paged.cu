// Paged key/value cache: appending rows with the position rotation, and
// attention over the pages, with or without a prefix that sequences share.
#include <cuda_fp16.h>
#include <float.h>
#include <limits.h>

#include "kernels.cuh"
#include "ptx.cuh"

namespace dllm {

namespace {

template <bool F16>
DLLM_DEV float2 unpack2(uint32_t u) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&u));
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}
template <bool F16>
DLLM_DEV uint32_t pack2(float a, float b) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Rows [r0, r1) of sequence s, clamped to the row buffers whatever row_start holds.
DLLM_DEV void seq_rows(const PagedBatch& bt, int s, int& r0, int& r1) {
  r0 = min(max(bt.row_start[s], 0), bt.n_rows);
  r1 = min(max(bt.row_start[s + 1], r0), bt.n_rows);
}

// The two key segments of sequence s as disjoint ranges [a0, e0), [a1, e1)
// inside the positions that the page table covers.
struct Segs {
  int a0, e0, a1, e1;
};
DLLM_DEV Segs seq_segs(const PagedAttnParams& p, int s) {
  const int* g = p.segs + 4 * (size_t)s;
  const long long cap = (long long)p.bt.max_pages << p.kv.page_shift;
  long long a[2], e[2];
  bool cut = false;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const long long st = g[2 * j], len = g[2 * j + 1];
    a[j] = max(st, 0ll);
    e[j] = max(min(st + max(len, 0ll), cap), a[j]);
    cut |= len > 0 && (st < 0 || st + len > cap);
    if (len <= 0 || a[j] >= cap) a[j] = e[j] = 0;
  }
  if (cut && p.status != nullptr) atomicOr(p.status, kErrIndex);
  if (a[0] < e[0] && a[1] < e[1]) {  // the part of the second that the first does not cover
    if (a[1] >= a[0]) {
      a[1] = max(a[1], e[0]);
    } else if (e[1] <= e[0]) {
      e[1] = min(e[1], a[0]);
    } else {  // the second covers the first
      a[0] = a[1];
      e[0] = e[1];
      a[1] = e[1] = 0;
    }
    if (a[1] >= e[1]) a[1] = e[1] = 0;
  }
  return Segs{(int)a[0], (int)e[0], (int)a[1], (int)e[1]};
}

}  // namespace

// ------------------------------------------------------------------ append
// One warp of the block resolves a row: its sequence (the count of
// row_start[1..] that are <= r, loaded side by side instead of searched one
// after the other), its slot, and the cosines and sines of its position,
// which all heads share.  The angle is position * theta^(-2i/D) in turns,
// reduced in 64 bits, so that far positions keep their fraction of a turn.
// Then the block's threads move 2 x 16 bytes of a head each: elements i.. and
// i + D/2.., which the rotation pairs.  The operator is bound by its bytes.
constexpr int kAppendThreads = 256;
constexpr int kAppendRows = 4;  // rows per block

template <int D, bool F16>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(
    const __grid_constant__ PagedAppendParams p) {
  constexpr int kHalf = D / 2;
  constexpr int kLanes = kHalf / 8;  // threads per head
  __shared__ float2 cs[kAppendRows][kHalf];
  __shared__ long long slot_off[kAppendRows];  // element offset of the row's slot, or -1
  __shared__ int row_ok[kAppendRows];
  grid_dep_wait();
  grid_dep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * kAppendRows;
  if (warp < kAppendRows) {
    const int r = row0 + warp;
    int n = 0;
    if (r < p.bt.n_rows)
      for (int i = lane; i < p.bt.n_seqs; i += 32) n += p.bt.row_start[i + 1] <= r;
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    bool ok = false;
    long long off = -1;
    if (r < p.bt.n_rows && n < p.bt.n_seqs) {
      const int first = p.bt.row_start[n];
      ok = first >= 0 && r >= first;
      const long long pos = (long long)p.pos[n] + (r - first);
      if (ok) {
        const long long pg = pos >> p.kv.page_shift;
        int page = -1;
        if (pos >= 0 && pg < p.bt.max_pages)
          page = p.bt.table[(size_t)n * p.bt.table_stride + pg];
        if (page >= 0 && page < p.kv.n_pages)
          off = page * p.kv.page_stride +
                (pos & ((1ll << p.kv.page_shift) - 1)) * p.kv.slot_stride;
        else if (lane == 0 && p.status != nullptr)
          atomicOr(p.status, kErrIndex);
        if (p.rope) {
          const double t = (double)(pos + (p.shift ? p.shift[n] : 0));
#pragma unroll
          for (int i = lane; i < kHalf; i += 32) {
            const double turn = t * p.turns[i];
            float s, c;
            sincospif(2.f * (float)(turn - rint(turn)), &s, &c);
            cs[warp][i] = make_float2(c, s);
          }
        }
      }
    }
    if (lane == 0) {
      slot_off[warp] = off;
      row_ok[warp] = ok;
    }
  }
  __syncthreads();
  using T = uint16_t;
  const int heads = p.Hq + 2 * p.kv.Hkv;
  const int per_row = heads * kLanes;
  for (int i = threadIdx.x; i < kAppendRows * per_row; i += kAppendThreads) {
    const int rr = i / per_row, x = i - rr * per_row;
    if (!row_ok[rr]) continue;
    const int hh = x / kLanes, e = (x - hh * kLanes) * 8;
    const long long r = row0 + rr;
    const T* src;
    T* dst;
    bool rot = p.rope != 0;
    if (hh < p.Hq) {
      src = static_cast<const T*>(p.q.data) + r * p.q.row_stride + hh * p.q.head_stride;
      dst = static_cast<T*>(p.q_out.data) + r * p.q_out.row_stride + hh * p.q_out.head_stride;
    } else {
      const long long off = slot_off[rr];
      if (off < 0) continue;
      int h = hh - p.Hq;
      if (h < p.kv.Hkv) {
        src = static_cast<const T*>(p.k.data) + r * p.k.row_stride + h * p.k.head_stride;
        dst = static_cast<T*>(p.kv.k) + off + h * p.kv.head_stride;
      } else {
        h -= p.kv.Hkv;
        src = static_cast<const T*>(p.v.data) + r * p.v.row_stride + h * p.v.head_stride;
        dst = static_cast<T*>(p.kv.v) + off + h * p.kv.head_stride;
        rot = false;
      }
    }
    uint4 lo = *reinterpret_cast<const uint4*>(src + e);
    uint4 hi = *reinterpret_cast<const uint4*>(src + kHalf + e);
    if (rot) {
      uint32_t* a = reinterpret_cast<uint32_t*>(&lo);
      uint32_t* b = reinterpret_cast<uint32_t*>(&hi);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 c = *reinterpret_cast<const float4*>(&cs[rr][e + 2 * j]);  // c0 s0 c1 s1
        const float2 u = unpack2<F16>(a[j]), w = unpack2<F16>(b[j]);
        a[j] = pack2<F16>(u.x * c.x - w.x * c.y, u.y * c.z - w.y * c.w);
        b[j] = pack2<F16>(w.x * c.x + u.x * c.y, w.y * c.z + u.y * c.w);
      }
    }
    *reinterpret_cast<uint4*>(dst + e) = lo;
    *reinterpret_cast<uint4*>(dst + kHalf + e) = hi;
  }
}

namespace {

template <class K, class P>
cudaError_t launch_pdl(K kern, dim3 grid, dim3 block, size_t smem, cudaStream_t s, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, cudaStream_t s) {
  const dim3 grid((p.bt.n_rows + kAppendRows - 1) / kAppendRows), block(kAppendThreads);
  const int D = p.kv.D;
  if (p.kv.f16)
    return D == 128  ? launch_pdl(paged_append_kernel<128, true>, grid, block, 0, s, p)
           : D == 64 ? launch_pdl(paged_append_kernel<64, true>, grid, block, 0, s, p)
                     : launch_pdl(paged_append_kernel<32, true>, grid, block, 0, s, p);
  return D == 128  ? launch_pdl(paged_append_kernel<128, false>, grid, block, 0, s, p)
         : D == 64 ? launch_pdl(paged_append_kernel<64, false>, grid, block, 0, s, p)
                   : launch_pdl(paged_append_kernel<32, false>, grid, block, 0, s, p);
}

// ------------------------------------------------------------------ attention
// One block per (row, query head): 128 keys at a time, one per thread, with a
// running maximum and sum; then each thread adds up its output elements.
constexpr int kSimpleThreads = 128;

template <bool F16>
DLLM_DEV float elem(const void* base, long long i) {
  const uint16_t u = static_cast<const uint16_t*>(base)[i];
  return unpack2<F16>(u).x;
}

template <int D, bool F16>
__global__ void __launch_bounds__(kSimpleThreads) paged_attn_simple_kernel(
    const __grid_constant__ PagedAttnParams p) {
  __shared__ float q_s[D], pr[kSimpleThreads], red[kSimpleThreads];
  __shared__ long long off_s[kSimpleThreads];
  grid_dep_wait();
  const int t = threadIdx.x, r = blockIdx.x, h = blockIdx.y;
  const int kvh = h / (p.Hq / p.kv.Hkv);
  int s = -1;
  for (int i = 0; i < p.bt.n_seqs; ++i) {
    int r0, r1;
    seq_rows(p.bt, i, r0, r1);
    if (r >= r0 && r < r1) s = i;
  }
  if (s < 0) return;
  int grp = -1;
  for (int i = 0; i < p.n_groups; ++i)
    if (s >= p.gseq[i] && s < p.gseq[i + 1]) grp = i;
  if (t < D) q_s[t] = elem<F16>(p.q.data, r * p.q.row_stride + h * p.q.head_stride + t);
  __syncthreads();
  float m = -FLT_MAX, l = 0.f, o = 0.f;  // o: element t % D
  auto range = [&](int a, int e, const int* table) {
    for (int k0 = a; k0 < e; k0 += kSimpleThreads) {
      const int k = k0 + t;
      float sc = -INFINITY;
      off_s[t] = -1;
      if (k < e) {
        const int page = table[k >> p.kv.page_shift];
        const bool ok = page >= 0 && page < p.kv.n_pages;
        if (!ok && p.status) atomicOr(p.status, kErrIndex);
        float d = 0.f;
        if (ok) {
          const long long off = page * p.kv.page_stride + kvh * p.kv.head_stride +
                                (k & ((1 << p.kv.page_shift) - 1)) * p.kv.slot_stride;
          off_s[t] = off;
          for (int i = 0; i < D; ++i) d += q_s[i] * elem<F16>(p.kv.k, off + i);
        }
        sc = d * p.scale_log2;
      }
      red[t] = sc;
      __syncthreads();
      float mt = m;
      for (int i = 0; i < kSimpleThreads; ++i) mt = fmaxf(mt, red[i]);
      pr[t] = exp2f(sc - mt);
      const float alpha = exp2f(m - mt);
      m = mt;
      __syncthreads();
      l *= alpha;
      o *= alpha;
      for (int i = 0; i < kSimpleThreads; ++i) {
        l += pr[i];
        if (off_s[i] >= 0) o += pr[i] * elem<F16>(p.kv.v, off_s[i] + t % D);
      }
      __syncthreads();
    }
  };
  if (grp >= 0) {
    const long long cap = (long long)p.pmax_pages << p.kv.page_shift;
    if (p.plen[grp] > cap && t == 0 && p.status) atomicOr(p.status, kErrIndex);
    range(0, (int)min((long long)p.plen[grp], cap), p.ptable + (size_t)grp * p.ptable_stride);
  }
  const Segs sg = seq_segs(p, s);
  const int lim = p.row_limit ? p.row_limit[r] : INT_MAX;
  range(sg.a0, min(sg.e0, lim), p.bt.table + (size_t)s * p.bt.table_stride);
  range(sg.a1, min(sg.e1, lim), p.bt.table + (size_t)s * p.bt.table_stride);
  if (t < D) {
    const uint32_t u = pack2<F16>(l > 0.f ? o / l : 0.f, 0.f);
    static_cast<uint16_t*>(p.out.data)[r * p.out.row_stride + h * p.out.head_stride + t] =
        (uint16_t)u;
  }
  if (t == 0 && p.lse)
    p.lse[(size_t)r * p.Hq + h] = l > 0.f ? 0.6931471805599453f * m + logf(l) : -INFINITY;
}

cudaError_t launch_paged_attn(const PagedAttnParams& p, cudaStream_t s) {
  const dim3 grid(p.bt.n_rows, p.Hq), block(kSimpleThreads);
  const int D = p.kv.D;
  if (p.kv.f16)
    return D == 128  ? launch_pdl(paged_attn_simple_kernel<128, true>, grid, block, 0, s, p)
           : D == 64 ? launch_pdl(paged_attn_simple_kernel<64, true>, grid, block, 0, s, p)
                     : launch_pdl(paged_attn_simple_kernel<32, true>, grid, block, 0, s, p);
  return D == 128  ? launch_pdl(paged_attn_simple_kernel<128, false>, grid, block, 0, s, p)
         : D == 64 ? launch_pdl(paged_attn_simple_kernel<64, false>, grid, block, 0, s, p)
                   : launch_pdl(paged_attn_simple_kernel<32, false>, grid, block, 0, s, p);
}

}  // namespace dllm
