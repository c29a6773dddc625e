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

template <class K, class... A>
cudaError_t launch_pdl(K kern, dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       const A&... args) {
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
  return cudaLaunchKernelEx(&cfg, kern, args...);
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
// Work.  An item is the own part of a sequence, or the prefix of a group: a
// range of rows, and a list of 128-key tiles (aligned to 128 positions, so
// that a tile is a whole number of pages or lies inside one).  The rows of an
// item times the G query heads of a kv head are packed into tiles of 128
// query rows, so a prefix is multiplied with the rows of all its sequences at
// once.  All (item, kv head, query tile, key tile) units in this order form
// one line that the CTAs (one per SM) cut into equal shares, whatever the
// lengths on the device are: no host knowledge of them is needed, and the
// shares of a ragged batch differ by one unit.  Every CTA finds its share
// itself by a prefix sum over the items.
//
// A share is a list of pieces (a query tile and a run of key tiles).  Roles:
//   warp 8      walks the share, describes each piece in a small queue, and
//               loads Q, K and V tiles through TMA; each lane fetches its
//               page's table entry and issues that page's boxes.  Pages that
//               hold no key of the tile are requested past the last page, which
//               TMA fills with zeros without reading.
//   warp 9      issues S = Q K^T and O += P V on tcgen05.
//   warps 0-3   softmax of the even key tiles of a piece, warps 4-7 of the odd
//               ones: two streams with their own S, P and O in TMEM, so that
//               the products of one run during the softmax of the other.  A
//               thread owns a query row; P overwrites S in TMEM as the A
//               operand of the second product.  O is rescaled only when the
//               row's maximum grew by more than 2^8 (the kept maximum is then
//               stale, which the final division cancels).
// At the end of a piece the two streams' O are merged.  A tile that one CTA
// did alone is written out; the parts of a cut tile go to the workspace in
// fp32, and a second kernel merges them in a fixed order.
constexpr int kKeyTile = 128;
constexpr int kAttnThreads = 320;
constexpr int kMaxItems = 2048;
constexpr int kQueue = 4;
constexpr float kGrow = 8.f;  // log2 of the growth of a maximum that rescales O

struct Piece {
  int r0, nrows, kvh, n;        // first row, rows, kv head, key tiles (-1: no more pieces)
  int kt0, kind;                // first key tile; 0 own part, 1 prefix
  int a0, e0, a1, e1;           // key ranges
  int dest;                     // kDestOut / kDestWhole / kDestPart
  int slot;                     // partial slot
  int where_x, where_y;         // row map entry to write, or where_x < 0
  int pad0, pad1;
};
enum : int { kDestOut = 0, kDestWhole = 1, kDestPart = 2 };
// Row map entry: x = dest | 4 if the row also has a prefix part | the row's
// place in its query tile << 3; y = first slot | parts << 16.

template <int D, int ST>
struct PagedCfg {
  static constexpr int kBoxD = D >= 64 ? 64 : D;
  static constexpr int kRowBytes = kBoxD * 2;
  static constexpr int kSw = kRowBytes == 128 ? 2 : 4;
  static constexpr int kNBox = D / kBoxD;
  static constexpr int kBoxBytes = 128 * kRowBytes;
  static constexpr int kTile = 128 * D * 2;  // bytes of a Q, K or V tile
  static constexpr int kScan = (kMaxItems + 1) * 8;
  static constexpr int kXBytes = 2 * 2 * 128 * 8;  // (max, sum) of both streams, two pieces
  static constexpr size_t kSmem =
      1024 + (1 + ST) * kTile + kScan + 8 + kXBytes + kQueue * sizeof(Piece) + 512;
};

struct Item {
  int r0, r1, kt, n0, tiles;
  Segs sg;
  const int* table;
  int kind, seq;
};

DLLM_DEV int key_tiles(int a, int e) { return e > a ? (e + kKeyTile - 1) / kKeyTile - a / kKeyTile : 0; }

DLLM_DEV Item load_item(const PagedAttnParams& p, int i) {
  Item it;
  if (i < p.n_groups) {
    const int g0 = min(max(p.gseq[i], 0), p.bt.n_seqs);
    const int g1 = min(max(p.gseq[i + 1], g0), p.bt.n_seqs);
    it.r0 = min(max(p.bt.row_start[g0], 0), p.bt.n_rows);
    it.r1 = min(max(p.bt.row_start[g1], it.r0), p.bt.n_rows);
    const int cap = p.pmax_pages << p.kv.page_shift;
    const int len = p.plen[i];
    if (len > cap && p.status != nullptr) atomicOr(p.status, kErrIndex);
    it.sg = Segs{0, min(max(len, 0), cap), 0, 0};
    it.table = p.ptable + (size_t)i * p.ptable_stride;
    it.kind = 1;
    it.seq = -1;
  } else {
    const int s = i - p.n_groups;
    seq_rows(p.bt, s, it.r0, it.r1);
    it.sg = seq_segs(p, s);
    it.table = p.bt.table + (size_t)s * p.bt.table_stride;
    it.kind = 0;
    it.seq = s;
  }
  it.n0 = key_tiles(it.sg.a0, it.sg.e0);
  it.kt = it.n0 + key_tiles(it.sg.a1, it.sg.e1);
  it.tiles = (it.r1 - it.r0 + p.rows_per_tile - 1) / p.rows_per_tile;
  return it;
}
// Units of one query tile and kv head: its key tiles, and one for an own part
// without keys, whose output has to be written all the same.
DLLM_DEV int tile_units(const Item& it) { return it.kind ? it.kt : max(it.kt, 1); }

// First position and visible range [lo, hi) of key tile t of the ranges.
DLLM_DEV void key_tile(int a0, int e0, int a1, int e1, int t, int& base, int& lo, int& hi) {
  const int n0 = key_tiles(a0, e0);
  const int a = t < n0 ? a0 : a1, e = t < n0 ? e0 : e1;
  base = (a / kKeyTile + (t < n0 ? t : t - n0)) * kKeyTile;
  lo = max(a, base);
  hi = min(e, base + kKeyTile);
}

// Whether sequence s lies in a group with a prefix (whole warp).
DLLM_DEV bool has_prefix(const PagedAttnParams& p, int s, int lane) {
  bool in = false;
  for (int g = lane; g < p.n_groups; g += 32)
    in |= p.gseq[g] <= s && s < p.gseq[g + 1] && p.plen[g] > 0;
  return __any_sync(0xffffffffu, in);
}

// A wait that ends when another role gave up; sets the flag when it gives up itself.
DLLM_DEV bool wait_or_abort(uint64_t* bar, uint32_t parity, int* status, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63u) == 0u) {
      if (*abort) return false;
      if (global_ns() - t0 > kWaitLimitNs) {
        *abort = 1;
        if (status) atomicOr(status, kErrTimeout);
        return false;
      }
    }
  }
}

template <int D, bool F16, int ST>
__global__ void __launch_bounds__(kAttnThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ PagedAttnParams p) {
  using C = PagedCfg<D, ST>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base_s = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
  uint8_t* q_s = base_s;
  uint8_t* kv_s = q_s + C::kTile;  // [ST]
  long long* upfx = reinterpret_cast<long long*>(kv_s + ST * C::kTile);  // [items + 1]
  float2* x_s = reinterpret_cast<float2*>(upfx + kMaxItems + 2);         // [2][2][128]
  Piece* queue = reinterpret_cast<Piece*>(x_s + 2 * 2 * 128);
  uint64_t* bars = reinterpret_cast<uint64_t*>(queue + kQueue);
  uint64_t* kv_full = bars;             // [ST]
  uint64_t* kv_empty = kv_full + ST;    // [ST]
  uint64_t* d_full = kv_empty + ST;     // [kQueue]
  uint64_t* d_empty = d_full + kQueue;  // [kQueue]
  uint64_t* s_full = d_empty + kQueue;  // [2]
  uint64_t* p_full = s_full + 2;        // [2]
  uint64_t* q_full = p_full + 2;
  uint64_t* q_empty = q_full + 1;
  uint64_t* o_full = q_empty + 1;
  uint64_t* o_empty = o_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_empty + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if (t == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], 257);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 128);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(o_full, 1);
    mbar_init(o_empty, 256);
    *abort = 0;
    fence_barrier_init();
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  grid_dep_wait();

  // ---- prefix sum of the items' units
  const int n_items = p.n_groups + p.bt.n_seqs;
  const int per = (n_items + kAttnThreads - 1) / kAttnThreads;
  {
    long long mine = 0;
    for (int j = 0; j < per; ++j) {
      const int i = t * per + j;
      if (i >= n_items) break;
      const Item it = load_item(p, i);
      upfx[i + 1] = mine += (long long)it.tiles * p.kv.Hkv * tile_units(it);
    }
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    long long* sums = reinterpret_cast<long long*>(x_s);
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    long long before = inc - mine;
    for (int w = 0; w < warp; ++w) before += sums[w];
    for (int j = 0; j < per; ++j) {
      const int i = t * per + j;
      if (i >= n_items) break;
      upfx[i + 1] += before;
    }
    if (t == 0) upfx[0] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();
  const uint32_t tmem = *tmem_slot;
  const long long U = upfx[n_items];
  const int G = (int)min((long long)gridDim.x, U);  // CTAs with work
  const int cta = blockIdx.x;

  if (warp == 8) {
    // ================================================================ producer
    long long u = 0, u1 = 0;
    if (cta < G) {
      u = (long long)cta * U / G;
      u1 = (long long)(cta + 1) * U / G;
    }
    int lo = 0, hi = n_items;  // the last item that starts at or before u and has units
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (upfx[mid] <= u)
        lo = mid;
      else
        hi = mid;
    }
    int i = lo;
    Item it{};
    bool pfx = false;
    if (u < u1) {
      it = load_item(p, i);
      pfx = it.kind == 0 && p.n_groups > 0 && has_prefix(p, it.seq, lane);
    }
    int4 cut = make_int4(0, 0, 0, 0);
    int pos = 0, n_piece = 0, n_q = 0;  // ring position, pieces, pieces with keys
    bool ok = true, first = true;
    const int page_boxes = max(1, kKeyTile >> p.kv.page_shift);
    const int slot_mask = (1 << p.kv.page_shift) - 1;
    const int page_keys = min(kKeyTile, slot_mask + 1);
    while (ok && u < u1) {
      while (u >= upfx[i + 1]) {
        ++i;
        if (u < upfx[i + 1]) {
          it = load_item(p, i);
          pfx = it.kind == 0 && p.n_groups > 0 && has_prefix(p, it.seq, lane);
        }
      }
      const int kt = tile_units(it);
      const long long local = u - upfx[i];
      const int tile = (int)(local / kt), k0 = (int)(local - (long long)tile * kt);
      const int k1 = (int)min((long long)kt, k0 + (u1 - u));
      const int kvh = tile / it.tiles, rt = tile - kvh * it.tiles;
      const int r0 = it.r0 + rt * p.rows_per_tile;
      const int nrows = min(p.rows_per_tile, it.r1 - r0);
      int n = it.kt > 0 ? k1 - k0 : 0;
      if (it.kind == 0 && p.row_limit != nullptr) {  // no row sees the last tiles
        int lim = 0;
        for (int r = lane; r < nrows; r += 32) lim = max(lim, p.row_limit[r0 + r]);
        lim = __reduce_max_sync(0xffffffffu, lim);
        while (n > 0) {
          int kb, kl, kh;
          key_tile(it.sg.a0, it.sg.e0, it.sg.a1, it.sg.e1, k0 + n - 1, kb, kl, kh);
          if (kl < lim) break;
          --n;
        }
      }
      const bool whole = k0 == 0 && k1 == kt;
      const int slot = 2 * cta + (first ? 0 : 1);
      int parts = 1;
      if (!whole && k0 == 0) {  // the CTA of the tile's last unit
        const long long last = upfx[i] + (long long)tile * kt + kt - 1;
        parts = (int)(((last + 1) * G + U - 1) / U) - 1 - cta + 1;
        cut = make_int4(r0, nrows, kvh, parts | (slot & 1) << 16);
      }
      const int qi = n_piece % kQueue;
      if (lane == 0) {
        ok = n_piece < kQueue ||
             wait_or_abort(&d_empty[qi], (n_piece / kQueue - 1) & 1, p.status, abort);
        if (ok) {
          Piece& d = queue[qi];
          d.r0 = r0;
          d.nrows = nrows;
          d.kvh = kvh;
          d.n = n;
          d.kt0 = k0;
          d.kind = it.kind;
          d.a0 = it.sg.a0;
          d.e0 = it.sg.e0;
          d.a1 = it.sg.a1;
          d.e1 = it.sg.e1;
          d.dest = !whole ? kDestPart : (it.kind || pfx) ? kDestWhole : kDestOut;
          d.slot = slot;
          d.where_x = p.n_groups > 0 && k0 == 0 ? d.dest | (pfx ? 4 : 0) : -1;
          d.where_y = slot | parts << 16;
          mbar_arrive(&d_full[qi]);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      ++n_piece;
      first = false;
      if (ok && n > 0) {
        if (lane == 0) {
          ok = n_q == 0 || wait_or_abort(q_empty, (n_q - 1) & 1, p.status, abort);
          if (ok) {
            mbar_arrive_expect_tx(q_full, C::kNBox * p.G * p.rows_per_tile * C::kRowBytes);
#pragma unroll
            for (int b = 0; b < C::kNBox; ++b)
              tma_load_3d(q_s + b * C::kBoxBytes, &qmap, q_full, b * C::kBoxD, kvh * p.G, r0);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        ++n_q;
        // this lane's page of key tile k0 + j (n_pages: nothing to read there)
        auto entry = [&](int j) {
          int page = p.kv.n_pages;
          if (lane < page_boxes) {
            int kb, kl, kh;
            key_tile(it.sg.a0, it.sg.e0, it.sg.a1, it.sg.e1, k0 + j, kb, kl, kh);
            const int at = kb + lane * page_keys;
            if (at < kh && at + page_keys > kl) {
              page = it.table[at >> p.kv.page_shift];
              if (page < 0 || page >= p.kv.n_pages) {
                if (p.status != nullptr) atomicOr(p.status, kErrIndex);
                page = p.kv.n_pages;
              }
            }
          }
          return page;
        };
        auto load = [&](const CUtensorMap* m, int j, int page) {
          const int st = pos % ST;
          if (lane == 0) {
            ok = pos < ST || wait_or_abort(&kv_empty[st], (pos / ST - 1) & 1, p.status, abort);
            if (ok) mbar_arrive_expect_tx(&kv_full[st], C::kTile);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (ok) {
            if (lane < page_boxes) {
              int kb, kl, kh;
              key_tile(it.sg.a0, it.sg.e0, it.sg.a1, it.sg.e1, k0 + j, kb, kl, kh);
              uint8_t* dst = kv_s + st * C::kTile + lane * page_keys * C::kRowBytes;
#pragma unroll
              for (int b = 0; b < C::kNBox; ++b)
                tma_load_4d(dst + b * C::kBoxBytes, m, &kv_full[st], b * C::kBoxD,
                            page_keys == kKeyTile ? kb & slot_mask : 0, kvh, page);
            }
            ++pos;
          }
        };
        // in the order the products take them: K0 K1 V0 K2 V1 ...
        int e0 = entry(0), e1 = n > 1 ? entry(1) : 0;
        if (ok) load(&kmap, 0, e0);
        if (ok && n > 1) load(&kmap, 1, e1);
        for (int j = 0; ok && j < n; ++j) {
          const int e2 = j + 2 < n ? entry(j + 2) : 0;
          load(&vmap, j, e0);
          if (ok && j + 2 < n) load(&kmap, j + 2, e2);
          e0 = e1;
          e1 = e2;
        }
      }
      u += k1 - k0;
    }
    if (lane == 0) {
      const int qi = n_piece % kQueue;
      if (ok && (n_piece < kQueue ||
                 wait_or_abort(&d_empty[qi], (n_piece / kQueue - 1) & 1, p.status, abort))) {
        queue[qi].n = -1;
        mbar_arrive(&d_full[qi]);
      }
      if (cta < kNumSMs) p.cut[cta] = cut;
      if (*abort) {  // copies in flight land before the block goes
        for (int x = max(0, pos - ST); x < pos; ++x)
          mbar_wait(&kv_full[x % ST], (x / ST) & 1, p.status);
        if (n_q > 0) mbar_wait(q_full, (n_q - 1) & 1, p.status);
      }
    }
  } else if (warp == 9) {
    // ================================================================ products
    if (lane == 0) {
      constexpr uint32_t kIdS = idesc_16(F16, 128, kKeyTile, 0, 0);
      constexpr uint32_t kIdO = idesc_16(F16, 128, D, 0, 1);
      const uint32_t qa = smem_u32(q_s), kva = smem_u32(kv_s);
      int pos = 0, n_piece = 0, n_q = 0;
      int cnt[2] = {0, 0};  // P tiles taken of each stream
      bool ok = true;
      while (ok) {
        const int qi = n_piece % kQueue;
        ok = wait_or_abort(&d_full[qi], (n_piece / kQueue) & 1, p.status, abort);
        if (!ok) break;
        const int n = queue[qi].n;
        mbar_arrive(&d_empty[qi]);
        ++n_piece;
        if (n < 0) break;
        if (n == 0) continue;
        auto wait_kv = [&]() {
          return wait_or_abort(&kv_full[pos % ST], (pos / ST) & 1, p.status, abort);
        };
        auto s_mma = [&](int j) {
          if (!wait_kv()) return false;
          tc_fence_after();
          const uint32_t ka = kva + (pos % ST) * C::kTile;
          const uint32_t d = tmem + (j & 1) * 128;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off =
                (kk * 16 / C::kBoxD) * C::kBoxBytes + ((kk * 16) % C::kBoxD) * 2;
            umma_bf16(d, smem_desc(qa + off, 16, 8 * C::kRowBytes, C::kSw),
                      smem_desc(ka + off, 16, 8 * C::kRowBytes, C::kSw), kIdS, kk > 0);
          }
          umma_commit(&s_full[j & 1]);
          umma_commit(&kv_empty[pos % ST]);
          if (j == n - 1) umma_commit(q_empty);
          ++pos;
          return true;
        };
        ok = wait_or_abort(q_full, n_q & 1, p.status, abort) && s_mma(0) && (n < 2 || s_mma(1));
        for (int j = 0; ok && j < n; ++j) {
          const int x = j & 1;
          ok = wait_or_abort(&p_full[x], cnt[x] & 1, p.status, abort) &&
               (j > 0 || n_q == 0 || wait_or_abort(o_empty, (n_q - 1) & 1, p.status, abort)) &&
               wait_kv();
          if (!ok) break;
          ++cnt[x];
          tc_fence_after();
          const uint32_t va = kva + (pos % ST) * C::kTile;
#pragma unroll
          for (int kk = 0; kk < kKeyTile / 16; ++kk)
            umma_f16_ts(tmem + 256 + x * 128, tmem + x * 128 + kk * 8,
                        smem_desc(va + kk * 16 * C::kRowBytes, C::kBoxBytes, 8 * C::kRowBytes,
                                  C::kSw),
                        kIdO, j > 1 || kk > 0);
          umma_commit(&kv_empty[pos % ST]);
          ++pos;
          if (j + 2 < n) ok = s_mma(j + 2);
        }
        if (ok) umma_commit(o_full);
        ++n_q;
      }
    }
  } else {
    // ================================================================ softmax
    const int wg = warp >> 2, row = t & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + lane_off + wg * 128;
    const uint32_t o_tm = tmem + lane_off + 256;
    const int rr = row / p.G, hh = row - rr * p.G;
    const int page_keys = min(kKeyTile, 1 << p.kv.page_shift);
    int n_piece = 0, n_q = 0, s_cnt = 0, kv_base = 0;
    bool ok = true;
    while (ok) {
      const int qi = n_piece % kQueue;
      ok = wait_or_abort(&d_full[qi], (n_piece / kQueue) & 1, p.status, abort);
      if (!ok) break;
      const Piece d = queue[qi];
      mbar_arrive(&d_empty[qi]);
      ++n_piece;
      if (d.n < 0) break;
      const bool valid = rr < d.nrows && rr < p.rows_per_tile;
      const bool active = __any_sync(0xffffffffu, valid);
      const int r = d.r0 + rr;
      const int lim =
          valid && d.kind == 0 && p.row_limit != nullptr ? p.row_limit[r] : INT_MAX;
      float m = -FLT_MAX, l = 0.f;
      for (int j = wg; j < d.n; j += 2) {
        int kb, kl, kh;
        key_tile(d.a0, d.e0, d.a1, d.e1, d.kt0 + j, kb, kl, kh);
        ok = wait_or_abort(&s_full[wg], s_cnt & 1, p.status, abort);
        if (!ok) break;
        ++s_cnt;
        tc_fence_after();
        if (active) {
          float s[kKeyTile];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(s_tm + c * 32, s + c * 32);
          tmem_ld_wait();
          const int first_k = kl - kb, end_k = min(kh, lim) - kb;
          if (__any_sync(0xffffffffu, valid && (first_k > 0 || end_k < kKeyTile))) {
#pragma unroll
            for (int i = 0; i < kKeyTile; ++i)
              if (i < first_k || i >= end_k) s[i] = -INFINITY;
          }
          float mx[4] = {-FLT_MAX, -FLT_MAX, -FLT_MAX, -FLT_MAX};
#pragma unroll
          for (int i = 0; i < kKeyTile; ++i) mx[i & 3] = fmaxf(mx[i & 3], s[i]);
          const float m_new =
              fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2);
          if (j == wg) {
            m = m_new;
          } else if (__any_sync(0xffffffffu, valid && m_new > m + kGrow)) {
            // S of this tile is complete, hence also the products before it
            const float alpha = fast_exp2(m - m_new);
            m = m_new;
            l *= alpha;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              float v[16];
              tmem_ld16(o_tm + wg * 128 + c * 16, v);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] *= alpha;
              tmem_st16(o_tm + wg * 128 + c * 16, v);
            }
          }
          float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float p0 = fast_exp2(fmaf(s[h * 64 + 2 * i], p.scale_log2, -m));
              const float p1 = fast_exp2(fmaf(s[h * 64 + 2 * i + 1], p.scale_log2, -m));
              ls[i & 3] += p0 + p1;
              pk[i] = pack2<F16>(p0, p1);
            }
            tmem_st32(s_tm + h * 32, pk);
          }
          l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
          tmem_st_wait();
        }
        // Slots of a loaded page outside the tile's range may hold anything,
        // infinities and NaN included: their weight is zero, their values have
        // to be as well.
        if (kl > kb || kh < kb + kKeyTile) {
          const int vp = kv_base + min(2 * j + 2, 2 * d.n - 1);
          const int key = kb + row;
          const int pg = key & ~(page_keys - 1);
          ok = wait_or_abort(&kv_full[vp % ST], (vp / ST) & 1, p.status, abort);
          if (!ok) break;
          if ((key < kl || key >= kh) && pg < kh && pg + page_keys > kl) {
            uint4* v = reinterpret_cast<uint4*>(kv_s + (vp % ST) * C::kTile + row * C::kRowBytes);
#pragma unroll
            for (int b = 0; b < C::kNBox; ++b)
#pragma unroll
              for (int c = 0; c < C::kRowBytes / 16; ++c)
                v[b * (C::kBoxBytes / 16) + c] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(&p_full[wg]);
      }
      if (!ok) break;
      // ---- the piece's result: (max, sum) of both streams, then each group of
      // warps takes one half of the columns
      float a0 = 0.f, a1 = 0.f, mt = -FLT_MAX, lt = 0.f;
      if (d.n > 0) {
        float2* x = x_s + (n_q & 1) * 256;
        x[wg * 128 + row] = make_float2(m, l);
        named_bar_sync(1, 256);
        const float2 y0 = x[row], y1 = x[128 + row];
        mt = fmaxf(y0.x, y1.x);
        a0 = fast_exp2(y0.x - mt);
        a1 = d.n > 1 ? fast_exp2(y1.x - mt) : 0.f;
        lt = y0.y * a0 + (d.n > 1 ? y1.y * a1 : 0.f);
        kv_base += 2 * d.n;
        ok = wait_or_abort(o_full, n_q & 1, p.status, abort);
        if (!ok) break;
        ++n_q;
        tc_fence_after();
      }
      constexpr int kCols = D / 2;
      const int c0 = wg * kCols;
      const int head = d.kvh * p.G + hh;
      if (active) {
        if (d.dest == kDestOut) {
          const float inv = lt > 0.f ? 1.f / lt : 0.f;
          a0 *= inv;
          a1 *= inv;
        }
        uint16_t* out = static_cast<uint16_t*>(p.out.data) + r * p.out.row_stride +
                        head * p.out.head_stride + c0;
        float* part =
            d.dest == kDestPart
                ? p.part + ((size_t)d.slot * 128 + row) * D + c0
                : p.whole + (((size_t)d.kind * p.bt.n_rows + r) * p.Hq + head) * D + c0;
#pragma unroll
        for (int c = 0; c < kCols / 16; ++c) {
          float v[16];
          if (d.n > 0) {
            tmem_ld16(o_tm + c0 + c * 16, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= a0;
            if (d.n > 1) {
              float w[16];
              tmem_ld16(o_tm + 128 + c0 + c * 16, w);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = fmaf(w[i], a1, v[i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = 0.f;
          }
          if (valid) {
            if (d.dest == kDestOut) {
#pragma unroll
              for (int i = 0; i < 16; i += 8)
                *reinterpret_cast<uint4*>(out + c * 16 + i) =
                    make_uint4(pack2<F16>(v[i], v[i + 1]), pack2<F16>(v[i + 2], v[i + 3]),
                               pack2<F16>(v[i + 4], v[i + 5]), pack2<F16>(v[i + 6], v[i + 7]));
            } else {
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(part + c * 16 + i) =
                    make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
          }
        }
      }
      if (d.n > 0) {
        tc_fence_before();
        mbar_arrive(o_empty);
      }
      if (valid && wg == 0) {
        if (d.dest == kDestOut) {
          if (p.lse != nullptr)
            p.lse[(size_t)r * p.Hq + head] =
                lt > 0.f ? 0.6931471805599453f * mt + logf(lt) : -INFINITY;
        } else if (d.dest == kDestPart) {
          p.part_ml[d.slot * 128 + row] = make_float2(mt, lt);
        } else {
          p.whole_ml[((size_t)d.kind * p.bt.n_rows + r) * p.Hq + head] = make_float2(mt, lt);
        }
        if (d.where_x >= 0 && hh == 0)
          p.where[((size_t)d.kind * p.bt.n_rows + r) * p.kv.Hkv + d.kvh] =
              make_int2(d.where_x | (rr * p.G) << 3, d.where_y);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ merges
// Lane i of a warp holds D / 32 neighbouring elements of a row.
template <int D>
struct RowSum {
  static constexpr int kE = D / 32;
  float m = -FLT_MAX, l = 0.f, o[kE];
  DLLM_DEV RowSum() {
#pragma unroll
    for (int i = 0; i < kE; ++i) o[i] = 0.f;
  }
  DLLM_DEV void add(float2 ml, const float* part, int lane) {
    float v[kE];
    if constexpr (kE == 4)
      *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(part + 4 * lane);
    else if constexpr (kE == 2)
      *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(part + 2 * lane);
    else
      v[0] = part[lane];
    join(ml, v);
  }
  DLLM_DEV void join(float2 ml, const float* v) {
    const float mn = fmaxf(m, ml.x);
    const float a = fast_exp2(m - mn), b = fast_exp2(ml.x - mn);
    m = mn;
    l = l * a + ml.y * b;
#pragma unroll
    for (int i = 0; i < kE; ++i) o[i] = o[i] * a + v[i] * b;
  }
};

template <int D, bool F16>
DLLM_DEV void write_row(const PagedAttnParams& p, const RowSum<D>& s, int r, int head, int lane) {
  constexpr int kE = RowSum<D>::kE;
  const float inv = s.l > 0.f ? 1.f / s.l : 0.f;
  uint16_t* out =
      static_cast<uint16_t*>(p.out.data) + r * p.out.row_stride + head * p.out.head_stride;
  if constexpr (kE == 1) {
    out[lane] = (uint16_t)pack2<F16>(s.o[0] * inv, 0.f);
  } else {
    uint32_t w[kE / 2];
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) w[i] = pack2<F16>(s.o[2 * i] * inv, s.o[2 * i + 1] * inv);
    if constexpr (kE == 4)
      *reinterpret_cast<uint2*>(out + 4 * lane) = make_uint2(w[0], w[1]);
    else
      *reinterpret_cast<uint32_t*>(out + 2 * lane) = w[0];
  }
  if (lane == 0 && p.lse != nullptr)
    p.lse[(size_t)r * p.Hq + head] =
        s.l > 0.f ? 0.6931471805599453f * s.m + logf(s.l) : -INFINITY;
}

// Without groups: block (c, y) merges rows y, y + kMergeY, ... of the cut tile
// that starts in CTA c of the attention kernel; its parts are in that CTA's
// slot and in the first slots of the CTAs after it.  The block's warps share
// the parts of a row, in a fixed order.
constexpr int kMergeWarps = 8, kMergeY = 8;

template <int D, bool F16>
__global__ void __launch_bounds__(kMergeWarps * 32)
    paged_merge_cut_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int kE = RowSum<D>::kE;
  __shared__ float2 ml_s[kMergeWarps];
  __shared__ float o_s[kMergeWarps][D];
  grid_dep_wait();
  grid_dep_launch();
  const int4 c = p.cut[blockIdx.x];
  const int parts = c.w & 0xffff;
  if (parts < 2) return;
  const int slot0 = 2 * blockIdx.x + (c.w >> 16);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int x = blockIdx.y; x < c.y * p.G; x += kMergeY) {
    RowSum<D> s;
    for (int i = warp; i < parts; i += kMergeWarps) {
      const size_t at = (size_t)(i == 0 ? slot0 : 2 * (blockIdx.x + i)) * 128 + x;
      s.add(p.part_ml[at], p.part + at * D, lane);
    }
    if (lane == 0) ml_s[warp] = make_float2(s.m, s.l);
#pragma unroll
    for (int i = 0; i < kE; ++i) o_s[warp][lane * kE + i] = s.o[i];
    __syncthreads();
    if (warp == 0) {
      for (int w = 1; w < kMergeWarps; ++w) s.join(ml_s[w], &o_s[w][lane * kE]);
      const int rr = x / p.G;
      write_row<D, F16>(p, s, c.x + rr, c.z * p.G + x - rr * p.G, lane);
    }
    __syncthreads();
  }
}

// With groups: one warp per (row, query head) merges its own part and its
// prefix part, each whole or cut.  Rows of no sequence, and rows that the
// attention kernel wrote itself, are left alone.
template <int D, bool F16>
__global__ void __launch_bounds__(kMergeWarps * 32)
    paged_merge_rows_kernel(const __grid_constant__ PagedAttnParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const long long id = (long long)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
  const int r = (int)(id / p.Hq), head = (int)(id - (long long)r * p.Hq);
  if (r >= p.bt.n_rows || r < p.bt.row_start[0] || r >= p.bt.row_start[p.bt.n_seqs]) return;
  const int kvh = head / p.G;
  const int2 own = p.where[(size_t)r * p.kv.Hkv + kvh];
  if ((own.x & 3) == kDestOut) return;
  RowSum<D> s;
  for (int kind = 0; kind < ((own.x & 4) ? 2 : 1); ++kind) {
    const size_t row = (size_t)kind * p.bt.n_rows + r;
    const int2 w = kind ? p.where[row * p.kv.Hkv + kvh] : own;
    if ((w.x & 3) == kDestWhole) {
      const size_t at = row * p.Hq + head;
      s.add(p.whole_ml[at], p.whole + at * D, lane);
    } else if ((w.x & 3) == kDestPart) {
      // bounded whatever the entry holds: a row that a decreasing row_start
      // leaves without a tile has an old one
      const int c0 = min((w.y & 0xffff) >> 1, kNumSMs - 1), slot0 = 2 * c0 + (w.y & 1);
      const int parts = min(w.y >> 16, kNumSMs - c0);
      const int x = min(((w.x >> 3) & 127) + head - kvh * p.G, 127);
      for (int i = 0; i < parts; ++i) {
        const size_t at = (size_t)(i == 0 ? slot0 : 2 * (c0 + i)) * 128 + x;
        s.add(p.part_ml[at], p.part + at * D, lane);
      }
    }
  }
  write_row<D, F16>(p, s, r, head, lane);
}

namespace {

constexpr int kStages = 5;

template <int D, bool F16>
cudaError_t launch_paged_attn_t(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm,
                                const PagedAttnParams& p, cudaStream_t s) {
  const cudaError_t e =
      launch_pdl(paged_attn_kernel<D, F16, kStages>, dim3(kNumSMs), dim3(kAttnThreads),
                 PagedCfg<D, kStages>::kSmem, s, qm, km, vm, p);
  if (e != cudaSuccess) return e;
  const dim3 block(kMergeWarps * 32);
  if (p.n_groups == 0)
    return launch_pdl(paged_merge_cut_kernel<D, F16>, dim3(kNumSMs, kMergeY), block, 0, s, p);
  const long long warps = (long long)p.bt.n_rows * p.Hq;
  return launch_pdl(paged_merge_rows_kernel<D, F16>,
                    dim3((unsigned)((warps + kMergeWarps - 1) / kMergeWarps)), block, 0, s, p);
}

template <int D, bool F16>
cudaError_t prepare_t() {
  return cudaFuncSetAttribute(paged_attn_kernel<D, F16, kStages>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)PagedCfg<D, kStages>::kSmem);
}

}  // namespace

cudaError_t paged_attn_prepare() {
  cudaError_t e = prepare_t<128, false>();
  if (e == cudaSuccess) e = prepare_t<128, true>();
  if (e == cudaSuccess) e = prepare_t<64, false>();
  if (e == cudaSuccess) e = prepare_t<64, true>();
  if (e == cudaSuccess) e = prepare_t<32, false>();
  if (e == cudaSuccess) e = prepare_t<32, true>();
  return e;
}

cudaError_t launch_paged_attn(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm,
                              const PagedAttnParams& p, cudaStream_t s) {
  const int D = p.kv.D;
  if (p.kv.f16)
    return D == 128  ? launch_paged_attn_t<128, true>(qm, km, vm, p, s)
           : D == 64 ? launch_paged_attn_t<64, true>(qm, km, vm, p, s)
                     : launch_paged_attn_t<32, true>(qm, km, vm, p, s);
  return D == 128  ? launch_paged_attn_t<128, false>(qm, km, vm, p, s)
         : D == 64 ? launch_paged_attn_t<64, false>(qm, km, vm, p, s)
                   : launch_paged_attn_t<32, false>(qm, km, vm, p, s);
}

}  // namespace dllm
