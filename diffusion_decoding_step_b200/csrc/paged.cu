// Paged key/value cache: appending rows with the position rotation, and
// attention over the pages, with or without a prefix that sequences share.
#include <cuda_fp16.h>
#include <float.h>
#include <limits.h>

#include <type_traits>

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

// Visible range of (start, len) inside [0, cap); false if it reaches outside.
DLLM_DEV bool clip_range(int st, int len, int cap, int& a, int& e) {
  len = max(len, 0);
  a = max(st, 0);
  e = st < 0 ? min(st + len, cap) : a >= cap || len > cap - a ? cap : a + len;
  const bool inside = len == 0 || (st >= 0 && a < cap && len <= cap - a);
  if (len == 0 || e <= a) a = e = 0;
  return inside;
}

// The two key segments of sequence s as disjoint ranges [a0, e0), [a1, e1)
// inside the positions that the page table covers.
struct Segs {
  int a0, e0, a1, e1;
};
DLLM_DEV Segs make_segs(const PagedAttnParams& p, int s0, int l0, int s1, int l1) {
  const int cap = p.bt.max_pages << p.kv.page_shift;
  Segs r;
  const bool in0 = clip_range(s0, l0, cap, r.a0, r.e0), in1 = clip_range(s1, l1, cap, r.a1, r.e1);
  if (!(in0 && in1) && p.status != nullptr) atomicOr(p.status, kErrIndex);
  if (r.a1 < r.e0 && r.a0 < r.e1) {  // they overlap: together one range
    r.a0 = min(r.a0, r.a1);
    r.e0 = max(r.e0, r.e1);
    r.a1 = r.e1 = 0;
  }
  return r;
}
DLLM_DEV Segs seq_segs(const PagedAttnParams& p, int s) {
  const int* g = p.segs + 4 * (size_t)s;
  return make_segs(p, g[0], g[1], g[2], g[3]);
}

}  // namespace

// ------------------------------------------------------------------ append
// One warp of the block resolves a row: its sequence (row_start, positions and
// shifts are loaded by all lanes side by side, and the lane whose range holds the
// row has the answer), its slot, and the cosines and sines of its position, which
// all heads share.  The angle is position * theta^(-2i/D) in turns, reduced in 64
// bits, so that far positions keep their fraction of a turn.  Meanwhile the block's
// threads already load 2 x 16 bytes of a head each, several heads at a time:
// elements i.. and i + D/2.., which the rotation pairs.  The operator is bound by
// its bytes: 9.7 thousand rows of 28 + 2 x 4 heads 38.1 us, 179 MB, 4.7 TB/s of a
// copy's 6.5; 512 rows of 96 heads 6.6 us, 3.8 TB/s.  A few rows are bound by the two
// dependent loads (sequence, page): one row 3.2 us.
constexpr int kAppendThreads = 256;
constexpr int kAppendRows = 8;   // most rows of a block, one for each warp

// BATCH: heads a thread has in flight.
template <int D, bool F16, int BATCH>
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
  const int rows = min(p.rows_per_block, p.bt.n_rows - (int)blockIdx.x * p.rows_per_block);
  const int row0 = blockIdx.x * p.rows_per_block;
  using T = uint16_t;
  const int heads = p.Hq + 2 * p.kv.Hkv;
  const int e = (threadIdx.x % kLanes) * 8;
  // the thread's heads: every (kAppendThreads / kLanes)-th of the block's rows
  int next_row = 0, next_head = threadIdx.x / kLanes;
  struct Item {
    uint4 lo, hi;
    int rr, hh;
  };
  Item items[BATCH];
  auto fetch = [&]() {
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      Item& x = items[k];
      while (next_head >= heads) {
        next_head -= heads;
        ++next_row;
      }
      x.rr = next_row;
      x.hh = next_head;
      next_head += kAppendThreads / kLanes;
      if (x.rr < rows) {
        const long long r = row0 + x.rr;
        const int h = x.hh - p.Hq;
        const T* src;
        if (h < 0)
          src = static_cast<const T*>(p.q.data) + r * p.q.row_stride + x.hh * p.q.head_stride;
        else if (h < p.kv.Hkv)
          src = static_cast<const T*>(p.k.data) + r * p.k.row_stride + h * p.k.head_stride;
        else
          src = static_cast<const T*>(p.v.data) + r * p.v.row_stride +
                (h - p.kv.Hkv) * p.v.head_stride;
        x.lo = *reinterpret_cast<const uint4*>(src + e);
        x.hi = *reinterpret_cast<const uint4*>(src + kHalf + e);
      }
    }
  };
  fetch();

  if (warp < rows) {
    const int r = row0 + warp;
    int seq = -1, first = 0;
    long long at = 0, shift = 0;
    for (int i = 0; i < p.bt.n_seqs; i += 32) {
      const int s = min(i + lane, p.bt.n_seqs - 1);
      const int a = p.bt.row_start[s], b = p.bt.row_start[s + 1], ps = p.pos[s];
      const int sh = p.shift ? p.shift[s] : 0;
      const unsigned who = __ballot_sync(0xffffffffu, a >= 0 && a <= r && r < b && i + lane == s);
      if (who != 0) {  // the last one, should row_start name several
        const int l = 31 - __clz(who);
        seq = i + l;
        first = __shfl_sync(0xffffffffu, a, l);
        at = __shfl_sync(0xffffffffu, ps, l);
        shift = __shfl_sync(0xffffffffu, sh, l);
      }
    }
    long long off = -1;
    if (seq >= 0) {
      const long long pos = at + (r - first);
      const long long pg = pos >> p.kv.page_shift;
      int page = -1;
      if (pos >= 0 && pg < p.bt.max_pages)
        page = p.bt.table[(size_t)seq * p.bt.table_stride + pg];
      if (p.rope) {
        const double t = (double)(pos + shift);
#pragma unroll
        for (int i = lane; i < kHalf; i += 32) {
          const double turn = t * p.turns[i];
          float s, c;
          sincospif(2.f * (float)(turn - rint(turn)), &s, &c);
          cs[warp][i] = make_float2(c, s);
        }
      }
      if (page >= 0 && page < p.kv.n_pages)
        off = page * p.kv.page_stride + (pos & ((1ll << p.kv.page_shift) - 1)) * p.kv.slot_stride;
      else if (lane == 0 && p.status != nullptr)
        atomicOr(p.status, kErrIndex);
    }
    if (lane == 0) {
      slot_off[warp] = off;
      row_ok[warp] = seq >= 0;
    }
  }
  __syncthreads();
  while (items[0].rr < rows) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      Item& x = items[k];
      if (x.rr >= rows || !row_ok[x.rr]) continue;
      T* dst;
      bool rot = p.rope != 0;
      if (x.hh < p.Hq) {
        dst = static_cast<T*>(p.q_out.data) + (long long)(row0 + x.rr) * p.q_out.row_stride +
              x.hh * p.q_out.head_stride;
      } else {
        const long long off = slot_off[x.rr];
        if (off < 0) continue;
        int h = x.hh - p.Hq;
        dst = static_cast<T*>(p.kv.k);
        if (h >= p.kv.Hkv) {
          h -= p.kv.Hkv;
          dst = static_cast<T*>(p.kv.v);
          rot = false;
        }
        dst += off + h * p.kv.head_stride;
      }
      if (rot) {
        uint32_t* a = reinterpret_cast<uint32_t*>(&x.lo);
        uint32_t* b = reinterpret_cast<uint32_t*>(&x.hi);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // cos, sin of two pairs
          const float4 c = *reinterpret_cast<const float4*>(&cs[x.rr][e + 2 * j]);
          const float2 u = unpack2<F16>(a[j]), w = unpack2<F16>(b[j]);
          a[j] = pack2<F16>(u.x * c.x - w.x * c.y, u.y * c.z - w.y * c.w);
          b[j] = pack2<F16>(w.x * c.x + u.x * c.y, w.y * c.z + u.y * c.w);
        }
      }
      *reinterpret_cast<uint4*>(dst + e) = x.lo;
      *reinterpret_cast<uint4*>(dst + kHalf + e) = x.hi;
    }
    fetch();
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

namespace {

template <int D, bool F16>
cudaError_t launch_append_t(const PagedAppendParams& params, cudaStream_t s) {
  // Few rows spread over the SMs, a block for each with three heads in flight a
  // thread; many share a block's start, and more warps with one head each do
  // better: 512 rows of 96 heads 6.7 us the first way and 8.5 the second, 9.7
  // thousand rows of 36 heads 44.7 and 38.0.
  PagedAppendParams p = params;
  const bool few = p.bt.n_rows <= 8 * kNumSMs;
  p.rows_per_block = few ? 1 : kAppendRows;
  const dim3 grid((p.bt.n_rows + p.rows_per_block - 1) / p.rows_per_block), block(kAppendThreads);
  return few ? launch_pdl(paged_append_kernel<D, F16, 3>, grid, block, 0, s, p)
             : launch_pdl(paged_append_kernel<D, F16, 1>, grid, block, 0, s, p);
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, cudaStream_t s) {
  const int D = p.kv.D;
  if (p.kv.f16)
    return D == 128  ? launch_append_t<128, true>(p, s)
           : D == 64 ? launch_append_t<64, true>(p, s)
                     : launch_append_t<32, true>(p, s);
  return D == 128  ? launch_append_t<128, false>(p, s)
         : D == 64 ? launch_append_t<64, false>(p, s)
                   : launch_append_t<32, false>(p, s);
}

// ------------------------------------------------------------------ attention
// Work.  The rows of an item (a group of sequences that share a prefix, or a
// sequence outside every group) times the G query heads of a kv head are
// packed into query tiles, so that a prefix is multiplied with the rows of all
// its sequences at once.  A query tile's keys are a list of 128-key tiles: the
// prefix, then the own keys of each sequence that has rows in the tile, which
// the other rows do not see.  Key tiles are aligned to 128 positions, so a tile
// is a whole number of pages or lies inside one.
//
// Mathematics: out = sum_k exp(x_k - m) v_k / sum_k exp(x_k - m), x_k = scale q.k, in
// one pass with a running maximum m and sum in fp32; x is taken in log2 units.  P is
// rounded to the cache's type for the second product (half a step each, as its
// input type demands), the sum takes it unrounded.
//
// What bounds it, measured over twelve calls captured in a graph, on three inputs in
// turn (called one by one they take up to 6 us more, the longest 155 instead of 135 us):
// few query rows by the keys' bytes (a token each of 32 sequences, 28 heads over 4,
// 281 MB: 57 us, 4.9 TB/s; one token over 131,001 keys 54 us, the same rate; blocks of
// 32 rows of 16 sequences, 32 heads, 284 MB: 60 us, 4.7 TB/s; in the steady state 6
// TB/s, the rest is the start and the merge); many by the products and the softmax
// between them (32 blocks of 32 rows that share 8192 keys 135 us, 920 TFLOP/s) and by
// uneven shares under a limit (two chunks of 1024 rows at 2 to 4 thousand keys 86 us,
// 665 TFLOP/s: a query tile is allotted all keys of its sequence); short ones by
// latency (32 rows over 544 keys 14 us).  Figures of single steps below are from
// before and after that step.
//
// All query tiles of all items and kv heads, each with its key tiles plus a
// fixed cost, form one line that the CTAs (one per SM) cut into equal shares,
// whatever the lengths on the device are.  Every CTA finds its share itself by
// a prefix sum over the sequences, so the host needs no lengths and a captured
// launch follows new ones.  A group's tiles are allotted their average length
// on the line; a share of the allotment stands for the same share of the keys.
//
// A share is a list of pieces (a query tile and a run of its key tiles).  Roles:
//   warps 8, 10 walk the share and load K (with Q) and V through TMA; each lane
//               fetches its page's table entry and issues that page's boxes (one
//               warp alone could not issue the boxes of 16-slot pages in time:
//               32 tokens over small pages took 81 us, with two 63).  Pages without a
//               key of the tile are requested past the last page, which TMA fills
//               with zeros without reading.  Warp 8 also describes pieces and key
//               tiles in two small queues.
//   warp 9      issues S = Q K^T and O += P V on tcgen05.  (One warp for each stream
//               let the streams' products interleave and their softmaxes run at the
//               same time: 187 us where one warp took 161 for the 32 blocks.)
//   warp 11     is the watchdog: the waits of the others are unbounded until it finds
//               that nothing was multiplied for two seconds, reports that and lets
//               them go.  (A clock in every wait made the code a tenth longer, and a
//               launch pays for its code, which it fetches anew.)  In a launch that gives
//               up it waits for the copies and products in flight.  (The producers
//               waiting for their own at their end: 32 blocks 135 -> 138 us.)
//   warps 0-3 and 4-7   softmax of two streams with their own S, P and O in
//               TMEM, so that the products of one run during the softmax of the
//               other.  A thread owns a query row; P overwrites S in TMEM as the
//               A operand of the second product.  O is rescaled only when the
//               row's maximum grew by more than 2^8 (the kept maximum is then
//               stale, which the final division cancels).
// Query tiles and streams:
//   kSplit  128 rows; the streams take key tiles in turn and are merged at the
//           end of a piece.  (256 rows, a half for each stream, share K and V but
//           halve the number of tiles to spread.  Measured when 32 blocks took 140 us:
//           144; 32 rows over 544 keys 15.9 us instead of 14.0, the prompt chunks 87
//           instead of 90.)
//   kQuad   32 rows, in four copies on the 128 lanes of TMEM; the streams take key
//           tiles in turn, and warp w of a stream takes the w-th quarter
//           of a tile's keys alone (P is zero elsewhere in its copy), so a tile
//           costs each thread 32 exponentials instead of 128.  The eight partial
//           results of a row are merged at the end of a piece.
//
// Values that are not finite.  A row's weight is zero for the keys that it does not
// see, but zero times infinity is no number, and the product takes all keys for all
// rows.  So in a key tile that some rows see and others do not (other sequences' rows,
// earlier rows under a limit) the softmax looks through V while it is in shared memory.
// What is not finite is set to zero there, and the rows that see it note the column and
// the sign (both signs: NaN) and put it into their result at the end.
//
// A query tile that one CTA did alone is written out.  The parts of a cut tile
// go to the workspace in fp32, and a second kernel merges them in the order of
// the keys.
constexpr int kKeyTile = 128;
constexpr int kAttnThreads = 384;
constexpr int kMaxSeqs = 1024;
constexpr int kQueue = 4, kTileQueue = 8;
constexpr float kGrow = 8.f;  // log2 of the growth of a maximum that rescales O
constexpr int kTileCost = 2;  // fixed cost of a query tile, in key tiles
constexpr int kSplit = kPagedSplit, kQuad = kPagedQuad;

struct Piece {
  int r0, nrows, kvh, n;        // first row, rows, kv head, key tiles (-1: no more pieces)
  int parts;                    // parts of the query tile
  int slot;                     // partial slot: 2 * CTA, + 1 where it is not the CTA's first piece
};

template <int D, int MODE>
struct PagedCfg {
  // tiles of the K ring (2 to 6, see the key tile queue) and of the V ring
  static constexpr int kSTK = D == 128 ? (MODE == kSplit ? 3 : 2) : D == 64 ? 4 : 6;
  static constexpr int kSTV = D == 128 ? 2 : D == 64 ? 4 : 6;
  static constexpr int kBoxD = D >= 64 ? 64 : D;
  static constexpr int kRowBytes = kBoxD * 2;
  static constexpr int kSw = kRowBytes == 128 ? 2 : 4;
  static constexpr int kNBox = D / kBoxD;
  static constexpr int kBoxBytes = 128 * kRowBytes;
  static constexpr int kTile = 128 * D * 2;  // bytes of a Q, K or V tile
  static constexpr int kMerge = MODE == kQuad ? 2 * 128 * (D < 64 ? 16 : 32) * 4 : 0;
  // prefix sums of the units, row and group starts, prefix lengths, group of each
  // sequence
  static constexpr int kPlan = 4 * (kMaxSeqs + 4) * 4 + kMaxSeqs * 2;
  static constexpr int kX = 4096;  // (max, sum) of both streams, for two pieces
  static constexpr int kSpoil = 2 * 128 * (D / 32) * 8;  // column bits of both signs a row
  static constexpr size_t kSmem = 1024 + (1 + kSTK + kSTV) * kTile + kMerge + kPlan + kX + kSpoil +
                                  kQueue * sizeof(Piece) + kTileQueue * 16 + 640;
};

DLLM_DEV int key_tiles(int a, int e) {
  return e > a ? (e + kKeyTile - 1) / kKeyTile - a / kKeyTile : 0;
}
DLLM_DEV int seg_tiles(const Segs& g) { return key_tiles(g.a0, g.e0) + key_tiles(g.a1, g.e1); }

// First position and visible range [lo, hi) of key tile t of the ranges.
DLLM_DEV void key_tile(const Segs& g, int t, int& base, int& lo, int& hi) {
  const int n0 = key_tiles(g.a0, g.e0);
  const int a = t < n0 ? g.a0 : g.a1, e = t < n0 ? g.e0 : g.e1;
  base = (a / kKeyTile + (t < n0 ? t : t - n0)) * kKeyTile;
  lo = max(a, base);
  hi = min(e, base + kKeyTile);
}

DLLM_DEV int prefix_keys(const PagedAttnParams& p, int g) {
  const int cap = p.pmax_pages << p.kv.page_shift;
  const int len = p.plen[g];
  if (len > cap && p.status != nullptr) atomicOr(p.status, kErrIndex);
  return min(max(len, 0), cap);
}

// The line's shares: CTA c of G has units [start(c), start(c + 1)).
struct Shares {
  int each, rem;
  DLLM_DEV int start(int c) const { return c * each + min(c, rem); }
  DLLM_DEV int owner(int u) const {
    const int big = rem * (each + 1);
    return u < big ? (int)((unsigned)u / (unsigned)(each + 1))
                   : rem + (int)((unsigned)(u - big) / (unsigned)each);
  }
};

// A sum of zero is a row without keys; one that is not a number, of a query or key that
// is not finite, stays one.
DLLM_DEV float log_sum(float m, float l) {  // of a maximum in log2 units and a sum
  return l != 0.f ? fmaf(0.6931471805599453f, m, logf(l)) : -INFINITY;
}
DLLM_DEV float inverse_sum(float l) { return l != 0.f ? 1.f / l : 0.f; }

// Transpose of N units of 16 bytes among N neighbouring lanes (N = 2 or 4): after it
// unit i of a lane is unit (lane % N) of the i-th lane of the group.
template <int N>
DLLM_DEV void trade_units(uint4 (&u)[N], int lane) {
#pragma unroll
  for (int o = 1; o < N; o <<= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i & o) continue;
      uint4& a = u[i];
      uint4& b = u[i | o];
      uint4 x = up ? a : b;  // what the partner takes
      x.x = __shfl_xor_sync(0xffffffffu, x.x, o);
      x.y = __shfl_xor_sync(0xffffffffu, x.y, o);
      x.z = __shfl_xor_sync(0xffffffffu, x.z, o);
      x.w = __shfl_xor_sync(0xffffffffu, x.w, o);
      if (up)
        a = x;
      else
        b = x;
    }
  }
}

// A whole warp waits; false when the watchdog gave up.
DLLM_DEV bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort) {
  bool ok = true;
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) {
      ok = false;
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// The wait for copies or products that were issued, in a block that gives up: until they
// are done, or at most kSettleNs.
constexpr unsigned long long kSettleNs = 100000000ull;  // 0.1 s
DLLM_DEV void settle(uint64_t* bar, uint32_t parity) {
  const unsigned long long t0 = global_ns();
  while (!mbar_try_wait(bar, parity) && global_ns() - t0 < kSettleNs) {
  }
  __syncwarp();
}

// Warps meet at a barrier that counts one arrival of each; false when the watchdog
// gave up.  (At a hardware barrier they would wait for warps that have left.)
struct Meeting {
  uint64_t* bar;
  uint32_t parity = 0;
  // (withhold: the self-test's warp that does not arrive)
  DLLM_DEV bool join(int lane, const volatile int* abort, bool withhold = false) {
    __syncwarp();
    if (lane == 0 && !withhold) mbar_arrive(bar);
    const bool ok = warp_wait(bar, parity, abort);
    parity ^= 1;
    return ok;
  }
};

// Pairs of 16-bit elements of which one is not finite get its top bit set: the exponent
// is all ones.
template <bool F16>
DLLM_DEV uint32_t not_finite(uint32_t u) {
  constexpr uint32_t kExp = F16 ? 0x7c007c00u : 0x7f807f80u, kOne = F16 ? 0x04000400u : 0x00800080u;
  return ((u & kExp) + kOne) & 0x80008000u;
}
// What column col of a row gets from the values it saw that were not finite: infinity,
// NaN or nothing (zero), from its bits in n entries of 2 * W words, which are cleared.
template <int W>
DLLM_DEV float spoilt_by(uint32_t* bits, int first, int step, int n, int col) {
  const uint32_t bit = 1u << (col & 31);
  bool sign[2] = {false, false};
#pragma unroll 1
  for (int i = 0; i < n; ++i)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t* b = bits + (first + i * step) * 2 * W + x * W + (col >> 5);
      if (*b & bit) {
        atomicAnd(b, ~bit);
        sign[x] = true;
      }
    }
  return sign[0] && sign[1] ? NAN : sign[0] ? INFINITY : sign[1] ? -INFINITY : 0.f;
}

// Sum over the block's threads before this one (all threads; scratch of one
// entry per warp).
DLLM_DEV int block_before(int v, int* scratch, int warp, int lane) {
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  int before = inc - v;
#pragma unroll
  for (int w = 0; w < kAttnThreads / 32; ++w)
    if (w < warp) before += scratch[w];
  return before;
}

// GROUPS: whether there are shared prefixes (a launch's first pass through its code
// is slow enough for the rest to be left out).
template <int D, bool F16, int MODE, bool GROUPS>
__global__ void __launch_bounds__(kAttnThreads, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ PagedAttnParams p) {
  using C = PagedCfg<D, MODE>;
  constexpr bool QUAD = MODE == kQuad;
  constexpr int STK = C::kSTK, STV = C::kSTV;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base_s = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
  uint8_t* q_s = base_s;
  uint8_t* k_s = q_s + C::kTile;          // [STK]
  uint8_t* v_s = k_s + STK * C::kTile;    // [STV]
  float4* merge_s = reinterpret_cast<float4*>(v_s + STV * C::kTile);  // [2][4][SW / 4][32]
  int* upfx = reinterpret_cast<int*>(v_s + STV * C::kTile + C::kMerge);  // [n_seqs + 1]
  int* rs = upfx + kMaxSeqs + 4;                             // [n_seqs + 1]
  int* gs = rs + kMaxSeqs + 4;                               // [n_groups + 1]
  int* pk = gs + kMaxSeqs + 4;                               // [n_groups]
  short* gid = reinterpret_cast<short*>(pk + kMaxSeqs + 4);  // [n_seqs]
  float* x_s = reinterpret_cast<float*>(gid + kMaxSeqs);
  uint32_t* spoil_s = reinterpret_cast<uint32_t*>(x_s + C::kX / 4);  // [2][128][2 signs][D / 32]
  Piece* queue = reinterpret_cast<Piece*>(x_s + C::kX / 4 + C::kSpoil / 4);
  int4* tiles_s = reinterpret_cast<int4*>(queue + kQueue);
  // whether a stream took notes there, by pieces in turn [4][2 streams]
  int* spoilt_s = reinterpret_cast<int*>(tiles_s + kTileQueue);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(spoilt_s + 8);  // [STK]
  uint64_t* k_empty = k_full + STK;          // [STK]
  uint64_t* v_full = k_empty + STK;          // [STV]
  uint64_t* v_empty = v_full + STV;          // [STV]
  uint64_t* d_full = v_empty + STV;          // [kQueue]
  uint64_t* d_empty = d_full + kQueue;       // [kQueue]
  uint64_t* t_full = d_empty + kQueue;       // [kTileQueue]
  uint64_t* s_full = t_full + kTileQueue;    // [2]
  uint64_t* p_half = s_full + 2;             // [2]
  uint64_t* p_full = p_half + 2;             // [2]
  uint64_t* q_full = p_full + 2;
  uint64_t* q_empty = q_full + 1;
  uint64_t* o_full = q_empty + 1;
  uint64_t* o_empty = o_full + 1;
  uint64_t* meet = o_empty + 1;  // both streams; each one
  uint64_t* done = meet + 3;
  uint64_t* settled = done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(settled + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* progress = abort + 1;
  volatile int* issued_s = progress + 1;  // copies of K, V and Q, when their warps have left

  const int t = threadIdx.x, warp = uniform(t >> 5), lane = t & 31;
  const int tile_rows = p.rows_per_tile;
  if (t == 0) {
    for (int i = 0; i < STK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < STV; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], 9);  // a lane of each warp that reads it
    }
    for (int i = 0; i < kTileQueue; ++i) mbar_init(&t_full[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_half[i], 4);  // a lane of each warp of the stream
      mbar_init(&p_full[i], 4);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(o_full, 1);
    mbar_init(o_empty, 8);
    mbar_init(&meet[0], 8);
    mbar_init(&meet[1], 4);
    mbar_init(&meet[2], 4);
    mbar_init(done, 11);
    mbar_init(settled, 1);
    *abort = 0;
    *progress = 0;
    for (int i = 0; i < 8; ++i) spoilt_s[i] = 0;
    fence_barrier_init();
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  for (int i = t; i < C::kSpoil / 16; i += kAttnThreads)
    reinterpret_cast<uint4*>(spoil_s)[i] = make_uint4(0, 0, 0, 0);
  grid_dep_wait();

  // ---- the line: row starts and groups (made non-decreasing, whatever they
  // hold, so that all CTAs agree on disjoint items), then a prefix sum
  const int n_seqs = p.bt.n_seqs;
  {
    int4 raw = make_int4(0, 0, 0, 0);  // segments of sequence t
    if (t < n_seqs) {
      const int* g = p.segs + 4 * t;
      raw = make_int4(g[0], g[1], g[2], g[3]);
    }
#pragma unroll 1
    for (int i = t; i <= n_seqs; i += kAttnThreads)
      rs[i] = min(max(p.bt.row_start[i], 0), p.bt.n_rows);
    if constexpr (GROUPS) {
#pragma unroll 1
      for (int i = t; i <= p.n_groups; i += kAttnThreads) {
        const int first = p.gseq[i];
        if (i < p.n_groups) pk[i] = prefix_keys(p, i);
        gs[i] = min(max(first, 0), n_seqs);
      }
    }
    __syncthreads();
    bool bad = false;
#pragma unroll 1
    for (int i = t; i < n_seqs; i += kAttnThreads) bad |= rs[i + 1] < rs[i];
    if constexpr (GROUPS) {
#pragma unroll 1
      for (int i = t; i < p.n_groups; i += kAttnThreads) bad |= gs[i + 1] < gs[i];
    }
    if (__syncthreads_or(bad)) {
      if (t == 0) {
#pragma unroll 1
        for (int i = 0; i < n_seqs; ++i) rs[i + 1] = max(rs[i + 1], rs[i]);
        if constexpr (GROUPS) {
#pragma unroll 1
          for (int i = 0; i < p.n_groups; ++i) gs[i + 1] = max(gs[i + 1], gs[i]);
        }
      }
      __syncthreads();
    }
    int* opfx = reinterpret_cast<int*>(k_s);  // own key tiles of earlier sequences
    // v[1 .. n_seqs] becomes its prefix sum, v[0] zero; each thread has a run of it
    const int per = (n_seqs + kAttnThreads - 1) / kAttnThreads;
    auto prefix_sum = [&](int* v, int* scratch) {
      __syncthreads();
      const int i0 = min(t * per, n_seqs), i1 = min(i0 + per, n_seqs);
      int sum = 0;
#pragma unroll 1
      for (int i = i0; i < i1; ++i) sum += v[i + 1];
      int before = block_before(sum, scratch, warp, lane);
#pragma unroll 1
      for (int i = i0; i < i1; ++i) v[i + 1] = before += v[i + 1];
      if (t == 0) v[0] = 0;
    };
    int* scratch = reinterpret_cast<int*>(x_s);
#pragma unroll 1
    for (int i = t; i < n_seqs; i += kAttnThreads) {
      const int kt = seg_tiles(i == t ? make_segs(p, raw.x, raw.y, raw.z, raw.w) : seq_segs(p, i));
      const int rows = rs[i + 1] - rs[i];
      int g = -1;
      if constexpr (GROUPS) {
        int lo = 0, hi = p.n_groups;  // the last group that starts at or before i
#pragma unroll 1
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (gs[mid] <= i)
            lo = mid;
          else
            hi = mid;
        }
        if (gs[lo] <= i && i < gs[lo + 1] && pk[lo] > 0) g = lo;
        gid[i] = (short)g;
        opfx[i + 1] = rows > 0 ? kt * (rows / tile_rows + 1) : 0;
      }
      upfx[i + 1] =
          g < 0 ? (rows + tile_rows - 1) / tile_rows * p.kv.Hkv * (max(kt, 1) + kTileCost) : 0;
    }
    if constexpr (GROUPS) {
      prefix_sum(opfx, scratch + 16);
      __syncthreads();
#pragma unroll 1
      for (int g = t; g < p.n_groups; g += kAttnThreads) {
        const int i = gs[g], e = gs[g + 1];
        const int nt = (rs[e] - rs[i] + tile_rows - 1) / tile_rows;
        if (e > i && nt > 0 && pk[g] > 0)
          upfx[i + 1] = nt * p.kv.Hkv *
                        (key_tiles(0, pk[g]) + (opfx[e] - opfx[i] + nt - 1) / nt + kTileCost);
      }
    }
    prefix_sum(upfx, scratch);
    if constexpr (GROUPS) fence_proxy_async_smem();  // opfx was where K tiles will land
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();
  const uint32_t tmem = uniform(*tmem_slot);

  if (warp == 8 || warp == 10) {
    // ================================================================ producers
    const bool k_side = warp == 8;
    const int U = upfx[n_seqs];
    const int G = min((int)gridDim.x, U);  // CTAs with work
    const int cta = blockIdx.x;
    Shares sh{0, 0};
    int u = 0, u1 = 0;
    if (cta < G) {
      sh.each = (unsigned)U / (unsigned)G;
      sh.rem = U - sh.each * G;
      u = sh.start(cta);
      u1 = sh.start(cta + 1);
    }
    int4 cut = make_int4(0, 0, 0, 0);
    int i = 0, hi = n_seqs;  // the last sequence that starts at or before u
    while (hi - i > 1) {
      const int mid = (i + hi) / 2;
      if (upfx[mid] <= u)
        i = mid;
      else
        hi = mid;
    }
    int n_piece = 0, n_q = 0, n_tile = 0;  // pieces, with keys; key tiles
    int q_issued = 0, issued = 0;          // copies of Q, of key tiles
    uint8_t* ring = k_side ? k_s : v_s;
    uint64_t* full = k_side ? k_full : v_full;
    uint64_t* empty = k_side ? k_empty : v_empty;
    const CUtensorMap* map = k_side ? &kmap : &vmap;
    bool ok = true, first_piece = true;
    const int page_boxes = max(1, kKeyTile >> p.kv.page_shift);
    const int slot_mask = (1 << p.kv.page_shift) - 1;
    const int page_keys = min(kKeyTile, slot_mask + 1);
    while (ok && u < u1) {
      while (u >= upfx[i + 1]) ++i;
      // ---- the query tile at u
      const int g = GROUPS ? gid[i] : -1;
      const int seq_end = g >= 0 ? gs[g + 1] : i + 1;
      const int item_r0 = rs[i], item_r1 = rs[seq_end];
      const int nt = (item_r1 - item_r0 + tile_rows - 1) / tile_rows;
      const int cost = (unsigned)(upfx[i + 1] - upfx[i]) / (unsigned)(nt * p.kv.Hkv);
      const int tile = (unsigned)(u - upfx[i]) / (unsigned)cost;
      const int start = upfx[i] + tile * cost, end = start + cost;
      const int x0 = max(u, start + kTileCost), x1 = min(end, u1);
      u = x1;
      if (x1 <= x0) continue;
      const int kvh = tile / nt;
      const int r0 = item_r0 + (tile - kvh * nt) * tile_rows;
      const int nrows = min(tile_rows, item_r1 - r0);
      int sb = i;  // the sequence of the first row
      if constexpr (GROUPS) {
        for (int e = seq_end; e - sb > 1;) {
          const int mid = (sb + e) / 2;
          if (rs[mid] <= r0)
            sb = mid;
          else
            e = mid;
        }
      }
      // with groups 32 sequences at a time: each lane holds one's segments and tiles
      const int s_first = sb;
      Segs sg{0, 0, 0, 0};
      int kt = 0, incl = 0, own_before = 0;
      auto load_chunk = [&]() {
        const int s = sb + lane;
        sg = Segs{0, 0, 0, 0};
        if (s < seq_end && rs[s + 1] > max(rs[s], r0) && rs[s] < r0 + nrows) sg = seq_segs(p, s);
        kt = seg_tiles(sg);
        incl = kt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += x;
        }
      };
      int own_total;
      if constexpr (GROUPS) {
        load_chunk();
        own_total = __shfl_sync(0xffffffffu, incl, 31);
      } else {
        sg = seq_segs(p, i);
        own_total = seg_tiles(sg);
      }
      // largest and least limit of sequence lim_s in this query tile: a slot beyond the
      // largest is treated like one outside the segments, and may hold anything
      int lim = INT_MAX, lim_lo = INT_MAX, lim_s = s_first;
      auto rows_limit = [&](int a, int b) {  // of the rows from a to b
        int hi = 0, lo = INT_MAX;
#pragma unroll 1
        for (int r = a + lane; r < b; r += 32) {
          const int x = p.row_limit[r];
          hi = max(hi, x);
          lo = min(lo, x);
        }
        lim = __reduce_max_sync(0xffffffffu, hi);
        lim_lo = __reduce_min_sync(0xffffffffu, lo);
      };
      if (p.row_limit != nullptr && rs[s_first + 1] >= r0 + nrows) {
        // all rows of one sequence: its last tiles may be beyond every row's limit
        rows_limit(r0, r0 + nrows);
        Segs s0 = sg;
        if constexpr (GROUPS)
          s0 = Segs{__shfl_sync(0xffffffffu, sg.a0, 0), __shfl_sync(0xffffffffu, sg.e0, 0),
                    __shfl_sync(0xffffffffu, sg.a1, 0), __shfl_sync(0xffffffffu, sg.e1, 0)};
        while (own_total > 0) {
          int kb, kl, kh;
          key_tile(s0, own_total - 1, kb, kl, kh);
          if (kl < lim) break;
          --own_total;
        }
      }
      if constexpr (GROUPS) {
        while (sb + 32 < seq_end && rs[sb + 32] < r0 + nrows) {
          sb += 32;
          load_chunk();
          own_total += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (sb != s_first) {
          sb = s_first;
          load_chunk();
        }
      }
      const int ktp = g >= 0 ? key_tiles(0, pk[g]) : 0;
      const int total = ktp + own_total, allot = cost - kTileCost;
      int k0 = x0 - start - kTileCost, k1 = x1 - start - kTileCost;
      if (total != allot) {
        k0 = (int)((long long)k0 * total / allot);
        k1 = (int)((long long)k1 * total / allot);
      }
      const int n = k1 - k0;

      // ---- its description
      const int qi = n_piece % kQueue;
      if (k_side) {
        ok = n_piece < kQueue ||
             warp_wait(&d_empty[qi], (n_piece / kQueue - 1) & 1, abort);
        if (ok && lane == 0) {
          Piece d{r0, nrows, kvh, n, 1, 2 * cta + (first_piece ? 0 : 1)};
          if (x0 > start + kTileCost || x1 < end) {
            const int first = sh.owner(start + kTileCost);
            d.parts = sh.owner(end - 1) - first + 1;
            if (first == cta) cut = make_int4(r0, nrows | kvh << 12, d.parts, d.slot);  // (lane 0's)
          }
          queue[qi] = d;
          if (p.stall != kStallPiece) mbar_arrive(&d_full[qi]);
        }
      }
      ++n_piece;
      first_piece = false;
      if (!ok || n == 0) continue;

      // ---- its loads
      if (k_side) {
        ok = n_q == 0 || warp_wait(q_empty, (n_q - 1) & 1, abort);
        const int q_row = uniform(r0), q_head = uniform(kvh) * p.G;
        if (ok && elect_one()) {
          constexpr int kCopies = QUAD ? 4 : 1;
          mbar_arrive_expect_tx(q_full,
                                kCopies * C::kNBox * p.G * p.rows_per_tile * C::kRowBytes);
#pragma unroll
          for (int h = 0; h < kCopies; ++h)
#pragma unroll
            for (int b = 0; b < C::kNBox; ++b)
              tma_load_3d(q_s + h * 32 * C::kRowBytes + b * C::kBoxBytes, &qmap, q_full,
                          b * C::kBoxD, q_head, q_row);
        }
        q_issued += ok;
      }
      ++n_q;

      struct Loc {
        int kb, kl, kh, w, page;
      };
      // key tile k of the list, and this lane's page of it (n_pages: nothing to read)
      // c.w: its rows, from | to << 9; whether their limits count (own keys) << 18;
      // whether some of the query tile's rows see keys of it that others do not << 19
      auto locate = [&](int k) {
        Loc c;
        Segs x = sg;
        const int* table = p.bt.table + (size_t)i * p.bt.table_stride;
        int kk = k, own_lim = INT_MAX;
        if constexpr (!GROUPS) {
          c.w = nrows << 9 | 1 << 18;
          own_lim = lim;
        } else if (k < ktp) {
          x = Segs{0, pk[g], 0, 0};
          table = p.ptable + (size_t)g * p.ptable_stride;
          c.w = nrows << 9;
        } else {
          const int o = k - ktp;
          while (o - own_before >= __shfl_sync(0xffffffffu, incl, 31) && sb + 32 < seq_end) {
            own_before += __shfl_sync(0xffffffffu, incl, 31);
            sb += 32;
            load_chunk();
          }
          const int l = __ffs(__ballot_sync(0xffffffffu, incl > o - own_before)) - 1;
          x = Segs{__shfl_sync(0xffffffffu, sg.a0, l), __shfl_sync(0xffffffffu, sg.e0, l),
                   __shfl_sync(0xffffffffu, sg.a1, l), __shfl_sync(0xffffffffu, sg.e1, l)};
          kk = o - own_before - __shfl_sync(0xffffffffu, incl - kt, l);
          const int s = sb + l;
          table = p.bt.table + (size_t)s * p.bt.table_stride;
          const int from = max(rs[s] - r0, 0), to = min(rs[s + 1] - r0, nrows);
          c.w = from | to << 9 | 1 << 18;
          if (p.row_limit != nullptr && (s != lim_s || lim == INT_MAX)) {
            rows_limit(r0 + from, r0 + to);
            lim_s = s;
          }
          own_lim = lim;
          if (to - from < nrows) c.w |= 1 << 19;
        }
        key_tile(x, kk, c.kb, c.kl, c.kh);
        c.kh = min(c.kh, own_lim);
        if ((c.w >> 18 & 1) && lim_lo < c.kh) c.w |= 1 << 19;
        c.page = p.kv.n_pages;
        const int at = c.kb + lane * page_keys;
        if (lane < page_boxes && at < c.kh && at + page_keys > c.kl) {
          c.page = table[at >> p.kv.page_shift];
          if (c.page < 0 || c.page >= p.kv.n_pages) {
            if (p.status != nullptr) atomicOr(p.status, kErrIndex);
            c.page = p.kv.n_pages;
          }
        }
        return c;
      };
      // The description of a key tile goes with its K.  Its slot in the queue is
      // free: the K that had this place, at most 6 tiles ago, has been multiplied,
      // so the softmax is done with the tile two before it.
      Loc c = locate(k0);
      for (int j = 0; ok && j < n; ++j) {
        Loc next = c;
        if (j + 1 < n) next = locate(k0 + j + 1);
        const int ti = n_tile + j;
        const int round = k_side ? ti / STK : ti / STV;
        const int st = uniform(k_side ? ti % STK : ti % STV);
        ok = round == 0 || warp_wait(&empty[st], (round - 1) & 1, abort);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&full[st], C::kTile);
        const int slot = uniform(page_keys == kKeyTile ? c.kb & slot_mask : 0);
        const int head = uniform(kvh);
        uint8_t* dst = ring + st * C::kTile;
#pragma unroll 1
        for (int b = 0; b < page_boxes; ++b) {
          const int page = __shfl_sync(0xffffffffu, c.page, b);
          if (elect_one()) {
#pragma unroll
            for (int x = 0; x < C::kNBox; ++x)
              tma_load_4d(dst + x * C::kBoxBytes, map, &full[st], x * C::kBoxD, slot, head, page);
          }
          dst += page_keys * C::kRowBytes;
        }
        if (k_side && lane == 0) {
          tiles_s[ti % kTileQueue] = make_int4(c.kb, c.kl, c.kh, c.w);
          mbar_arrive(&t_full[ti % kTileQueue]);
        }
        ++issued;
        c = next;
      }
      n_tile += n;
    }
    if (k_side) {
      const int qi = n_piece % kQueue;
      ok = ok && (n_piece < kQueue ||
                  warp_wait(&d_empty[qi], (n_piece / kQueue - 1) & 1, abort));
      if (lane == 0) {
        if (ok) {
          queue[qi].n = -1;
          mbar_arrive(&d_full[qi]);
        }
        p.cut[cta] = cut;
      }
    }
    if (lane == 0) {
      issued_s[k_side ? 0 : 1] = issued;
      if (k_side) issued_s[2] = q_issued;
    }
  } else if (warp == 9) {
    // ================================================================ products
    {
      constexpr uint32_t kIdS = idesc_16(F16, 128, kKeyTile, 0, 0);
      constexpr uint32_t kIdO = idesc_16(F16, 128, D, 0, 1);
      const uint64_t q_desc = smem_desc(smem_u32(q_s), 16, 8 * C::kRowBytes, C::kSw);
      const uint64_t k_desc = smem_desc(smem_u32(k_s), 16, 8 * C::kRowBytes, C::kSw);
      const uint64_t v_desc = smem_desc(smem_u32(v_s), C::kBoxBytes, 8 * C::kRowBytes, C::kSw);
      int n_piece = 0, n_q = 0, n_tile = 0;
      int k_st = 0, v_st = 0;  // places in the rings, and the parities of their barriers
      uint32_t k_ph = 0, v_ph = 0, p_ph = 0;  // (of P: a bit a stream)
      bool ok = true;
      while (ok) {
        const int qi = n_piece % kQueue;
        ok = warp_wait(&d_full[qi], (n_piece / kQueue) & 1, abort);
        if (!ok) break;
        const int n = uniform(queue[qi].n);
        if (elect_one()) mbar_arrive(&d_empty[qi]);
        ++n_piece;
        if (n < 0) break;
        if (n == 0) continue;
        // (one thread) S of the next key tile into stream x; then K, after the last tile
        // Q, is free
        auto s_steps = [&](int x, bool last) {
          const uint64_t kd = k_desc + (uint64_t)(k_st * C::kTile >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            constexpr int kPerBox = C::kBoxD / 16;
            const int off = (kk / kPerBox) * C::kBoxBytes + (kk % kPerBox) * 32;
            umma_bf16(tmem + x * 128, q_desc + (off >> 4), kd + (off >> 4), kIdS, kk > 0);
          }
          umma_commit(&s_full[x]);
          umma_commit(&k_empty[k_st]);
          if (last) umma_commit(q_empty);
        };
        auto next_k = [&]() {
          if (++k_st == STK) {
            k_st = 0;
            k_ph ^= 1;
          }
        };
        // O of stream x with key tile j, then (MORE) S of tile j + 2.  128-key rows have
        // the second half of P ready first: where the whole is not there yet, its
        // products start, and K is waited for, so that the S follows P at once (32
        // blocks 141 -> 135 us).  32-row tiles wait for K behind the product, since
        // there the keys come late (16 sequences' blocks 60.4 the other way, 59.5).
        auto turn = [&](int x, int j, auto more) {
          constexpr bool MORE = decltype(more)::value;
          const uint64_t vd = v_desc + (uint64_t)(v_st * C::kTile >> 4);
          constexpr int kSteps = kKeyTile / 16;
          auto steps = [&](int from, bool acc) {
#pragma unroll
            for (int k = 0; k < kSteps / 2; ++k)
              umma_f16_ts(tmem + 256 + x * 128, tmem + x * 128 + (from + k) * 8,
                          vd + ((from + k) * 16 * C::kRowBytes >> 4), kIdO, acc || k > 0);
          };
          const uint32_t parity = p_ph >> x & 1;
          p_ph ^= 1u << x;
          if (!warp_wait(&v_full[v_st], v_ph, abort)) return false;
          if constexpr (!QUAD) {
            if (!warp_wait(&p_half[x], parity, abort)) return false;
            tc_fence_after();
            if (elect_one()) steps(kSteps / 2, j > 1);
            __syncwarp();
          }
          if (!QUAD && MORE && !warp_wait(&k_full[k_st], k_ph, abort)) return false;
          if (!warp_wait(&p_full[x], parity, abort)) return false;
          tc_fence_after();
          if (elect_one()) {
            if constexpr (QUAD) steps(kSteps / 2, j > 1);
            steps(0, true);
            umma_commit(&v_empty[v_st]);
            if constexpr (!QUAD && MORE) s_steps(x, j + 3 == n);
            *progress = n_tile + j + 1;
          }
          __syncwarp();
          if constexpr (QUAD && MORE) {
            if (!warp_wait(&k_full[k_st], k_ph, abort)) return false;
            if (elect_one()) s_steps(x, j + 3 == n);
            __syncwarp();
          }
          if (++v_st == STV) {
            v_st = 0;
            v_ph ^= 1;
          }
          if constexpr (MORE) next_k();
          return true;
        };
        ok = warp_wait(q_full, n_q & 1, abort);
        if (!ok) break;
        // The streams take turns, from the one that the last piece did not end with.
        const int b = n_tile & 1;
#pragma unroll 1
        for (int j = 0; ok && j < min(n, 2); ++j) {
          ok = warp_wait(&k_full[k_st], k_ph, abort);
          tc_fence_after();
          if (ok && elect_one()) s_steps((b + j) & 1, j + 1 == n);
          __syncwarp();
          next_k();
        }
        if (ok) ok = n_q == 0 || warp_wait(o_empty, (n_q - 1) & 1, abort);
        int j = 0;
#pragma unroll 1
        for (; ok && j + 2 < n; ++j) ok = turn((b + j) & 1, j, std::true_type());
#pragma unroll 1
        for (; ok && j < n; ++j) ok = turn((b + j) & 1, j, std::false_type());
        if (ok && p.stall != kStallProducts && elect_one()) umma_commit(o_full);
        __syncwarp();
        n_tile += n;
        ++n_q;
      }
      if (elect_one()) umma_commit(settled);
    }
  } else if (warp < 8) {
    // ================================================================ softmax
    const int wg = warp >> 2, row = t & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + lane_off + wg * 128;
    const uint32_t o_tm = tmem + lane_off + 256;
    const int qrow = QUAD ? lane : row;  // query row of the tile
    const int rr = qrow / p.G, hh = qrow - rr * p.G;
    const int page_keys = min(kKeyTile, 1 << p.kv.page_shift);
    int n_piece = 0, n_q = 0, s_cnt = 0, n_tile = 0;
    Meeting all{meet}, own_wg{meet + 1 + wg};
    bool ok = true;
    while (ok) {
      const int qi = n_piece % kQueue;
      ok = warp_wait(&d_full[qi], (n_piece / kQueue) & 1, abort);
      if (!ok) break;
      const Piece d{uniform(queue[qi].r0), uniform(queue[qi].nrows), uniform(queue[qi].kvh),
                    uniform(queue[qi].n), uniform(queue[qi].parts), uniform(queue[qi].slot)};
      if (lane == 0) mbar_arrive(&d_empty[qi]);
      ++n_piece;
      if (d.n < 0) break;
      const bool valid = rr < d.nrows;
      const bool active = __any_sync(0xffffffffu, valid);
      const int r = d.r0 + rr;
      // (below zero is as zero, and the differences with positions stay in range)
      const int limit = valid && p.row_limit != nullptr ? max(p.row_limit[r], 0) : INT_MAX;
      float m = -FLT_MAX, l = 0.f;
      // take the new maximum over; O and the sum are rescaled when it grew a lot
      auto grow = [&](bool first, float m_new) {
        if (first) {
          m = m_new;
        } else if (__any_sync(0xffffffffu, valid && m_new > m + kGrow)) {
          // S of this tile is complete, hence also the products before it
          const float alpha = fast_exp2(m - m_new);
          m = m_new;
          l *= alpha;
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            float v[16];
            tmem_ld16(o_tm + wg * 128 + c * 16, v);
            tmem_ld_wait16(v);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] *= alpha;
            tmem_st16(o_tm + wg * 128 + c * 16, v);
          }
        }
      };
      const int j0 = (wg ^ n_tile) & 1;  // the streams take tiles in turn
      for (int j = j0; j < d.n; j += 2) {
        const int ti = n_tile + j;
        ok = warp_wait(&t_full[ti % kTileQueue], (ti / kTileQueue) & 1, abort);
        if (!ok) break;
        const int4 tl = tiles_s[ti % kTileQueue];  // base, lo, hi, rows
        const bool own = tl.w >> 18 & 1, mixed = tl.w >> 19;
        const bool member = valid && rr >= (tl.w & 511) && rr < ((tl.w >> 9) & 511);
        const int first_k = tl.y - tl.x;
        const int end_k = member ? min(tl.z, own ? limit : INT_MAX) - tl.x : 0;
        const bool sees = __any_sync(0xffffffffu, end_k > first_k);
        const bool masked =
            __any_sync(0xffffffffu, valid && (first_k > 0 || end_k < kKeyTile));
        ok = warp_wait(&s_full[wg], s_cnt & 1, abort);
        if (!ok) break;
        ++s_cnt;
        tc_fence_after();
        // Slots of a loaded page outside the tile's range may hold anything,
        // infinities and NaN included: their weight is zero, their values have
        // to be as well.  So do values that are not finite in a mixed tile.  A warp sees
        // to 32 keys.  (S is complete, so the products before it are, and the V tile that
        // had this place had landed: the wait is for this tile's.)  This comes after
        // the first probabilities, since V lands later than K: 32 blocks behind one prefix
        // 134.3 us, and 144.5 with it before the maximum.
        const bool clean = tl.y > tl.x || tl.z < tl.x + kKeyTile || mixed;
        auto clean_values = [&]() {
          const int key = tl.x + row;
          const int pg = key & ~(page_keys - 1);
          constexpr int kUnits = C::kRowBytes / 16;
          uint8_t* v_tile = v_s + (ti % STV) * C::kTile;
          // unit c of box b of a key, where the swizzle has put it
          auto unit = [&](int k, int b, int c) {
            return reinterpret_cast<uint4*>(v_tile + b * C::kBoxBytes + k * C::kRowBytes +
                                            (c ^ (k * C::kRowBytes >> 7 & (kUnits - 1))) * 16);
          };
          if (!warp_wait(&v_full[ti % STV], (ti / STV) & 1, abort)) return false;
          if ((key < tl.y || key >= tl.z) && pg < tl.z && pg + page_keys > tl.y) {
#pragma unroll
            for (int b = 0; b < C::kNBox; ++b)
#pragma unroll 1
              for (int c = 0; c < kUnits; ++c) *unit(row, b, c) = make_uint4(0, 0, 0, 0);
          }
          uint32_t any = 0;
          if (mixed) {
#pragma unroll
            for (int b = 0; b < C::kNBox; ++b)
#pragma unroll
              for (int c = 0; c < kUnits; ++c) {
                const uint4 u = *unit(row, b, c);
                any |= not_finite<F16>(u.x) | not_finite<F16>(u.y) | not_finite<F16>(u.z) |
                       not_finite<F16>(u.w);
              }
          }
          unsigned bad = __ballot_sync(0xffffffffu, any != 0);
          if (bad != 0) {
            constexpr int W = D / 32;
            // the notes of the last piece have been read and cleared
            if (n_q > 0 && !warp_wait(o_empty, (n_q - 1) & 1, abort)) return false;
            if (lane == 0) spoilt_s[(n_q & 3) * 2 + wg] = 1;
#pragma unroll 1
            for (; bad != 0; bad &= bad - 1) {
              const int k = (warp & 3) * 32 + __ffs(bad) - 1;
#pragma unroll 1
              for (int w = 0; w < W; ++w) {  // a lane a column
                const int e = w * 32 + lane;
                const uint32_t u = reinterpret_cast<const uint16_t*>(
                    unit(k, e / C::kBoxD, e % C::kBoxD / 8))[e & 7];
                const bool is = not_finite<F16>(u), nan = u & (F16 ? 0x3ffu : 0x7fu), minus = u >> 15;
                const unsigned pos = __ballot_sync(0xffffffffu, is && (nan || !minus));
                const unsigned neg = __ballot_sync(0xffffffffu, is && (nan || minus));
#pragma unroll 1
                for (int x = lane; x < (QUAD ? 32 : 128); x += 32) {  // the rows that see it
                  const int xr = x / p.G;
                  if (xr >= d.nrows || xr < (tl.w & 511) || xr >= (tl.w >> 9 & 511)) continue;
                  if (own && p.row_limit != nullptr && p.row_limit[d.r0 + xr] <= tl.x + k) continue;
                  uint32_t* note =
                      spoil_s + (wg * 128 + (QUAD ? (warp & 3) * 32 : 0) + x) * 2 * W + w;
                  if (pos != 0) atomicOr(note, pos);
                  if (neg != 0) atomicOr(note + W, neg);
                }
                __syncwarp();
              }
            }
            __syncwarp();
            if (any != 0) {
#pragma unroll 1
              for (int e = 0; e < D; ++e) {
                uint16_t* u =
                    reinterpret_cast<uint16_t*>(unit(row, e / C::kBoxD, e % C::kBoxD / 8)) + (e & 7);
                if (not_finite<F16>(*u)) *u = 0;
              }
            }
          }
          fence_proxy_async_smem();
          return true;
        };
        if (!sees && active) {  // no row of this warp sees the tile
          const float none[16] = {};
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_st16(s_tm + c * 16, none);
        }
        if constexpr (QUAD) {
          const int q0 = (warp & 3) * 32;  // this warp's quarter of the keys
          if (sees) {
            float s[32];
            tmem_ld32(s_tm + q0, s);
            tmem_ld_wait32(s);
            if (masked) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (q0 + i < first_k || q0 + i >= end_k) s[i] = -INFINITY;
            }
            float mx[4] = {-FLT_MAX, -FLT_MAX, -FLT_MAX, -FLT_MAX};
#pragma unroll
            for (int i = 0; i < 32; ++i) mx[i & 3] = fmaxf(mx[i & 3], s[i]);
            const float m_new =
                fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2);
            grow(j == j0, m_new);
            float pk[16], ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float p0 = fast_exp2(fmaf(s[2 * i], p.scale_log2, -m));
              const float p1 = fast_exp2(fmaf(s[2 * i + 1], p.scale_log2, -m));
              ls[i & 3] += p0 + p1;
              pk[i] = __uint_as_float(pack2<F16>(p0, p1));
            }
            l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
            const float none[16] = {};
#pragma unroll
            for (int c = 1; c < 4; ++c) tmem_st16(s_tm + (((warp & 3) + c) & 3) * 16, none);
            tmem_st16(s_tm + (warp & 3) * 16, pk);
          }
          if (clean) {
            ok = clean_values();
            if (!ok) break;
          }
          tmem_st_wait();
        } else {
          // Half of the row stays in registers between the maximum and the
          // probabilities, the other half is read again.
          constexpr int kH = kKeyTile / 2;
          float sa[kH];
          F2 ls[2] = {{0.f, 0.f}, {0.f, 0.f}};
          uint32_t pk[32];
          // P of 64 keys in 32 columns.  (A share of the exponentials as polynomials
          // on the FMA pipe was slower: 161 us for the 32 blocks became 168, 172 and
          // 193 with two, three and four of eight.)
          auto probs = [&](const float (&x)[kH], uint32_t (&pk)[32]) {
#pragma unroll
            for (int i = 0; i < kH; i += 2) {
              F2 e = fma2(F2{x[i], x[i + 1]}, F2{p.scale_log2, p.scale_log2}, F2{-m, -m});
              e = F2{fast_exp2(e.x), fast_exp2(e.y)};
              ls[(i >> 1) & 1] = add2(ls[(i >> 1) & 1], e);
              pk[i / 2] = pack2<F16>(e.x, e.y);
            }
          };
          if (sees) {
            if (masked) {
#pragma unroll 1
              for (int c = 0; c < 4; ++c) {
                float s[32];
                tmem_ld32(s_tm + c * 32, s);
                tmem_ld_wait32(s);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  if (c * 32 + i < first_k || c * 32 + i >= end_k) s[i] = -INFINITY;
                tmem_st32(s_tm + c * 32, reinterpret_cast<const uint32_t*>(s));
              }
              tmem_st_wait();
            }
            float sb[kH];
            float mx[4] = {-FLT_MAX, -FLT_MAX, -FLT_MAX, -FLT_MAX};
            auto maxima = [&](const float (&x)[kH]) {
#pragma unroll
              for (int i = 0; i < kH; i += 2)
                mx[(i >> 1) & 3] = fmaxf(mx[(i >> 1) & 3], fmaxf(x[i], x[i + 1]));
            };
            auto load_half = [&](int h, float (&x)[kH]) {
              tmem_ld32(s_tm + h * kH, x);
              tmem_ld32(s_tm + h * kH + 32, x + 32);
            };
            auto landed = [&](float (&x)[kH]) {
              tmem_ld_wait32(x);
              tmem_ld_wait32(x + 32);
            };
            load_half(0, sa);
            landed(sa);
            load_half(1, sb);
            maxima(sa);
            landed(sb);
            maxima(sb);
            grow(j == j0, fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2));
            load_half(0, sa);
            probs(sb, pk);
            landed(sa);
            tmem_st32(s_tm + 32, pk);
          }
          if (clean) {
            ok = clean_values();
            if (!ok) break;
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_half[wg]);
          if (sees) {
            probs(sa, pk);
            tmem_st32(s_tm, pk);
            l += (ls[0].x + ls[0].y) + (ls[1].x + ls[1].y);
            tmem_st_wait();
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[wg]);
      }
      if (!ok) break;
      // whether each stream had tiles
      const bool some0 = d.n > 1 || (d.n == 1 && (n_tile & 1) == 0);
      const bool some1 = d.n > 1 || (d.n == 1 && (n_tile & 1) == 1);
      n_tile += d.n;
      // ---- the piece's result
      float a0 = 1.f, a1 = 0.f, mt = m, lt = l;
      int spoilt_all = 0;  // a bit for each stream that has notes
      if (d.n > 0) {  // (max, sum) of both streams; each takes half of the columns
        float2* x = reinterpret_cast<float2*>(x_s) + (n_q & 1) * 256;
        x[wg * 128 + row] = make_float2(m, l);
        ok = all.join(lane, abort, p.stall == kStallMeeting && warp == 0);
        if (!ok) break;
        spoilt_all = spoilt_s[(n_q & 3) * 2] | spoilt_s[(n_q & 3) * 2 + 1] << 1;
        // for the next piece but one, which no warp starts before all met for the next
        if ((t & 127) == 0) spoilt_s[((n_q + 2) & 3) * 2 + wg] = 0;
        const float2 y0 = x[row], y1 = x[128 + row];  // a stream without tiles has sum 0
        mt = fmaxf(y0.x, y1.x);
        if constexpr (QUAD) {
#pragma unroll
          for (int k = 1; k < 4; ++k)
            mt = fmaxf(mt, fmaxf(x[(row + 32 * k) & 127].x, x[128 + ((row + 32 * k) & 127)].x));
          lt = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) {  // the same order in every warp
            const float2 y = x[k * 32 + lane];
            lt += y.y * fast_exp2(y.x - mt);
          }
        }
        a0 = fast_exp2(y0.x - mt);
        a1 = fast_exp2(y1.x - mt);
        if constexpr (!QUAD) lt = y0.y * a0 + y1.y * a1;
        ok = warp_wait(o_full, n_q & 1, abort);
        if (!ok) break;
        ++n_q;
        tc_fence_after();
      }
      constexpr int kCols = D / 2;
      constexpr int kC = kCols < 32 ? kCols : 32;
      const int c0 = wg * kCols;
      const int head = d.kvh * p.G + hh;
      // a slot is [D / 4][slot_rows] groups of four elements: neighbouring rows are
      // neighbours, as in the lanes that write them
      float4* part =
          reinterpret_cast<float4*>(p.part) + (size_t)d.slot * p.slot_rows * (D / 4) + qrow;
      const bool whole = d.parts == 1;
      if (whole) {
        const float inv = inverse_sum(lt);
        a0 *= inv;
        a1 *= inv;
      }
      uint16_t* out = static_cast<uint16_t*>(p.out.data) + r * p.out.row_stride +
                      head * p.out.head_stride + c0;
      // over the row's columns from c on that values which are not finite go to
      auto spoil = [&](int c, int n) {
#pragma unroll 1
        for (int col = c; col < c + n; ++col) {
          float v = 0.f;
#pragma unroll 1
          for (int x = 0; x < 2; ++x)
            if (spoilt_all >> x & 1)
              v += spoilt_by<D / 32>(spoil_s, x * 128 + (QUAD ? lane : row), 32, QUAD ? 4 : 1, col);
          if (v == 0.f) continue;
          if (whole)
            out[col - c0] = (uint16_t)pack2<F16>(v, 0.f);
          else
            reinterpret_cast<float*>(part + col / 4 * p.slot_rows)[col & 3] = v;
        }
      };
      if constexpr (QUAD) {
        // each warp brings the sum of its streams for its quarter of the keys; the
        // four are added through shared memory, SW columns at a time, of which
        // each warp finishes SW / 4
        constexpr int SW = kC, kOwn = SW / 4;
        float4* ms = merge_s + wg * (4 * SW / 4 * 32);
#pragma unroll 1
        for (int c = 0; c < kCols / SW; ++c) {
          float v[SW];
#pragma unroll
          for (int i = 0; i < SW; ++i) v[i] = 0.f;
          if (active) {
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
              if (!(x ? some1 : some0)) continue;
              float w[SW];
              const uint32_t at = o_tm + c0 + c * SW + x * 128;
              if constexpr (SW == 32) {
                tmem_ld32(at, w);
                tmem_ld_wait32(w);
              } else {
                tmem_ld16(at, reinterpret_cast<float(&)[16]>(w));
                tmem_ld_wait16(w);
              }
              const float a = x ? a1 : a0;
#pragma unroll
              for (int i = 0; i < SW; ++i) v[i] = fmaf(w[i], a, v[i]);
            }
          }
          if (c == kCols / SW - 1 && d.n > 0 && !spoilt_all) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(o_empty);
          }
          ok = own_wg.join(lane, abort);  // the buffer is free
          if (!ok) break;
#pragma unroll
          for (int k = 0; k < SW / 4; ++k)
            ms[((warp & 3) * (SW / 4) + k) * 32 + lane] =
                make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          ok = own_wg.join(lane, abort);
          if (!ok) break;
          float o[kOwn];
#pragma unroll
          for (int k = 0; k < kOwn / 4; ++k) {
            const int at = ((warp & 3) * (kOwn / 4) + k) * 32 + lane;
            float4 z = ms[at];
#pragma unroll
            for (int w = 1; w < 4; ++w) {
              const float4 y = ms[at + w * (SW / 4) * 32];
              z.x += y.x;
              z.y += y.y;
              z.z += y.z;
              z.w += y.w;
            }
            o[4 * k] = z.x;
            o[4 * k + 1] = z.y;
            o[4 * k + 2] = z.z;
            o[4 * k + 3] = z.w;
          }
          if (valid) {
            const int col = c * SW + (warp & 3) * kOwn;
            if (whole) {
              uint32_t u[kOwn / 2];
#pragma unroll
              for (int i = 0; i < kOwn / 2; ++i) u[i] = pack2<F16>(o[2 * i], o[2 * i + 1]);
              if constexpr (kOwn == 8)
                *reinterpret_cast<uint4*>(out + col) = make_uint4(u[0], u[1], u[2], u[3]);
              else
                *reinterpret_cast<uint2*>(out + col) = make_uint2(u[0], u[1]);
            } else if (d.n > 0) {
#pragma unroll
              for (int i = 0; i < kOwn; i += 4)
                part[(c0 + col + i) / 4 * p.slot_rows] =
                    make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
            if (spoilt_all) spoil(c0 + col, kOwn);
          }
        }
      } else if (active) {
#pragma unroll 1
        for (int c = 0; c < kCols / kC; ++c) {
          float v[kC], w[kC];
          auto add = [&](uint32_t at, float a) {
            if constexpr (kC == 32) {
              tmem_ld32(at, w);
              tmem_ld_wait32(w);
            } else {
              tmem_ld16(at, reinterpret_cast<float(&)[16]>(w));
              tmem_ld_wait16(w);
            }
#pragma unroll
            for (int i = 0; i < kC; ++i) v[i] = fmaf(w[i], a, v[i]);
          };
#pragma unroll
          for (int i = 0; i < kC; ++i) v[i] = 0.f;
          const uint32_t at = o_tm + c0 + c * kC;
          if (some0) add(at, a0);
          if (some1) add(at + 128, a1);
          if (!whole) {
            if (valid && d.n > 0) {
#pragma unroll
              for (int i = 0; i < kC; i += 4)
                part[(c0 + c * kC + i) / 4 * p.slot_rows] =
                    make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
          } else {
            // 16 bytes a row and store would touch 32 lines: four lanes trade
            // their units, so that each store covers 16 * kUnits bytes of a row
            constexpr int kUnits = kC / 8;
            uint4 un[kUnits];
#pragma unroll
            for (int i = 0; i < kUnits; ++i)
              un[i] = make_uint4(pack2<F16>(v[8 * i], v[8 * i + 1]),
                                 pack2<F16>(v[8 * i + 2], v[8 * i + 3]),
                                 pack2<F16>(v[8 * i + 4], v[8 * i + 5]),
                                 pack2<F16>(v[8 * i + 6], v[8 * i + 7]));
            trade_units<kUnits>(un, lane);
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
              const int from = (lane & ~(kUnits - 1)) + i;  // the lane whose row this is
              uint16_t* row_out = reinterpret_cast<uint16_t*>(
                  __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out), from));
              if (__shfl_sync(0xffffffffu, valid, from))
                *reinterpret_cast<uint4*>(row_out + c * kC + (lane & (kUnits - 1)) * 8) = un[i];
            }
          }
        }
      }
      if (!QUAD && spoilt_all) {
        __syncwarp();
        if (valid) spoil(c0, kCols);
      }
      if ((!QUAD && d.n > 0) || spoilt_all) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_empty);
      }
      if (valid && (warp == 0 || (!QUAD && wg == 0))) {
        if (!whole)
          p.part_ml[(size_t)d.slot * p.slot_rows + qrow] = make_float2(mt, d.n > 0 ? lt : -1.f);
        else if (p.lse != nullptr)
          p.lse[(size_t)r * p.Hq + head] = log_sum(mt, lt);
      }
    }
    tmem_st_wait();
  }
  if (warp == 11) {
    // ================================================================ watchdog
    int seen = 0;
    unsigned long long t0 = global_ns();
    while (!mbar_try_wait_sleep(done, 0, 100000u)) {
      const int now = *progress;
      if (now != seen) {
        seen = now;
        t0 = global_ns();
      } else if (!*abort && global_ns() - t0 > p.wait_ns) {
        *abort = 1;
        if (lane == 0 && p.status != nullptr) atomicOr(p.status, kErrTimeout);
      }
    }
    if (*abort) {  // copies and products in flight end before the block goes
      for (int k = max(issued_s[0] - STK, 0); k < issued_s[0]; ++k)
        settle(&k_full[k % STK], (k / STK) & 1);
      for (int k = max(issued_s[1] - STV, 0); k < issued_s[1]; ++k)
        settle(&v_full[k % STV], (k / STV) & 1);
      if (issued_s[2] > 0) settle(q_full, (issued_s[2] - 1) & 1);
      settle(settled, 0);
    }
  } else {
    __syncwarp();
    if (lane == 0) mbar_arrive(done);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ merge
// The cut query tiles of a launch are those that the CTAs recorded.  Every block
// gathers them in shared memory; then all warps of the grid share the work: an item
// is eight elements of 32 rows of a tile (a lane a row, as the parts are stored), and
// where there are fewer items than warps, several warps share an item's parts.  The
// parts of a tile are in the slot of the CTA it starts in and in the even slots of
// the CTAs after it; they are added in that order.  Bound by latency: 4 to 5 us for
// up to 19 MB of parts that are still in L2.  One resident wave of blocks: a grid
// with blocks for every CTA that mostly find nothing took 2 to 5 us more.
constexpr int kMergeWarps = 8, kMergeBlocks = 4 * kNumSMs;

struct RowSum {
  float m = -FLT_MAX, l = 0.f, o[8] = {};
  DLLM_DEV void join(float2 ml, const float4& x, const float4& y) {
    if (ml.y < 0.f) return;  // a part without key tiles, whose elements are not written
    const float mn = fmaxf(m, ml.x);
    const float a = fast_exp2(m - mn), b = fast_exp2(ml.x - mn);
    m = mn;
    l = l * a + ml.y * b;
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * a + v[i] * b;
  }
};

template <int D, bool F16>
__global__ void __launch_bounds__(kMergeWarps * 32, 4)
    paged_merge_kernel(const __grid_constant__ PagedAttnParams p) {
  __shared__ int4 tiles[kNumSMs];  // first row, rows | kv head << 12, parts, first slot
  __shared__ int counts[kMergeWarps];
  __shared__ float2 ml_s[kMergeWarps][32];
  __shared__ float4 o_s[kMergeWarps][2][32];
  static_assert(kNumSMs <= kMergeWarps * 32, "a thread for each record");
  grid_dep_wait();
  grid_dep_launch();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int4 cut = t < kNumSMs ? p.cut[t] : make_int4(0, 0, 0, 0);
  const bool is = cut.z > 1;
  const unsigned mask = __ballot_sync(0xffffffffu, is);
  if (lane == 0) counts[warp] = __popc(mask);
  __syncthreads();
  int before = __popc(mask & ((1u << lane) - 1)), n = 0;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    if (w < warp) before += counts[w];
    n += counts[w];
  }
  if (n == 0) return;
  if (is) tiles[before] = cut;
  __syncthreads();
  const int rows32 = (p.slot_rows + 31) / 32;  // warps for the rows of a tile
  const int per_tile = D / 8 * rows32;
  const int items = n * per_tile, warps = gridDim.x * kMergeWarps;
  const int split = items * 8 <= warps ? 8 : items * 4 <= warps ? 4 : items * 2 <= warps ? 2 : 1;
  const int wpart = warp % split;
  for (int i0 = blockIdx.x * (kMergeWarps / split); i0 < items; i0 += warps / split) {
    const int item = i0 + warp / split;
    const int ti = min(item / per_tile, n - 1), in_tile = item - ti * per_tile;
    const int4 tile = tiles[ti];
    const int col8 = in_tile / rows32;
    const int at = (in_tile - col8 * rows32) * 32 + lane;
    const int rr = at / p.G, hh = at % p.G;
    const bool have = item < items && rr < (tile.y & 0xfff);
    RowSum sum;
    if (have) {
      const float4* part = reinterpret_cast<const float4*>(p.part) + 2 * col8 * p.slot_rows + at;
      constexpr int kUn = 2;
      for (int i = wpart; i < tile.z; i += kUn * split) {
        float2 ml[kUn];
        float4 x[kUn], y[kUn];
#pragma unroll
        for (int k = 0; k < kUn; ++k) {
          const int ip = i + k * split;
          ml[k] = make_float2(-FLT_MAX, -1.f);
          if (ip < tile.z) {
            const size_t ro =
                (size_t)(ip == 0 ? tile.w : (tile.w & ~1) + 2 * ip) * p.slot_rows;
            ml[k] = p.part_ml[ro + at];
            x[k] = part[ro * (D / 4)];
            y[k] = part[ro * (D / 4) + p.slot_rows];
          }
        }
#pragma unroll
        for (int k = 0; k < kUn; ++k) sum.join(ml[k], x[k], y[k]);
      }
    }
    if (split > 1) {  // (then there is one round)
      ml_s[warp][lane] = make_float2(sum.m, sum.l);
      o_s[warp][0][lane] = make_float4(sum.o[0], sum.o[1], sum.o[2], sum.o[3]);
      o_s[warp][1][lane] = make_float4(sum.o[4], sum.o[5], sum.o[6], sum.o[7]);
      __syncthreads();
      if (wpart == 0)
        for (int k = 1; k < split; ++k)
          sum.join(ml_s[warp + k][lane], o_s[warp + k][0][lane], o_s[warp + k][1][lane]);
    }
    if (have && wpart == 0) {
      const float inv = inverse_sum(sum.l);
      const int r = tile.x + rr, head = (tile.y >> 12) * p.G + hh;
      uint16_t* out =
          static_cast<uint16_t*>(p.out.data) + r * p.out.row_stride + head * p.out.head_stride;
      *reinterpret_cast<uint4*>(out + 8 * col8) =
          make_uint4(pack2<F16>(inv * sum.o[0], inv * sum.o[1]),
                     pack2<F16>(inv * sum.o[2], inv * sum.o[3]),
                     pack2<F16>(inv * sum.o[4], inv * sum.o[5]),
                     pack2<F16>(inv * sum.o[6], inv * sum.o[7]));
      if (col8 == 0 && p.lse != nullptr)
        p.lse[(size_t)r * p.Hq + head] = log_sum(sum.m, sum.l);
    }
  }
}

namespace {

template <int D, bool F16, int MODE>
cudaError_t launch_mode(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm,
                        const PagedAttnParams& p, cudaStream_t s) {
  const dim3 grid(kNumSMs), block(kAttnThreads);
  constexpr size_t smem = PagedCfg<D, MODE>::kSmem;
  return p.n_groups > 0 ? launch_pdl(paged_attn_kernel<D, F16, MODE, true>, grid, block, smem, s,
                                     qm, km, vm, p)
                        : launch_pdl(paged_attn_kernel<D, F16, MODE, false>, grid, block, smem,
                                     s, qm, km, vm, p);
}

template <int D, bool F16>
cudaError_t launch_paged_attn_t(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm,
                                const PagedAttnParams& p, int mode, cudaStream_t s) {
  const cudaError_t e = mode == kQuad ? launch_mode<D, F16, kQuad>(qm, km, vm, p, s)
                                      : launch_mode<D, F16, kSplit>(qm, km, vm, p, s);
  if (e != cudaSuccess) return e;
  return launch_pdl(paged_merge_kernel<D, F16>, dim3(kMergeBlocks), dim3(kMergeWarps * 32), 0, s,
                    p);
}

template <int D, bool F16, int MODE>
cudaError_t prepare_mode() {
  static_assert(PagedCfg<D, MODE>::kSmem <= 227 * 1024, "shared memory of a CTA");
  static_assert(PagedCfg<D, MODE>::kSTK >= 2 && PagedCfg<D, MODE>::kSTK <= 6 &&
                    PagedCfg<D, MODE>::kSTV >= 2,
                "see the key tile queue");
  constexpr int smem = (int)PagedCfg<D, MODE>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(paged_attn_kernel<D, F16, MODE, false>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(paged_attn_kernel<D, F16, MODE, true>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

template <int D, bool F16>
cudaError_t prepare_t() {
  cudaError_t e = prepare_mode<D, F16, kSplit>();
  if (e == cudaSuccess) e = prepare_mode<D, F16, kQuad>();
  return e;
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
                              const PagedAttnParams& p, int mode, cudaStream_t s) {
  const int D = p.kv.D;
  if (p.kv.f16)
    return D == 128  ? launch_paged_attn_t<128, true>(qm, km, vm, p, mode, s)
           : D == 64 ? launch_paged_attn_t<64, true>(qm, km, vm, p, mode, s)
                     : launch_paged_attn_t<32, true>(qm, km, vm, p, mode, s);
  return D == 128  ? launch_paged_attn_t<128, false>(qm, km, vm, p, mode, s)
         : D == 64 ? launch_paged_attn_t<64, false>(qm, km, vm, p, mode, s)
                   : launch_paged_attn_t<32, false>(qm, km, vm, p, mode, s);
}

}  // namespace dllm
