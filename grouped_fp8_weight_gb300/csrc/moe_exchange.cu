// Token rows to the experts' slices and back, for sm_103a.
//
//   sort      row(t, j) = off_e + #{pairs before (t, j) routed to the same e},
//             off the exclusive prefix of the counts rounded up to `align`
//   dispatch  xs[row(t, j)] = x[t], zeros in padding rows
//   combine   y[t] = sum_j w[t, j] ye[row(t, j)]   (w absent: plain sum, which
//             is the gradient of dispatch)
//   backward  dye[row(t, j)] = w[t, j] dy[t],  dw[t, j] = <dy[t], ye[row(t, j)]>
//
// An unused pair has row -1: it gives nothing to any sum, and neither its
// weight nor any row is read for it.  Sums are FP32 in the order of j and are
// rounded once to the output type; no atomics touch them.
//
// Bound by memory, each row read and written once: the kernels work token by
// token, so a token's row is loaded once for all its experts.  8192 tokens of
// 7168 BF16 to 8 of 64 experts: dispatch 178 us and combine 154 (99 and 101 %
// of the copy rate), backward 305; the sort takes 13 us, most of it latency.
#include <algorithm>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "per_device.h"
#include "step_ops.h"

namespace dg {

namespace {

// ---------------------------------------------------------------- sort
// A warp owns a chunk of consecutive pairs and one counter per expert in
// shared memory; it walks its pairs 32 at a time in order, and lanes routed to
// the same expert find each other with __match_any_sync and take consecutive
// rows by their rank among those lanes, so rows follow the pair order without
// ordering by atomics.
// Eight groups of 32 pairs are loaded together, so that their latency is paid
// once.
constexpr int kSortUnroll = 8;

// Expert of pair i + 32 u for u = 0 .. 7 (-1 unused, -2 past the end i1).
__device__ __forceinline__ void sort_load(const int *idx, int64_t i, int64_t i1,
                                          int (&e)[kSortUnroll]) {
#pragma unroll
  for (int u = 0; u < kSortUnroll; ++u) e[u] = i + 32 * u < i1 ? idx[i + 32 * u] : -2;
}

__device__ __forceinline__ void sort_count(const int *idx, int64_t i0, int64_t i1, int G, int lane,
                                           int *cnt, DevStatus *status) {
  for (int64_t i = i0 + lane; i < i1; i += 32 * kSortUnroll) {
    int e[kSortUnroll];
    sort_load(idx, i, i1, e);
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) {
      if (i + 32 * u >= i1) break;
      if (e[u] >= 0 && e[u] < G)
        atomicAdd(cnt + e[u], 1);
      else if (e[u] != -1)
        atomicCAS(&status->code, DEV_OK, DEV_BAD_ROUTE);
    }
  }
}

__device__ __forceinline__ void sort_scatter(const MoeSortArgs &a, int64_t i0, int64_t i1, int lane,
                                             int *next) {
  const uint32_t lt = (1u << lane) - 1u;
  for (int64_t s = i0; s < i1; s += 32 * kSortUnroll) {
    int e[kSortUnroll];
    uint32_t peers[kSortUnroll];
    sort_load(a.idx, s + lane, i1, e);
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) {
      if (e[u] < 0 || e[u] >= a.G) e[u] = -1;
      peers[u] = __match_any_sync(0xffffffffu, e[u]);
    }
#pragma unroll
    for (int u = 0; u < kSortUnroll; ++u) {
      const int64_t i = s + 32 * u + lane;
      if (s + 32 * u >= i1) break;           // the whole warp
      int row = -1;
      if (e[u] >= 0) {
        row = next[e[u]] + __popc(peers[u] & lt);
        a.pair_rows[row] = static_cast<int>(i);
        if (a.src_rows != nullptr) a.src_rows[row] = static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(a.topk));
      }
      if (i < i1) a.row_of_pair[i] = row;
      __syncwarp();
      if (e[u] >= 0 && (peers[u] & lt) == 0) next[e[u]] += __popc(peers[u]);
      __syncwarp();
    }
  }
}

// Exclusive prefix over the experts of their padded counts, one or more
// experts per thread (blockDim.x >= 32, G <= 1024).  off[e] is written for
// every e; returns the layout's rows.
__device__ int expert_offsets(const int *total, int G, int align, int *off, int *warp_sum) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int base = 0;
  for (int e0 = 0; e0 < G; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    const int padded = e < G ? (total[e] + align - 1) / align * align : 0;
    int x = padded;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) warp_sum[w] = x;
    __syncthreads();
    int before = base, all = 0;
    const int used = min(nw, (G - e0 + 31) / 32);   // warps with experts
    for (int i = 0; i < used; ++i) {
      const int v = warp_sum[i];
      if (i < w) before += v;
      all += v;
    }
    if (e < G) off[e] = before + x - padded;
    base += all;
    __syncthreads();
  }
  return base;
}

// Padding rows of the slices and the rows past the layout's end.
__device__ __forceinline__ void sort_fill(const MoeSortArgs &a, const int *total, const int *off,
                                          int rows, int first_warp, int n_warps, int lane) {
  for (int e = first_warp; e < a.G && a.align > 1; e += n_warps) {
    const int end = off[e] + (total[e] + a.align - 1) / a.align * a.align;
    for (int r = off[e] + total[e] + lane; r < end; r += 32) {
      a.pair_rows[r] = -1;
      if (a.src_rows != nullptr) a.src_rows[r] = -1;
    }
  }
  for (int64_t r = rows + static_cast<int64_t>(first_warp) * 32 + lane; r < a.cap;
       r += static_cast<int64_t>(n_warps) * 32) {
    a.pair_rows[r] = -1;
    if (a.src_rows != nullptr) a.src_rows[r] = -1;
  }
}

// All pairs in one cluster of up to eight CTAs: a warp owns a contiguous part,
// the CTAs exchange their experts' totals through distributed shared memory.
// On the GPU (us, replayed from a graph; 64 experts, slices of 128), against the
// three launches below: 16384 pairs 7.5 and 12.5, 32768 pairs 10.3 and 13.1,
// 65536 pairs 15.4 and 12.7.  Latency bounds it: 8 pairs of 256 experts
// without padding rows take 2.4, a launch and six barriers.  The cluster is
// widened for the layout's rows too, whose padding it fills: 4096 pairs 9.6 with
// one CTA, 6.0 with four.
constexpr int kSortThreads = 1024;
constexpr int kSortWarpPairs = 128;   // pairs of a warp that a cluster is widened for
constexpr int kSortCluster = 8;
constexpr int64_t kSortFillRows = 4096;   // rows of the layout likewise
constexpr int kSortBatch = 8;         // counters read together
constexpr int64_t kSortOneCluster = 1 << 15;   // pairs

__device__ __forceinline__ int ld_cluster_s32(uint32_t cluster_addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(kSortThreads)
    sort_cluster_kernel(const MoeSortArgs a, int n_warps, int ctas) {
  kernel_begin();
  // counters [n_warps][G], the CTA's totals [G], all totals [G], offsets [G],
  // totals of the CTAs before [G]
  extern __shared__ int sm[];
  __shared__ int warp_sum[32];
  int *own = sm + n_warps * a.G, *total = own + a.G, *off = total + a.G, *first = off + a.G;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = ctas > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  for (int i = threadIdx.x; i < n_warps * a.G; i += blockDim.x) sm[i] = 0;
  __syncthreads();
  const int64_t warps = static_cast<int64_t>(n_warps) * ctas;
  const int64_t per = ((a.n + warps - 1) / warps + 31) / 32 * 32;
  const int64_t i0 = min(a.n, (static_cast<int64_t>(cta) * n_warps + w) * per);
  const int64_t i1 = w < n_warps ? min(a.n, i0 + per) : i0;
  if (w < n_warps) sort_count(a.idx, i0, i1, a.G, lane, sm + w * a.G, a.status);
  __syncthreads();
  for (int e = threadIdx.x; e < a.G; e += blockDim.x) {
    int run = 0;
    for (int i0 = 0; i0 < n_warps; i0 += kSortBatch) {
      int v[kSortBatch];
#pragma unroll
      for (int i = 0; i < kSortBatch; ++i) v[i] = i0 + i < n_warps ? sm[(i0 + i) * a.G + e] : 0;
#pragma unroll
      for (int i = 0; i < kSortBatch; ++i) {
        if (i0 + i < n_warps) sm[(i0 + i) * a.G + e] = run;
        run += v[i];
      }
    }
    own[e] = run;
  }
  if (ctas > 1) cluster_sync(); else __syncthreads();
  for (int e = threadIdx.x; e < a.G; e += blockDim.x) {
    int before = 0, all = 0;
    if (ctas > 1) {
      int v[kSortCluster];
#pragma unroll
      for (int c = 0; c < kSortCluster; ++c)
        v[c] = c < ctas ? ld_cluster_s32(mapa_shared(smem_u32(own + e), c)) : 0;
#pragma unroll
      for (int c = 0; c < kSortCluster; ++c) {
        if (c < cta) before += v[c];
        all += v[c];
      }
    } else {
      all = own[e];
    }
    total[e] = all;
    first[e] = before;
    if (cta == 0) a.counts[e] = (all + a.align - 1) / a.align * a.align;
  }
  if (ctas > 1) cluster_sync(); else __syncthreads();   // nobody reads another CTA's totals any more
  const int rows = expert_offsets(total, a.G, a.align, off, warp_sum);
  if (w < n_warps) {
    for (int e = lane; e < a.G; e += 32) sm[w * a.G + e] += off[e] + first[e];
    __syncwarp();
    sort_scatter(a, i0, i1, lane, sm + w * a.G);
  }
  const int nw = blockDim.x >> 5;
  sort_fill(a, total, off, rows, cta * nw + w, ctas * nw, lane);
}

// More pairs than that: chunks of `per` pairs, one warp each, over the
// whole device in three launches.
constexpr int kSortWarps = 8;         // chunks per CTA
constexpr int kSortMaxChunks = 2048;

int sort_chunk(int64_t n) {
  const int64_t per = (n + kSortMaxChunks - 1) / kSortMaxChunks;
  return static_cast<int>(std::max<int64_t>(512, (per + 31) / 32 * 32));
}

__global__ void __launch_bounds__(kSortWarps * 32)
    sort_count_kernel(const MoeSortArgs a, int per, int n_chunks, int *counts) {
  kernel_begin();
  extern __shared__ int sm[];          // [kSortWarps][G]
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * kSortWarps + w;
  int *cnt = sm + w * a.G;
  if (c >= n_chunks) return;           // whole warps leave together
  for (int e = lane; e < a.G; e += 32) cnt[e] = 0;
  __syncwarp();
  const int64_t i0 = static_cast<int64_t>(c) * per;
  sort_count(a.idx, i0, min(a.n, i0 + per), a.G, lane, cnt, a.status);
  __syncwarp();
  for (int e = lane; e < a.G; e += 32) counts[static_cast<int64_t>(c) * a.G + e] = cnt[e];
}

// 32 experts a CTA: thread (x, y) sums expert x's counts over the y-th part of
// the chunks, the parts are prefixed in shared memory, and each thread then
// replaces its counts by their exclusive prefix.
__global__ void __launch_bounds__(1024)
    sort_scan_kernel(const MoeSortArgs a, int n_chunks, int *counts, int *total) {
  kernel_begin();
  __shared__ int part[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + x;
  const int per = (n_chunks + 31) / 32;
  const int c0 = min(n_chunks, y * per), c1 = min(n_chunks, c0 + per);
  int sum = 0;
  if (e < a.G)
    for (int c = c0; c < c1; ++c) sum += counts[static_cast<int64_t>(c) * a.G + e];
  part[y][x] = sum;
  __syncthreads();
  int run = 0, all = 0;
  for (int i = 0; i < 32; ++i) {
    const int v = part[i][x];
    if (i < y) run += v;
    all += v;
  }
  if (e >= a.G) return;
  for (int c = c0; c < c1; ++c) {
    int *p = counts + static_cast<int64_t>(c) * a.G + e;
    const int v = *p;
    *p = run;
    run += v;
  }
  if (y == 0) {
    total[e] = all;
    a.counts[e] = (all + a.align - 1) / a.align * a.align;
  }
}

__global__ void __launch_bounds__(kSortWarps * 32)
    sort_scatter_kernel(const MoeSortArgs a, int per, int n_chunks, const int *counts,
                        const int *total) {
  kernel_begin();
  extern __shared__ int sm[];          // offsets [G], then [kSortWarps][G]
  __shared__ int warp_sum[32];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = expert_offsets(total, a.G, a.align, sm, warp_sum);
  const int c = blockIdx.x * kSortWarps + w;
  if (c < n_chunks) {
    int *next = sm + (1 + w) * a.G;
    for (int e = lane; e < a.G; e += 32)
      next[e] = sm[e] + counts[static_cast<int64_t>(c) * a.G + e];
    __syncwarp();
    const int64_t i0 = static_cast<int64_t>(c) * per;
    sort_scatter(a, i0, min(a.n, i0 + per), lane, next);
  }
  sort_fill(a, total, sm, rows, c, gridDim.x * kSortWarps, lane);
}

// ---------------------------------------------------------------- rows
// A row is C elements in 16-byte pieces.  `piece` functions work on one piece
// as floats: eight BF16 or four FP32.
template <bool kBf16>
struct Piece {
  static constexpr int N = kBf16 ? 8 : 4;
  static __device__ __forceinline__ void get(const uint4 &v, float (&f)[N]) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kBf16) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      } else {
        f[i] = __uint_as_float(u[i]);
      }
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[N]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kBf16) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t *>(&b);
      } else {
        u[i] = __float_as_uint(f[i]);
      }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};

// Rows of token t's pairs j0 .. j0 + kN - 1, loaded together: negative for an
// unused slot or one past topk.  An index past R counts as unused; true if there
// is one, for the caller to record once its own loads are on their way.
template <int kN>
__device__ __forceinline__ bool load_rows(const MoeMoveArgs &a, int64_t t, int j0, int (&r)[kN]) {
  const int *rows = a.rows + t * a.topk + j0;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kN; ++j) r[j] = j0 + j < a.topk ? rows[j] : -1;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    if (r[j] < a.R) continue;
    bad = true;
    r[j] = -1;
  }
  return bad;
}
__device__ __forceinline__ void record_bad_pair(const MoeMoveArgs &a) {
  atomicCAS(&a.status->code, DEV_OK, DEV_BAD_PAIR);
}

constexpr int kRowThreads = 512;

// Zeros in the rows that no pair owns, one warp per row.
__device__ __forceinline__ void zero_unused_rows(const MoeMoveArgs &a, int pieces, int first_warp,
                                                 int n_warps, int lane) {
  uint4 *out = static_cast<uint4 *>(a.out);
  for (int64_t r = first_warp; r < a.R; r += n_warps) {
    if (a.pairs[r] >= 0) continue;
    for (int c = lane; c < pieces; c += 32) out[r * pieces + c] = make_uint4(0, 0, 0, 0);
  }
}

// Rows of a token loaded together (with 4, tokens to one expert 1.7 % slower; with
// 1, equal within 1 %).
constexpr int kRowsAhead = 2;

__global__ void __launch_bounds__(kRowThreads)
    dispatch_kernel(const MoeMoveArgs a, int pieces, int blocks) {
  kernel_begin();
  const uint4 *x = static_cast<const uint4 *>(a.x);
  uint4 *out = static_cast<uint4 *>(a.out);
  if (static_cast<int>(blockIdx.x) >= blocks) {
    const int w = (blockIdx.x - blocks) * (kRowThreads / 32) + (threadIdx.x >> 5);
    zero_unused_rows(a, pieces, w, (gridDim.x - blocks) * (kRowThreads / 32), threadIdx.x & 31);
    return;
  }
  const int64_t all = a.T * pieces;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; i < all;
       i += static_cast<int64_t>(blocks) * kRowThreads) {
    const int64_t t = i / pieces;
    const int c = static_cast<int>(i - t * pieces);
    const uint4 v = x[i];
    for (int j0 = 0; j0 < a.topk; j0 += kRowsAhead) {
      int r[kRowsAhead];
      const bool bad = load_rows(a, t, j0, r);
#pragma unroll
      for (int j = 0; j < kRowsAhead; ++j)
        if (r[j] >= 0) out[static_cast<int64_t>(r[j]) * pieces + c] = v;
      if (bad) record_bad_pair(a);
    }
  }
}

constexpr int kSlots = 8;   // pairs of a token whose pieces are in flight together

// kPer: pairs in flight together, topk rounded up to a power of two or kSlots:
// slots past topk cost instructions.  Tokens of 1928 BF16 values to 1 and 2
// experts each (35770 of them) take 53 and 64 us, 20000 of 2048 FP32 values to 4
// 117; with kSlots whatever topk is an earlier form took 96, 108 and 139 instead
// of 56, 67 and 118.  CTAs a multiprocessor, same form: with three for one and two
// pairs 65 and 76 us, with two for four 136, with three for eight 477 against 353
// (a training batch's exchange).  No form spills registers: the piece's place is
// stepped along instead of divided out (with a division 12 to 64 bytes spilled).
template <bool kBf16, int kPer>
__global__ void __launch_bounds__(kRowThreads, kPer == 8 ? 2 : kPer == 4 ? 3 : 4)
    combine_kernel(const MoeMoveArgs a, int pieces, int dt, int dc) {
  kernel_begin();
  using P = Piece<kBf16>;
  const uint4 *ye = static_cast<const uint4 *>(a.x);
  // this thread's pieces are a grid apart: dt tokens and dc pieces
  const uint32_t first = blockIdx.x * kRowThreads + threadIdx.x;
  int c = first % pieces;
  for (int64_t t = first / pieces; t < a.T; t += dt) {
    float acc[P::N] = {};
    int j0 = 0;
    do {                                   // once, but for the largest form
      uint4 v[kPer];
      float w[kPer];
      int r[kPer];
      const bool bad = load_rows(a, t, j0, r);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        v[j] = r[j] >= 0 ? ye[static_cast<int64_t>(r[j]) * pieces + c] : make_uint4(0, 0, 0, 0);
        w[j] = r[j] < 0 ? 0.f : a.w != nullptr ? a.w[t * a.topk + j0 + j] : 1.f;
      }
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        float f[P::N];
        P::get(v[j], f);
#pragma unroll
        for (int k = 0; k < P::N; ++k) acc[k] = fmaf(w[j], f[k], acc[k]);
      }
      if (bad) record_bad_pair(a);
      j0 += kPer;
    } while (kPer == kSlots && j0 < a.topk);
    static_cast<uint4 *>(a.out)[t * pieces + c] = P::put(acc);
    if ((c += dc) >= pieces) {
      c -= pieces;
      ++t;
    }
  }
}

// One CTA per token (grid-stride) of up to kTokenThreads (128 against 256 and
// 512: 474, 503, 542 us for a training batch's gradient); each thread keeps its share of the dot
// products of kSlots pairs, which are then added across the CTA in a fixed
// order.  Eight CTAs a multiprocessor (64 registers, no spills) against what
// the compiler takes by itself: 30.9 against 33.1 us for 1021 FP32 tokens of
// 2048 values, 460 against 464 us for the training batch.
constexpr int kTokenThreads = 128;

template <bool kBf16>
__global__ void __launch_bounds__(kTokenThreads, 8)
    combine_backward_kernel(const MoeMoveArgs a, int pieces, int blocks) {
  kernel_begin();
  using P = Piece<kBf16>;
  __shared__ float part[kTokenThreads / 32][kSlots];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if (static_cast<int>(blockIdx.x) >= blocks) {
    zero_unused_rows(a, pieces, (blockIdx.x - blocks) * nw + w, (gridDim.x - blocks) * nw, lane);
    return;
  }
  const uint4 *dy = static_cast<const uint4 *>(a.x), *ye = static_cast<const uint4 *>(a.ye);
  uint4 *dye = static_cast<uint4 *>(a.out);
  for (int64_t t = blockIdx.x; t < a.T; t += blocks) {
    for (int j0 = 0; j0 < a.topk; j0 += kSlots) {
      int row[kSlots];
      float wj[kSlots], dot[kSlots];
      const bool bad = load_rows(a, t, j0, row);
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        wj[j] = row[j] < 0 ? 0.f : a.w[t * a.topk + j0 + j];
        dot[j] = 0.f;
      }
      if (bad) record_bad_pair(a);
      for (int c = threadIdx.x; c < pieces; c += blockDim.x) {
        float g[P::N];
        P::get(dy[t * pieces + c], g);
        uint4 v[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          v[j] = row[j] >= 0 ? ye[static_cast<int64_t>(row[j]) * pieces + c]
                             : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
          if (row[j] < 0) continue;
          float f[P::N], o[P::N];
          P::get(v[j], f);
#pragma unroll
          for (int k = 0; k < P::N; ++k) {
            dot[j] = fmaf(g[k], f[k], dot[j]);
            o[k] = wj[j] * g[k];
          }
          dye[static_cast<int64_t>(row[j]) * pieces + c] = P::put(o);
        }
      }
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
#pragma unroll
        for (int d = 16; d; d >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], d);
        if (lane == 0) part[w][j] = dot[j];
      }
      __syncthreads();
      if (threadIdx.x < kSlots && j0 + static_cast<int>(threadIdx.x) < a.topk) {
        float s = 0.f;
        for (int i = 0; i < nw; ++i) s += part[i][threadIdx.x];
        a.dw[t * a.topk + j0 + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
}

}  // namespace

size_t moe_sort_scratch_bytes(int64_t n, int G) {
  if (n <= kSortOneCluster) return 0;
  const int64_t chunks = (n + sort_chunk(n) - 1) / sort_chunk(n);
  return static_cast<size_t>((chunks + 1) * G) * sizeof(int);
}

cudaError_t launch_moe_sort(const MoeSortArgs &a, cudaStream_t stream) {
  if (a.n <= kSortOneCluster) {
    int ctas = 1;
    while (ctas < kSortCluster && (a.n > 32ll * kSortWarpPairs * ctas || a.cap > kSortFillRows * ctas)) ctas *= 2;
    const int n_warps = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(32, (a.n + 31) / 32)));
    // a whole CTA where slices have padding rows to fill
    const unsigned threads =
        a.align > 1 ? kSortThreads : std::min(kSortThreads, std::max({32 * n_warps, (a.G + 31) / 32 * 32, 128}));
    const size_t smem = static_cast<size_t>(n_warps + 4) * a.G * sizeof(int);
    static OnceOnDevice once;
    const cudaError_t set = once.run([] {
      return cudaFuncSetAttribute(sort_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  36 * 1024 * sizeof(int));
    });
    if (set != cudaSuccess) return set;
    return launch_step(sort_cluster_kernel, ctas, threads, smem, stream, ctas, a, n_warps, ctas);
  }
  const int per = sort_chunk(a.n);
  const int n_chunks = static_cast<int>((a.n + per - 1) / per);
  int *counts = static_cast<int *>(a.scratch), *total = counts + static_cast<int64_t>(n_chunks) * a.G;
  const unsigned blocks = (n_chunks + kSortWarps - 1) / kSortWarps;
  const size_t smem = static_cast<size_t>(kSortWarps) * a.G * sizeof(int);   // <= 32 KB
  cudaError_t e = launch_step(sort_count_kernel, blocks, kSortWarps * 32, smem, stream, 1, a, per,
                              n_chunks, counts);
  if (e == cudaSuccess)
    e = launch_step(sort_scan_kernel, (a.G + 31) / 32, 1024, 0, stream, 1, a, n_chunks, counts, total);
  if (e == cudaSuccess)
    e = launch_step(sort_scatter_kernel, blocks, kSortWarps * 32, smem + a.G * sizeof(int), stream, 1, a,
                    per, n_chunks, counts, total);
  return e;
}

namespace {

// CTAs for `items` CTA-sized items: all of them up to 64 a multiprocessor, so
// that they end evenly (a training batch's exchange: 372 us with 16, 356 with
// 64, 358 with no limit).
int blocks_for(int64_t items, int sms) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(items, 64ll * sms)));
}

}  // namespace

cudaError_t launch_moe_dispatch(const MoeMoveArgs &a, int sms, cudaStream_t stream) {
  const int pieces = a.C / (a.bf16 ? 8 : 4);
  const int blocks = a.T > 0 ? blocks_for((a.T * pieces + kRowThreads - 1) / kRowThreads, sms) : 0;
  const int zero = blocks_for((a.R + kRowThreads / 32 - 1) / (kRowThreads / 32), sms);
  return launch_step(dispatch_kernel, blocks + zero, kRowThreads, 0, stream, 1, a, pieces, blocks);
}

cudaError_t launch_moe_combine(const MoeMoveArgs &a, int sms, cudaStream_t stream) {
  const int pieces = a.C / (a.bf16 ? 8 : 4);
  const int blocks = blocks_for((a.T * pieces + kRowThreads - 1) / kRowThreads, sms);
  const int grid = blocks * kRowThreads;   // threads: below 2^31
  void (*const kernels[4][2])(const MoeMoveArgs, int, int, int) = {
      {combine_kernel<false, 1>, combine_kernel<true, 1>},
      {combine_kernel<false, 2>, combine_kernel<true, 2>},
      {combine_kernel<false, 4>, combine_kernel<true, 4>},
      {combine_kernel<false, kSlots>, combine_kernel<true, kSlots>}};
  const int k = a.topk > 4 ? 3 : a.topk > 2 ? 2 : a.topk > 1 ? 1 : 0;
  return launch_step(kernels[k][a.bf16 ? 1 : 0], blocks, kRowThreads, 0, stream, 1, a, pieces,
                     grid / pieces, grid % pieces);
}

cudaError_t launch_moe_combine_backward(const MoeMoveArgs &a, int sms, cudaStream_t stream) {
  const int pieces = a.C / (a.bf16 ? 8 : 4);
  // as few threads as give every thread the same number of pieces, or one less
  const int iters = (pieces + kTokenThreads - 1) / kTokenThreads;
  const int threads = ((pieces + iters - 1) / iters + 31) / 32 * 32;
  const int blocks = a.T > 0 ? blocks_for(a.T, sms) : 0;
  const int zero = blocks_for((a.R + 7) / 8, sms);
  return launch_step(a.bf16 ? combine_backward_kernel<true> : combine_backward_kernel<false>,
                     blocks + zero, threads, 0, stream, 1, a, pieces, blocks);
}

}  // namespace dg
