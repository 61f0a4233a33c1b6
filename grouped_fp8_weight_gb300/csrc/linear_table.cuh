// Tiles of the experts' forward product from the counts on the device, shared
// by its two kernels.
#pragma once

#include "linear_fp8.h"

namespace dg {

// Prefix sums over the experts, in shared memory: tile0[e] tiles and row0[e]
// rows before expert e, for e = 0 .. G.
struct LinearTable {
  int *tile0, *row0;
  int G, nt;                  // experts, tiles along N
};
constexpr int kTableBytes = 2 * (kMaxExperts + 4) * 4;

struct LinearTile {
  int expert, n0;             // first row of W_e
  int row, rows;              // first token, tokens
};

// An expert's tiles are kTok tokens by kN columns, n fastest, so that running
// tiles share tokens and one expert's W; the last along the tokens has the rest.
template <int kTok, int kN>
__device__ __forceinline__ LinearTile tile_at(const LinearTable &t, int u) {
  int lo = 0, hi = t.G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.tile0[mid] <= u) lo = mid; else hi = mid - 1;
  }
  const int lt = u - t.tile0[lo], mt = lt / t.nt;
  LinearTile r;
  r.expert = lo;
  r.n0 = (lt - mt * t.nt) * kN;
  r.row = t.row0[lo] + mt * kTok;
  r.rows = min(t.row0[lo + 1] - r.row, kTok);
  return r;
}

// Fills the table (all threads of the CTA, at most 32 warps; scan: 64 numbers of
// shared memory).  Negative counts are none and rows past R belong to nobody;
// both are recorded.
template <int kTok>
__device__ void build_table(const LinearParams &p, const LinearTable &tab, int64_t *scan) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int64_t rows = 0;
  int tiles = 0;
  int64_t *row_sum = scan, *tile_sum = scan + 32;
  bool bad = false;
  for (int e0 = 0; e0 < p.G; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    const int m = e < p.G ? p.ms[e] : 0;
    bad |= m < 0;
    int64_t r = max(m, 0);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, r, d);
      if (lane >= d) r += a;
    }
    if (lane == 31) row_sum[w] = r;
    __syncthreads();
    int64_t all = rows;
    for (int i = 0; i < nw; ++i) {
      if (i == w) r += all;
      all += row_sum[i];
    }
    // clipped to R: what lies past it is left out
    const int end = static_cast<int>(min(r, p.R));
    const int first = static_cast<int>(min(r - max(m, 0), p.R));
    int t = (end - first + kTok - 1) / kTok * tab.nt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, t, d);
      if (lane >= d) t += a;
    }
    if (lane == 31) tile_sum[w] = t;
    __syncthreads();
    int all_t = tiles;
    for (int i = 0; i < nw; ++i) {
      if (i == w) t += all_t;
      all_t += static_cast<int>(tile_sum[i]);
    }
    if (e < p.G) {
      tab.tile0[e + 1] = t;
      tab.row0[e + 1] = end;
    }
    rows = all;
    tiles = all_t;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    tab.tile0[0] = tab.row0[0] = 0;
    bad |= rows > p.R;
  }
  if (bad) atomicCAS(&p.status->code, DEV_OK, DEV_BAD_COUNT);
  __syncthreads();
}

}  // namespace dg
