// Row cast for sm_103a: BF16 rows to E4M3 with one FP32 scale for each 128
// columns, the left operand of the experts' forward product, optionally sent
// to the experts' rows on the way.
//
//   amax = max |x| over the block,  s = max(amax, 2^-100) * (1 / 448)
//   q = E4M3 round-to-nearest-even of x * (1 / s), |.| limited to 448
//
// with 1 / 448 and 1 / s the FP32 numbers nearest to them: each operation is
// one correctly rounded FP32 operation, so the codes are those of the same
// steps anywhere.  The floor keeps 1 / s finite; a block below it loses bits
// gradually, and a padding row is codes 0 with the floor's scale.
//
// Bound by memory: 2 bytes read per element, and 1 + 1/32 written for every
// row the token goes to (16384 tokens of 7168 to 4 of 64 experts 121 us, 97 % of
// the copy rate).  Eight lanes hold a block, sixteen elements (two 16-byte loads)
// each, and reduce its maximum with three shuffles.  The row map is read entry
// by entry: four entries ahead took 39 registers, and 10.0 us against 9.2 for 9000
// tokens of 2048 to one expert.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "step_ops.h"

namespace dg {

namespace {

constexpr int kThreads = 256;
constexpr float kFloor = 0x1p-100f;
constexpr float kInv448 = 1.0f / 448.0f;

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t max_abs(const uint4 &v) {   // pairs of BF16 magnitudes
  // (non-negative BF16 order like their bit patterns)
  return __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                  __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
}
__device__ __forceinline__ uint2 cast8(const uint4 &v, float inv) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = e4m3x2(__fmul_rn(__uint_as_float(u[i] << 16), inv),
                  __fmul_rn(__uint_as_float(u[i] & 0xffff0000u), inv));
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// Item i: 8 lanes on block i % nb of row i / nb.  The first `blocks` CTAs
// cast, the rest (with a row map) write the rows that no pair owns.
__global__ void __launch_bounds__(kThreads)
    quant_rows_kernel(const QuantRowsArgs a, int nb, int blocks) {
  kernel_begin();
  const int l8 = threadIdx.x & 7;
  const uint4 *x = static_cast<const uint4 *>(a.x);
  uint4 *q = reinterpret_cast<uint4 *>(a.q);
  const int pieces = a.C / 16;         // 16-element pieces of a row
  if (static_cast<int>(blockIdx.x) >= blocks) {
    const int lane = threadIdx.x & 31, nw = (gridDim.x - blocks) * (kThreads / 32);
    for (int64_t r = (blockIdx.x - blocks) * (kThreads / 32) + (threadIdx.x >> 5); r < a.R; r += nw) {
      if (a.pairs[r] >= 0) continue;
      for (int c = lane; c < pieces; c += 32) q[r * pieces + c] = make_uint4(0, 0, 0, 0);
      for (int b = lane; b < nb; b += 32) a.s[r * nb + b] = __fmul_rn(kFloor, kInv448);
    }
    return;
  }
  const int64_t all = a.T * nb;
  constexpr int kItems = kThreads / 8;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kItems; i0 < all;
       i0 += static_cast<int64_t>(blocks) * kItems) {
    const int64_t i = i0 + (threadIdx.x >> 3);
    const bool live = i < all;         // all lanes of a warp take part in the shuffles
    const int64_t t = live ? i / nb : 0;
    const int b = static_cast<int>(i - t * nb);
    const int c = b * 8 + l8;
    const bool in = live && c < pieces;
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
    if (in) {
      v0 = x[(t * pieces + c) * 2];
      v1 = x[(t * pieces + c) * 2 + 1];
    }
    uint32_t m = __vmaxu2(max_abs(v0), max_abs(v1));
#pragma unroll
    for (int d = 4; d; d >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float amax = __uint_as_float(max(m & 0xffffu, m >> 16) << 16);
    const float s = __fmul_rn(fmaxf(amax, kFloor), kInv448);
    const float inv = __frcp_rn(s);
    const uint2 lo = cast8(v0, inv), hi = cast8(v1, inv);
    const uint4 code = make_uint4(lo.x, lo.y, hi.x, hi.y);
    if (a.rows == nullptr) {
      if (in) q[t * pieces + c] = code;
      if (live && l8 == 0) a.s[t * nb + b] = s;
      continue;
    }
    if (!live) continue;
    for (int j = 0; j < a.topk; ++j) {
      const int r = a.rows[t * a.topk + j];
      if (r < 0) continue;
      if (r >= a.R) {
        atomicCAS(&a.status->code, DEV_OK, DEV_BAD_PAIR);
        continue;
      }
      if (in) q[static_cast<int64_t>(r) * pieces + c] = code;
      if (l8 == 0) a.s[static_cast<int64_t>(r) * nb + b] = s;
    }
  }
}

}  // namespace

cudaError_t launch_quant_rows(const QuantRowsArgs &a, int sms, cudaStream_t stream) {
  const int nb = (a.C + 127) / 128;
  const auto fit = [&](int64_t n) {
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(n, 16ll * sms)));
  };
  const int blocks = a.T > 0 ? fit((a.T * nb + kThreads / 8 - 1) / (kThreads / 8)) : 0;
  const int zero = a.pairs != nullptr ? fit((a.R + 7) / 8) : 0;
  if (blocks + zero == 0) return cudaSuccess;
  return launch_step(quant_rows_kernel, blocks + zero, kThreads, 0, stream, 1, a, nb, blocks);
}

}  // namespace dg
