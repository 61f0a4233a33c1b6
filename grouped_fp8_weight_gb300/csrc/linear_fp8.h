// Arguments of the experts' forward product (linear_fp8.cu).
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace dg {

constexpr int kMaxExperts = 1024;

struct LinearParams {
  CUtensorMap tm_w;     // w as {K, G N}, boxes of 128 x 128, 128-byte swizzle
  CUtensorMap tm_x;     // x as {K, R}, boxes of 128 x (tokens of a tile)
  CUtensorMap tm_y;     // launch_linear_pair: y as {N, R}, boxes of 64 x 32, 128-byte swizzle
  const float *sx;      // [R, kb]
  const float *sw;      // [G, nb, kb]
  const int *ms;        // [G] rows of each expert
  void *y;              // BF16 [R, N]
  int64_t R;
  int G, N;
  int nb, kb;           // ceil(N / 128), ceil(K / 128)
  DevStatus *status;
  uint64_t wait_limit_ns;
};

// Tokens of a tile for R rows over G experts: 16 or 32 (launch_linear_fp8) or
// 256 (launch_linear_pair).
int linear_tile_tokens(int64_t R, int G, int N, int sms);
// Tiles of `tokens` tokens that any counts summing to R can need, along the tokens.
int64_t linear_max_tiles(int64_t R, int G, int tokens);
cudaError_t launch_linear_fp8(const LinearParams &p, int tokens, int sms, cudaStream_t stream);
// CTA pairs with tiles of up to 256 tokens; tm_x with boxes of 128 x
// linear_pair_x_box().
int linear_pair_x_box();
cudaError_t launch_linear_pair(const LinearParams &p, int sms, cudaStream_t stream);

}  // namespace dg
