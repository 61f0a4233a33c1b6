// Kernel arguments and launchers of the MoE step's operators around the
// GEMMs: tokens to the experts' rows and back (moe_exchange.cu), the row cast
// (quant_rows.cu) and the optimizer (adamw.cu); and the per-device context
// their entry points (step_api.cu) take from api.cu.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "dg_wgrad.h"
#include "ptx.cuh"

namespace dg {

// Device resources of the library on the current device, created on first use.
struct DeviceCtx {
  int sms;
  DevStatus *status;
  cudaMemPool_t pool;
};
dg_status device_ctx(DeviceCtx *out);   // api.cu; sets the thread's message
// A tiled tensor map of `ptr` (api.cu; sets the thread's message).
dg_status encode_map(CUtensorMap *m, CUtensorMapDataType dt, const void *ptr, int rank,
                     const uint64_t *dims, const uint64_t *strides_bytes, const uint32_t *box,
                     CUtensorMapSwizzle sw, CUtensorMapL2promotion l2, const char *what);

// DG_PDL=0 in the environment (read at each call) launches every kernel only
// after the one before it has completed (api.cu).
bool pdl_requested();

// Launches `kernel` as a programmatic dependent: its CTAs may start while the
// kernel before it in the stream is finishing.  Each kernel launched this way
// begins with kernel_begin(), in every thread.  `cluster` CTAs form a cluster.
template <class... P, class... A>
cudaError_t launch_step(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem,
                        cudaStream_t stream, unsigned cluster, const A &...args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_requested() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
#ifdef __CUDACC__
// Lets the next kernel of the stream start as this one ends, and waits until
// the one before has completed and its memory is visible.  What that kernel may
// have written is read with ordinary loads, which stay behind the wait: the
// read-only path (__ldg) is for data that does not change while the kernel
// runs, and this kernel may run while its inputs are being written.
__device__ __forceinline__ void kernel_begin() {
  griddep_launch_dependents();
  griddep_wait();
}
#endif

// ---------------------------------------------------------------- exchange
struct MoeSortArgs {
  const int *idx;      // [n] expert of each pair, -1 unused
  int64_t n;
  int topk, G, align;
  int *counts;         // [G] padded rows of each expert
  int *row_of_pair;    // [n]
  int *pair_rows;      // [cap]
  int *src_rows;       // [cap] or null
  int64_t cap;
  void *scratch;       // moe_sort_scratch_bytes(n, G), null where that is 0
  DevStatus *status;
};
size_t moe_sort_scratch_bytes(int64_t n, int G);
cudaError_t launch_moe_sort(const MoeSortArgs &a, cudaStream_t stream);

// `rows` is row_of_pair [T, topk], `pairs` is pair_rows [R].
struct MoeMoveArgs {
  const void *x;       // dispatch: x [T, C]; combine: ye [R, C]; backward: dy [T, C]
  const void *ye;      // backward: ye [R, C]
  const int *rows, *pairs;
  const float *w;      // [T, topk] or null (combine)
  void *out;           // dispatch: xs [R, C]; combine: y [T, C]; backward: dye [R, C]
  float *dw;           // backward: [T, topk]
  int64_t T, R;
  int topk, C, bf16;   // bf16 0: FP32 rows
  DevStatus *status;
};
cudaError_t launch_moe_dispatch(const MoeMoveArgs &a, int sms, cudaStream_t stream);
cudaError_t launch_moe_combine(const MoeMoveArgs &a, int sms, cudaStream_t stream);
cudaError_t launch_moe_combine_backward(const MoeMoveArgs &a, int sms, cudaStream_t stream);

// ---------------------------------------------------------------- row cast
struct QuantRowsArgs {
  const void *x;             // BF16 [T, C]
  const int *rows, *pairs;   // null: output row t is row t
  uint8_t *q;                // [R, C]
  float *s;                  // [R, ceil(C / 128)]
  int64_t T, R;
  int topk, C;
  DevStatus *status;
};
cudaError_t launch_quant_rows(const QuantRowsArgs &a, int sms, cudaStream_t stream);

// ---------------------------------------------------------------- AdamW
struct AdamwHyper {
  float decay, c1, c2, eps;   // 1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  float b1, a1, b2, a2;       // betas and 1 - beta
  const float *grad_scale;    // device scalar or null
  uint32_t seed;
};
// All tensors of the list with elements; `eight`: 8-bit states.
cudaError_t launch_adamw(const dg_adamw_tensor *list, int n, const AdamwHyper &h, bool eight,
                         bool bf16_grad, int sms, cudaStream_t stream);

}  // namespace dg
