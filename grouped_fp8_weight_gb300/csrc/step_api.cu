// C-ABI entry points of the MoE step's operators: argument checks and launches
// for the exchange with the experts, the row cast, the experts' forward
// product and AdamW.
#include <cmath>
#include <cstring>

#include "dg_wgrad.h"
#include "grouped_plan.h"
#include "linear_fp8.h"
#include "step_ops.h"

namespace {

using dg::failf;

dg_status done(const char *fn, cudaError_t e) {
  if (e != cudaSuccess)
    return failf(DG_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
  dg::set_last_error("");
  return DG_OK;
}

bool aligned(const void *p, uintptr_t to = 16) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0;
}

constexpr int64_t kMaxRows = 0x7FFFFF00ll;

// Sizes that the row operators share: T tokens, topk slots, R expert rows of C
// elements (`mult` divides C).
dg_status check_rows(const char *fn, int64_t T, int topk, int64_t R, int C, int mult) {
  if (T < 0 || R < 0 || topk < 1)
    return failf(DG_ERR_INVALID_ARG, "%s: T = %lld, topk = %d, R = %lld", fn, (long long)T, topk,
                 (long long)R);
  if (C <= 0 || C % mult)
    return failf(DG_ERR_INVALID_ARG, "%s: C = %d must be a positive multiple of %d", fn, C, mult);
  if (T > kMaxRows || R > kMaxRows || T > kMaxRows / topk)
    return failf(DG_ERR_UNSUPPORTED, "%s: T * topk or R above 2^31 - 256", fn);
  return DG_OK;
}

dg_status bad_pointers(const char *fn) {
  return failf(DG_ERR_INVALID_ARG, "%s: device pointers must be non-NULL and 16-byte aligned", fn);
}

dg_status bad_dtype(const char *fn, int dt) {
  return failf(DG_ERR_INVALID_ARG, "%s: unknown row dtype %d", fn, dt);
}

dg::MoeMoveArgs move_args(int64_t T, int topk, int64_t R, int C, dg_dtype dtype,
                          const int *row_of_pair, const int *pair_rows) {
  dg::MoeMoveArgs a;
  std::memset(&a, 0, sizeof(a));
  a.T = T;
  a.R = R;
  a.topk = topk;
  a.C = C;
  a.bf16 = dtype == DG_BF16;
  a.rows = row_of_pair;
  a.pairs = pair_rows;
  return a;
}

}  // namespace

extern "C" {

dg_status dg_moe_sort(const int *topk_idx, int64_t T, int topk, int G, int align, int *counts,
                      int *row_of_pair, int *pair_rows, int *src_rows, int64_t cap,
                      dg_stream_t stream) {
  const char *fn = "dg_moe_sort";
  if (T < 0 || topk < 1)
    return failf(DG_ERR_INVALID_ARG, "%s: T = %lld, topk = %d", fn, (long long)T, topk);
  if (G < 1 || G > DG_MAX_GROUPS)
    return failf(G < 1 ? DG_ERR_INVALID_ARG : DG_ERR_UNSUPPORTED, "%s: G = %d (1..%d)", fn, G,
                 DG_MAX_GROUPS);
  if (align < 1 || align > 65536)
    return failf(DG_ERR_INVALID_ARG, "%s: align = %d (1..65536)", fn, align);
  if (T > kMaxRows / topk || T * topk + static_cast<int64_t>(G) * (align - 1) > kMaxRows)
    return failf(DG_ERR_UNSUPPORTED, "%s: layout rows above 2^31 - 256", fn);
  const int64_t n = T * topk, need = n + static_cast<int64_t>(G) * (align - 1);
  if (cap < need)
    return failf(DG_ERR_INVALID_ARG, "%s: cap = %lld < T * topk + G * (align - 1) = %lld", fn,
                 (long long)cap, (long long)need);
  if (!aligned(counts) || (n > 0 && (!aligned(topk_idx) || !aligned(row_of_pair))) ||
      (cap > 0 && !aligned(pair_rows)) || (src_rows != nullptr && !aligned(src_rows)))
    return bad_pointers(fn);
  dg::DeviceCtx dev;
  dg_status s = dg::device_ctx(&dev);
  if (s != DG_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  dg::MoeSortArgs a{topk_idx, n, topk, G, align, counts, row_of_pair, pair_rows, src_rows, cap,
                    nullptr, dev.status};
  const size_t bytes = dg::moe_sort_scratch_bytes(n, G);
  if (bytes > 0) {
    const cudaError_t e = cudaMallocFromPoolAsync(&a.scratch, bytes, dev.pool, st);
    if (e != cudaSuccess) return failf(DG_ERR_CUDA, "%s: scratch: %s", fn, cudaGetErrorString(e));
  }
  const cudaError_t e = dg::launch_moe_sort(a, st);
  if (bytes > 0) cudaFreeAsync(a.scratch, st);   // after the kernels in stream order
  return done(fn, e);
}

dg_status dg_moe_dispatch(const void *x, dg_dtype dtype, int64_t T, int C, int topk,
                          const int *row_of_pair, const int *pair_rows, int64_t R, void *xs,
                          dg_stream_t stream) {
  const char *fn = "dg_moe_dispatch";
  if (dtype != DG_F32 && dtype != DG_BF16) return bad_dtype(fn, dtype);
  dg_status s = check_rows(fn, T, topk, R, C, 8);
  if (s != DG_OK) return s;
  if (R == 0) return done(fn, cudaSuccess);
  if (!aligned(xs) || !aligned(pair_rows) || (T > 0 && (!aligned(x) || !aligned(row_of_pair))))
    return bad_pointers(fn);
  dg::DeviceCtx dev;
  if ((s = dg::device_ctx(&dev)) != DG_OK) return s;
  dg::MoeMoveArgs a = move_args(T, topk, R, C, dtype, row_of_pair, pair_rows);
  a.x = x;
  a.out = xs;
  a.status = dev.status;
  return done(fn, dg::launch_moe_dispatch(a, dev.sms, reinterpret_cast<cudaStream_t>(stream)));
}

dg_status dg_moe_combine(const void *ye, dg_dtype dtype, int64_t R, int C, int64_t T, int topk,
                         const int *row_of_pair, const float *w, void *y, dg_stream_t stream) {
  const char *fn = "dg_moe_combine";
  if (dtype != DG_F32 && dtype != DG_BF16) return bad_dtype(fn, dtype);
  dg_status s = check_rows(fn, T, topk, R, C, 8);
  if (s != DG_OK) return s;
  if (T == 0) return done(fn, cudaSuccess);
  if (!aligned(y) || !aligned(row_of_pair) || (R > 0 && !aligned(ye)) ||
      (w != nullptr && !aligned(w)))
    return bad_pointers(fn);
  dg::DeviceCtx dev;
  if ((s = dg::device_ctx(&dev)) != DG_OK) return s;
  dg::MoeMoveArgs a = move_args(T, topk, R, C, dtype, row_of_pair, nullptr);
  a.x = ye;
  a.w = w;
  a.out = y;
  a.status = dev.status;
  return done(fn, dg::launch_moe_combine(a, dev.sms, reinterpret_cast<cudaStream_t>(stream)));
}

dg_status dg_moe_combine_backward(const void *dy, const void *ye, dg_dtype dtype, int64_t T, int C,
                                  int topk, const int *row_of_pair, const int *pair_rows,
                                  int64_t R, const float *w, void *dye, float *dw,
                                  dg_stream_t stream) {
  const char *fn = "dg_moe_combine_backward";
  if (dtype != DG_F32 && dtype != DG_BF16) return bad_dtype(fn, dtype);
  dg_status s = check_rows(fn, T, topk, R, C, 8);
  if (s != DG_OK) return s;
  if (T == 0 && R == 0) return done(fn, cudaSuccess);
  if ((T > 0 && (!aligned(dy) || !aligned(row_of_pair) || !aligned(w) || !aligned(dw))) ||
      (R > 0 && (!aligned(ye) || !aligned(dye) || !aligned(pair_rows))))
    return bad_pointers(fn);
  dg::DeviceCtx dev;
  if ((s = dg::device_ctx(&dev)) != DG_OK) return s;
  dg::MoeMoveArgs a = move_args(T, topk, R, C, dtype, row_of_pair, pair_rows);
  a.x = dy;
  a.ye = ye;
  a.w = w;
  a.out = dye;
  a.dw = dw;
  a.status = dev.status;
  return done(fn,
              dg::launch_moe_combine_backward(a, dev.sms, reinterpret_cast<cudaStream_t>(stream)));
}

dg_status dg_quant_rows_fp8(const void *x, int64_t T, int C, int topk, const int *row_of_pair,
                            const int *pair_rows, int64_t R, void *q, float *s_out,
                            dg_stream_t stream) {
  const char *fn = "dg_quant_rows_fp8";
  // (an empty map may be NULL: no tokens, or no rows)
  const bool map = row_of_pair != nullptr || pair_rows != nullptr;
  if (map && ((T > 0 && row_of_pair == nullptr) || (R > 0 && pair_rows == nullptr)))
    return failf(DG_ERR_INVALID_ARG, "%s: row_of_pair and pair_rows go together", fn);
  dg_status s = check_rows(fn, T, topk, R, C, 16);
  if (s != DG_OK) return s;
  if (!map && R + T > 0 && (R != T || topk != 1))
    return failf(DG_ERR_INVALID_ARG, "%s: without a row map R must be T and topk 1", fn);
  if (R == 0) return done(fn, cudaSuccess);
  if (!aligned(q) || !aligned(s_out) || (T > 0 && !aligned(x)) ||
      (map && (!aligned(pair_rows) || (T > 0 && !aligned(row_of_pair)))))
    return bad_pointers(fn);
  dg::DeviceCtx dev;
  if ((s = dg::device_ctx(&dev)) != DG_OK) return s;
  dg::QuantRowsArgs a{x, row_of_pair, pair_rows, static_cast<uint8_t *>(q), s_out, T, R, topk, C,
                      dev.status};
  return done(fn, dg::launch_quant_rows(a, dev.sms, reinterpret_cast<cudaStream_t>(stream)));
}

dg_status dg_m_grouped_fp8_linear(const void *x, const float *sx, const void *w, const float *sw,
                                  void *y, int G, int K, int N, int64_t R, const int *ms_dev,
                                  dg_stream_t stream) {
  const char *fn = "dg_m_grouped_fp8_linear";
  if (G < 0) return failf(DG_ERR_INVALID_ARG, "%s: G = %d < 0", fn, G);
  if (G > DG_MAX_GROUPS)
    return failf(DG_ERR_UNSUPPORTED, "%s: G = %d above DG_MAX_GROUPS", fn, G);
  if (K <= 0 || K % 16 || N <= 0 || N % 16)
    return failf(DG_ERR_INVALID_ARG, "%s: K = %d, N = %d must be positive multiples of 16", fn, K, N);
  if (R < 0) return failf(DG_ERR_INVALID_ARG, "%s: R < 0", fn);
  if (G == 0 && R > 0) return failf(DG_ERR_INVALID_ARG, "%s: G = 0 but R = %lld", fn, (long long)R);
  if (R > kMaxRows || static_cast<int64_t>(G) * N > kMaxRows)
    return failf(DG_ERR_UNSUPPORTED, "%s: R or G * N above 2^31 - 256", fn);
  if (R == 0) return done(fn, cudaSuccess);
  if (!aligned(x) || !aligned(sx) || !aligned(w) || !aligned(sw) || !aligned(y) || !aligned(ms_dev))
    return bad_pointers(fn);
  const int nb = (N + 127) / 128;
  if (dg::linear_max_tiles(R, G, 16) * nb > 0x7FFFFFFFll / 8)
    return failf(DG_ERR_UNSUPPORTED, "%s: more than 2^28 - 1 tiles", fn);
  dg::DeviceCtx dev;
  dg_status s = dg::device_ctx(&dev);
  if (s != DG_OK) return s;
  const int tokens = dg::linear_tile_tokens(R, G, N, dev.sms);
  static thread_local dg::LinearParams p;
  p.sx = sx;
  p.sw = sw;
  p.ms = ms_dev;
  p.y = y;
  p.R = R;
  p.G = G;
  p.N = N;
  p.nb = nb;
  p.kb = (K + 127) / 128;
  p.status = dev.status;
  p.wait_limit_ns = dg::wait_limit_ns();
  const uint64_t UK = K, stride[1] = {UK};
  const uint64_t dw[2] = {UK, static_cast<uint64_t>(G) * N}, dx[2] = {UK, static_cast<uint64_t>(R)};
  const bool pair = tokens == 256;
  const uint32_t bw[2] = {128, 128};
  const uint32_t bx[2] = {128, static_cast<uint32_t>(pair ? dg::linear_pair_x_box() : tokens)};
  if ((s = dg::encode_map(&p.tm_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, 2, dw, stride, bw,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, "w")) ||
      (s = dg::encode_map(&p.tm_x, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, 2, dx, stride, bx,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, "x")))
    return s;
  if (pair) {
    const uint64_t dy[2] = {static_cast<uint64_t>(N), static_cast<uint64_t>(R)}, ys[1] = {2ull * N};
    const uint32_t by[2] = {64, 32};
    if ((s = dg::encode_map(&p.tm_y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, 2, dy, ys, by,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, "y")))
      return s;
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return done(fn, pair ? dg::launch_linear_pair(p, dev.sms, st) : dg::launch_linear_fp8(p, tokens, dev.sms, st));
}

dg_status dg_adamw_step(const dg_adamw_tensor *tensors, int n, dg_dtype grad_dtype, int state_bits,
                        int64_t step, double lr, double beta1, double beta2, double eps,
                        double weight_decay, const float *grad_scale, uint64_t seed,
                        dg_stream_t stream) {
  const char *fn = "dg_adamw_step";
  if (n < 0 || (n > 0 && tensors == nullptr))
    return failf(DG_ERR_INVALID_ARG, "%s: n = %d tensors", fn, n);
  if (grad_dtype != DG_F32 && grad_dtype != DG_BF16)
    return failf(DG_ERR_INVALID_ARG, "%s: unknown gradient dtype %d", fn, (int)grad_dtype);
  if (state_bits != 8 && state_bits != 32)
    return failf(DG_ERR_INVALID_ARG, "%s: state_bits = %d (8 or 32)", fn, state_bits);
  if (step < 1) return failf(DG_ERR_INVALID_ARG, "%s: step = %lld < 1", fn, (long long)step);
  if (!(beta1 >= 0 && beta1 < 1 && beta2 >= 0 && beta2 < 1))
    return failf(DG_ERR_INVALID_ARG, "%s: betas %g, %g must lie in [0, 1)", fn, beta1, beta2);
  if (!(eps >= 0) || !std::isfinite(eps) || !std::isfinite(lr) || !std::isfinite(weight_decay))
    return failf(DG_ERR_INVALID_ARG, "%s: lr, eps and weight_decay must be finite, eps >= 0", fn);
  if (grad_scale != nullptr && !aligned(grad_scale, 4))
    return failf(DG_ERR_INVALID_ARG, "%s: grad_scale must be 4-byte aligned", fn);
  for (int i = 0; i < n; ++i) {
    const dg_adamw_tensor &t = tensors[i];
    if (t.n < 0 || t.n > (1ll << 40))
      return failf(DG_ERR_INVALID_ARG, "%s: tensor %d has %lld elements", fn, i, (long long)t.n);
    if (t.n == 0) continue;
    if (!aligned(t.p) || !aligned(t.g) || !aligned(t.m) || !aligned(t.v) ||
        (t.copy != nullptr && !aligned(t.copy)))
      return failf(DG_ERR_INVALID_ARG,
                   "%s: tensor %d: p, g, m, v (and copy) must be non-NULL and 16-byte aligned", fn, i);
    if ((state_bits == 8) != (t.sm != nullptr) || (state_bits == 8) != (t.sv != nullptr))
      return failf(DG_ERR_INVALID_ARG, "%s: tensor %d: scales sm and sv go with 8-bit states", fn, i);
  }
  dg::DeviceCtx dev;
  dg_status s = dg::device_ctx(&dev);
  if (s != DG_OK) return s;
  dg::AdamwHyper h;
  h.decay = static_cast<float>(1.0 - lr * weight_decay);
  h.c1 = static_cast<float>(lr / (1.0 - std::pow(beta1, static_cast<double>(step))));
  h.c2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, static_cast<double>(step))));
  h.eps = static_cast<float>(eps);
  h.b1 = static_cast<float>(beta1);
  h.a1 = static_cast<float>(1.0 - beta1);
  h.b2 = static_cast<float>(beta2);
  h.a2 = static_cast<float>(1.0 - beta2);
  h.grad_scale = grad_scale;
  h.seed = static_cast<uint32_t>(seed ^ (seed >> 32));
  return done(fn, dg::launch_adamw(tensors, n, h, state_bits == 8, grad_dtype == DG_BF16, dev.sms,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
