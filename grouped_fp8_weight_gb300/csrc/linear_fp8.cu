// The experts' forward product for sm_103a: y[t] = x[t] W_e^T for the rows t
// of expert e, E4M3 operands, x with one FP32 scale per row and 128 columns,
// W_e with one per 128 x 128 block:
//
//   y[t, n] = sum_b sx[t, b] sw[e, n / 128, b] sum_{k in b} x[t, k] w[e, n, k]
//
// FP32 scales are not powers of two, so the tensor core cannot apply them: it
// forms each block's sum over 128 k from zero in tensor memory, and the
// promoting warps read it and add it, scaled, to their FP32 registers.
// The counts stay on the device: every CTA finds its own tile from them.
//
// A tile is 128 rows of W_e (the MMA's M side) by NT tokens (its N side): few
// tokens leave no tensor-core row empty and W, which bounds the product then,
// is read once.  Two CTAs per multiprocessor walk the tiles, each with five
// stages of W in flight, so that one's start and end lie beside the
// other's loads.  Few tiles are shared: with `split` > 1 the CTAs of a cluster
// each take a part of K and one tile, and add their sums up through
// distributed shared memory, every CTA a share of the tokens, in CTA order.
//
// Bound by W's bytes: 8 rows over 64 experts of 4096 x 7168 in 39..41 us (86 to
// 90 % of the copy rate), 1024 rows over 64 of 7168 x 2048 in 148..153 (94 to
// 97 %); one CTA per tile instead of persistent ones took 42 and 193.
//
// Roles: warp 0 TMA producer, warp 1 tensor memory and MMA, warp 2 scale loader
// (cp.async of the tile's sx column of a k-block), warps 4..7 promotion and
// output, one for each 32 tensor-memory lanes.
#include <algorithm>

#include <cuda_bf16.h>

#include "linear_table.cuh"
#include "per_device.h"
#include "step_ops.h"

namespace dg {

namespace {

enum : int { W_PROD_EMPTY = 0x41, W_PROD_DRAIN = 0x42, W_MMA_ACCE = 0x51, W_MMA_FULL = 0x52,
             W_MMA_DRAIN = 0x53, W_PROM_ACCF = 0x61, W_PROM_SX = 0x62, W_SX_EMPTY = 0x71 };

template <int NT>
struct Cfg {
  static constexpr int BK = 128;
  static constexpr int W_BYTES = 128 * BK, X_BYTES = NT * BK;
  static constexpr int STAGES = 5;
  static constexpr int PROM_WARPS = 4;
  static constexpr int THREADS = 128 + 32 * PROM_WARPS;
  static constexpr int ACCS = 4;
  static constexpr int TMEM_COLS = ACCS * NT;              // 64, 128
  static constexpr int SX_SLOTS = 8;
  static constexpr int OFF_X = STAGES * W_BYTES;
  static constexpr int OFF_SX = OFF_X + STAGES * X_BYTES;
  static constexpr int OFF_TAB = OFF_SX + SX_SLOTS * NT * 4;
  static constexpr int OFF_BAR = OFF_TAB + kTableBytes;
  static constexpr int NUM_BARS = 2 * STAGES + 2 * ACCS + 2 * SX_SLOTS + 1;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int SMEM = OFF_MISC + 64 + 1024;
  static_assert(2 * (SMEM + 1024 + 512) <= 233472, "two CTAs per multiprocessor");
  static_assert(NT * 128 * 4 <= OFF_X, "sums to add up lie in the first stages of W");
  static_assert(OFF_BAR % 8 == 0, "barriers");
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}

template <int NT, bool kBrief>
__global__ void __launch_bounds__(Cfg<NT>::THREADS, 2)
    linear_kernel(const __grid_constant__ LinearParams p, int split) {
  using C = Cfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t scan[64];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
  uint64_t *empty = full + C::STAGES;
  uint64_t *accf = empty + C::STAGES;    // block sum ready
  uint64_t *acce = accf + C::ACCS;       // read by every promoting warp
  uint64_t *sxf = acce + C::ACCS;        // scales of a k-block landed
  uint64_t *sxe = sxf + C::SX_SLOTS;
  uint64_t *drain = sxe + C::SX_SLOTS;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
  float *sx_s = reinterpret_cast<float *>(smem + C::OFF_SX);

  // (the broadcast tells the compiler that the number is the warp's)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint64_t lim = p.wait_limit_ns;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < C::ACCS; ++i) {
      mbar_init(&accf[i], 1);
      mbar_init(&acce[i], C::PROM_WARPS);
    }
    for (int i = 0; i < C::SX_SLOTS; ++i) {
      mbar_init(&sxf[i], 32);
      mbar_init(&sxe[i], C::PROM_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  const LinearTable tab{reinterpret_cast<int *>(smem + C::OFF_TAB),
                        reinterpret_cast<int *>(smem + C::OFF_TAB) + kMaxExperts + 4, p.G, p.nb};
  tc_fence_before();
  kernel_begin();                        // nothing before this reads or writes the caller's memory
  build_table<NT>(p, tab, scan);         // synchronises the CTA
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const int n_tiles = tab.tile0[p.G];
  // this CTA's tiles, and its part [k0, k1) of their k-blocks
  const int part = blockIdx.x % split, first = blockIdx.x / split, step = gridDim.x / split;
  const int k0 = p.kb * part / split, k1 = p.kb * (part + 1) / split;

  if (warp == 0) {
    const bool el = elect_one();           // the lane that issues; the loop is the warp's
    if (el) {
      prefetch_tmap(&p.tm_w);
      prefetch_tmap(&p.tm_x);
    }
    const uint64_t keep = l2_policy_evict_last();
    int s = 0;
    uint32_t ph = 0, armed = 0;
    bool ok = true;
    for (int u = first; ok && u < n_tiles; u += step) {
      const LinearTile t = tile_at<NT, 128>(tab, u);
      const int row_w = t.expert * p.N + t.n0;
      for (int j = k0; j < k1; ++j) {
        ok = warp_wait<kBrief>(smem_u32(&empty[s]), ph ^ 1, abort_flag, lim, p.status, W_PROD_EMPTY, u);
        if (!ok) break;
        if (el) {
          mbar_arrive_expect_tx(&full[s], C::W_BYTES + C::X_BYTES);
          tma_load_2d(smem + s * C::W_BYTES, &p.tm_w, &full[s], j * C::BK, row_w);
          tma_load_2d_hint(smem + C::OFF_X + s * C::X_BYTES, &p.tm_x, &full[s], j * C::BK, t.row, keep);
        }
        __syncwarp();
        ++armed;
        if (++s == C::STAGES) { s = 0; ph ^= 1; }
      }
    }
    // every load lands before the CTA can exit
    for (uint32_t i = armed > C::STAGES ? armed - C::STAGES : 0; i < armed; ++i)
      if (!mbar_wait(&full[i % C::STAGES], (i / C::STAGES) & 1, abort_flag, drain_limit_ns(lim),
                     p.status, W_PROD_DRAIN, static_cast<int>(i), false))
        break;
  } else if (warp == 1) {
    const bool el = elect_one();
    constexpr uint32_t idesc = idesc_f8(128, NT);
    const uint64_t w_desc0 = smem_desc(smem_u32(smem), 16, 1024, 2);
    const uint64_t x_desc0 = smem_desc(smem_u32(smem + C::OFF_X), 16, 1024, 2);
    int s = 0, b = 0;
    uint32_t ph = 0, bph = 0;
    bool ok = true;
    for (int u = first; ok && u < n_tiles; u += step) {
      for (int j = k0; j < k1; ++j) {
        ok = warp_wait<kBrief>(smem_u32(&acce[b]), bph ^ 1, abort_flag, lim, p.status, W_MMA_ACCE, u) &&
             warp_wait<kBrief>(smem_u32(&full[s]), ph, abort_flag, lim, p.status, W_MMA_FULL, u);
        if (!ok) break;
        tc_fence_after();
        if (el) {
          const uint64_t wd = w_desc0 + static_cast<uint64_t>(s * (C::W_BYTES >> 4));
          const uint64_t xd = x_desc0 + static_cast<uint64_t>(s * (C::X_BYTES >> 4));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f8(tmem_base + b * NT, wd + 2 * k, xd + 2 * k, idesc, k != 0);
          mma_commit(&empty[s]);
          mma_commit(&accf[b]);
        }
        __syncwarp();
        if (++s == C::STAGES) { s = 0; ph ^= 1; }
        if (++b == C::ACCS) { b = 0; bph ^= 1; }
      }
    }
    // every MMA completes before tensor memory is released
    if (el) mma_commit(drain);
    __syncwarp();
    mbar_wait(drain, 0, abort_flag, drain_limit_ns(lim), p.status, W_MMA_DRAIN, 0, false);
  } else if (warp == 2) {
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int u = first; ok && u < n_tiles; u += step) {
      const LinearTile t = tile_at<NT, 128>(tab, u);
      for (int j = k0; j < k1; ++j) {
        ok = warp_wait<kBrief>(smem_u32(&sxe[s]), ph ^ 1, abort_flag, lim, p.status, W_SX_EMPTY, u);
        if (!ok) break;
#pragma unroll
        for (int i = lane; i < NT; i += 32) {
          const bool live = i < t.rows;
          cp_async4(sx_s + s * NT + i, p.sx + (live ? static_cast<int64_t>(t.row + i) * p.kb + j : 0),
                    live);
        }
        cp_async_arrive(&sxf[s]);
        if (++s == C::SX_SLOTS) { s = 0; ph ^= 1; }
      }
    }
    cp_async_wait_all();
  } else if (warp >= 4) {
    const int quad = warp & 3, n_lane = quad * 32 + lane;
    const uint32_t t_addr = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
    int b = 0, s = 0;
    uint32_t bph = 0, sph = 0;
    bool ok = true;
    for (int u = first; ok && u < n_tiles; u += step) {
      const LinearTile t = tile_at<NT, 128>(tab, u);
      const float *sw = p.sw + (static_cast<int64_t>(t.expert) * p.nb + t.n0 / 128) * p.kb;
      float acc[NT] = {};
      float sw_v = 0.f;
      for (int j = k0; j < k1; ++j) {
        if (((j - k0) & 31) == 0) sw_v = j + lane < k1 ? sw[j + lane] : 0.f;
        const float w = __shfl_sync(0xffffffffu, sw_v, (j - k0) & 31);
        ok = warp_wait<kBrief>(smem_u32(&sxf[s]), sph, abort_flag, lim, p.status, W_PROM_SX, u) &&
             warp_wait<kBrief>(smem_u32(&accf[b]), bph, abort_flag, lim, p.status, W_PROM_ACCF, u);
        if (!ok) break;
        tc_fence_after();
        const float4 *sx4 = reinterpret_cast<const float4 *>(sx_s + s * NT);
        uint32_t r[NT];
        tmem_ld_row<NT>(t_addr + b * NT, r);
        tmem_wait_ld();
        tmem_reg_fence_n<NT>(r);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acce[b]);
#pragma unroll
        for (int i = 0; i < NT; i += 4) {
          const float4 f = sx4[i / 4];
          acc[i] = fmaf(__uint_as_float(r[i]), w * f.x, acc[i]);
          acc[i + 1] = fmaf(__uint_as_float(r[i + 1]), w * f.y, acc[i + 1]);
          acc[i + 2] = fmaf(__uint_as_float(r[i + 2]), w * f.z, acc[i + 2]);
          acc[i + 3] = fmaf(__uint_as_float(r[i + 3]), w * f.w, acc[i + 3]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sxe[s]);
        if (++s == C::SX_SLOTS) { s = 0; sph ^= 1; }
        if (++b == C::ACCS) { b = 0; bph ^= 1; }
      }
      if (!ok) break;
      if (split > 1) {
        // The tile is the CTA's only one: its stages are free for the sums.
        float *mine = reinterpret_cast<float *>(smem) + n_lane;
#pragma unroll
        for (int c = 0; c < NT; ++c) mine[c * 128] = acc[c];
      } else if (t.n0 + n_lane < p.N) {
        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(p.y) + static_cast<int64_t>(t.row) * p.N +
                           t.n0 + n_lane;
#pragma unroll
        for (int c = 0; c < NT; ++c)
          if (c < t.rows) y[static_cast<int64_t>(c) * p.N] = __float2bfloat16_rn(acc[c]);
      }
    }
  }
  tc_fence_before();
  if (split > 1) {
    cluster_sync();                      // every part's sums are in shared memory
    if (warp >= 4 && first < n_tiles && *abort_flag == 0) {
      const LinearTile t = tile_at<NT, 128>(tab, first);
      const int n_lane = threadIdx.x - 128;
      if (t.n0 + n_lane < p.N) {
        __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(p.y) + static_cast<int64_t>(t.row) * p.N +
                           t.n0 + n_lane;
        const uint32_t mine = smem_u32(smem) + 4 * n_lane;
        for (int c = part; c < t.rows; c += split) {
          float sum = 0.f;
          for (int i = 0; i < split; ++i) sum += ld_cluster_f32(mapa_shared(mine + 512 * c, i));
          y[static_cast<int64_t>(c) * p.N] = __float2bfloat16_rn(sum);
        }
      }
    }
    cluster_sync();                      // the others have read this CTA's sums
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

template <int NT, bool kBrief>
cudaError_t launch(const LinearParams &p, int sms, cudaStream_t stream) {
  using C = Cfg<NT>;
  const auto kernel = linear_kernel<NT, kBrief>;
  static OnceOnDevice once;
  const cudaError_t set = once.run([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (set != cudaSuccess) return set;
  const int64_t tiles = linear_max_tiles(p.R, p.G, NT) * p.nb;
  // Measured (us with 1, 2, 4, 8 parts at most): 1 row of 4096 x 7168 20.3, 12.8,
  // 9.6, 7.9; 3 rows of 544 x 7168 19.7, 12.5, 8.4, 6.6; 4 rows of 7168 x 2048
  // 8.4, 7.5, 6.8, 6.8; 1 of 256 x 1024 (two parts of 4 blocks) 5.3, 5.1.
  int split = 1;
  while (split < 8 && tiles * split * 2 <= 2 * sms && p.kb / (2 * split) >= 4) split *= 2;
  // split: one tile per cluster, whatever the counts
  const int64_t grid = split > 1 ? tiles * split : std::min<int64_t>(tiles, 2ll * sms);
  return launch_step(kernel, static_cast<unsigned>(grid), C::THREADS, C::SMEM, stream, split, p,
                     split);
}

}  // namespace

int64_t linear_max_tiles(int64_t R, int G, int tokens) {
  return R / tokens + std::min<int64_t>(R, G);
}

// Measured at 64 experts of 7168 x 2048 with square-root skew and 32 of 4096 x
// 7168 with equal counts (us; 16, 32 and 256 tokens a tile): 4 rows each 145,
// 148, 147 and 142, 143, 148; 16 each 153, 149, 149 and 144, 147, 151; 24 each
// 167, 154, 150 and 165, 147, 152; 64 each 287, 209, 159 and 247, 170, 156.  Few
// pair tiles leave most of the device idle: one expert of 4096 x 7168, 16 of
// them for 76 pairs, takes 19 against 20 us at 64 rows, 24 against 23 at 128 and
// 25 against 27 at 256; one of 7168 x 2048, 28 of them, 9.4 against 9.7, 10.7
// against 10.9 and 16.8 against 12.9.
int linear_tile_tokens(int64_t R, int G, int N, int sms) {
  const int64_t each = (R + G - 1) / G;
  if (each <= 8) return 16;
  if (each <= 24) return 32;
  const int64_t pair_tiles = linear_max_tiles(R, G, 256) * ((N + 255) / 256);
  return each <= 128 && pair_tiles < sms / 4 ? 32 : 256;
}


cudaError_t launch_linear_fp8(const LinearParams &p, int tokens, int sms, cudaStream_t stream) {
  const bool brief = brief_limit(p.wait_limit_ns);
  switch (tokens) {
    case 16: return brief ? launch<16, true>(p, sms, stream) : launch<16, false>(p, sms, stream);
    case 32: return brief ? launch<32, true>(p, sms, stream) : launch<32, false>(p, sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace dg
