// The experts' forward product (see linear_fp8.cu) for many tokens per expert,
// run by persistent CTA pairs with the 2-SM tensor-core MMA.
//
// An expert's tokens are cut into tiles of 256 and a rest, each against 256
// rows of W_e.  A full tile has its tokens on the MMA's M side (128 per CTA)
// and the rows of W_e on its N side (each CTA stages 128 of them).  A rest of
// up to 160 has them the other way round: with the tokens on the N side, which
// goes in steps of 32, a ragged expert costs what its tokens cost.
//
// Per 128-k block the tensor core forms the tile's sums from zero in one of
// two tensor-memory buffers, and the eight promoting warps of each CTA add
// them, scaled, to FP32 registers (128 sums a thread) while the next block's
// MMAs run.  Two loader warps write the scales sx[t, b] sw[e, n / 128, b] to
// shared memory, four k-blocks at a time.  In a full tile a thread holds 128
// columns of one token: one scale per thread and k-block, and the reads of
// tensor memory (16 columns at a time) follow one another without a gap.  In a
// rest tile a thread holds pairs of tokens of two rows (the 16-lane read), so
// that it reads each scale pair once for four sums.
//
// Measured: 32768 rows over 32 skewed experts, 4096 x 7168, in 722 us (50 calls
// in a row; 2665 TFLOP/s, 76 % of the dense FP8 rate that cuBLASLt reaches here)
// before the power cap, 809 us (2378 TFLOP/s) in a row of 6000 at a median of 1627
// MHz under it (1366 of 1400 W); 714 to 830 us by box and length of the row.  A
// k-block of a full tile takes 804 cycles, 512 of them MMAs; loads and scales are always there.  What
// bounds it is the promoting warps' way round a buffer: 147 cycles until they
// have seen its sums (57 % of the time these are there before them), 367 until
// they have read them, 84 for the last sums, 40 for the output spread over 56
// blocks; the MMA warp waits for the buffer six times out of seven.  Without
// the promotion's sums and reads (a copy) the rest takes 617 cycles.
//
// What did not help: single CTAs of 128 x 256 with the N side multicast to both
// (893 against 850 us: 96 KB through one shared memory for each block instead of
// 64); 256 columns as two halves with barriers of their own (992, N = 128 MMAs
// read the M side twice as often); three buffers of 160 columns (1100) or four
// of 128 (more hand-overs; for rests, which would leave room for four, 1 % at
// 128 tokens and 9 % more time at 96); sixteen promoting warps (1127);
// packed FP32 pairs (1169 against 1088, a register move for each); the 16-lane
// read for all tiles (985: 524 cycles for the 128 lanes x 256 columns that the
// 32-lane read takes 137 for); the next block's first read begun ahead of the
// last sums (860 against 772); reads of 32 columns (784).
//
// Roles per CTA (384 threads, their registers split 208 : 88): warps 0..7
// promotion and output, warp w on tensor-memory lanes 32 (w % 4) and, in full
// tiles, columns 128 (w / 4) on, in rest tiles every other 32-token chunk;
// warp 8 TMA; warp 9 tensor memory and (even CTA) MMA; warps 10, 11 scales.
// Output: BF16 through shared memory; 32 tokens of one expert leave by bulk tensor
// stores of 64 columns (790 us with 64-byte pieces of rows from the threads'
// registers), a group with fewer, and a rest, in 64-byte pieces of rows.
#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>

#include "linear_table.cuh"
#include "per_device.h"
#include "step_ops.h"

namespace dg {

namespace {

enum : int { W_PROD_EMPTY = 0x81, W_PROD_DRAIN = 0x82, W_MMA_ACCE = 0x91, W_MMA_FULL = 0x92,
             W_MMA_DRAIN = 0x93, W_PROM_ACCF = 0xa1, W_PROM_S = 0xa2, W_S_EMPTY = 0xb1 };

constexpr int kStages = 5;
constexpr int kTok = 256;                     // tokens of a full tile
constexpr int kPromWarps = 8;
constexpr int kThreads = 32 * (kPromWarps + 4);
constexpr int kWBytes = 128 * 128;            // this CTA's rows of W, and
constexpr int kXBytes = 128 * 128;            // its half of the tokens
constexpr int kXBox = 64;                     // tokens of one x box
constexpr int kGroups = 3;                    // scale slots, four k-blocks each
constexpr int kGroupBytes = 4 * kTok * 4;
constexpr int kStgPitch = 80;                 // bytes of a staged token: 32 rows of W and a gap
constexpr int kStgBytes = 32 * 128;           // per promoting warp: 32 tokens of 64 columns
constexpr int OFF_X = kStages * kWBytes;
constexpr int OFF_S = OFF_X + kStages * kXBytes;
constexpr int OFF_STG = OFF_S + kGroups * kGroupBytes;
constexpr int OFF_TAB = OFF_STG + kPromWarps * kStgBytes;
constexpr int OFF_BAR = OFF_TAB + kTableBytes;
constexpr int kBars = 2 * kStages + 4 + 2 * kGroups + 1;
// bytes from accf to sf and se (accf and acce, two each, come before)
constexpr int kToSf = 4 * 8, kToSe = kToSf + kGroups * 8;
constexpr int OFF_MISC = OFF_BAR + kBars * 8;
constexpr int kSmem = OFF_MISC + 64 + 1024;
static_assert(kSmem <= 232448, "shared memory");
static_assert(OFF_BAR % 8 == 0 && OFF_STG % 1024 == 0, "barriers, swizzled buffers");
static_assert(kWBytes == kXBytes, "the operands' buffers change roles");

struct Tile : LinearTile {
  int n;                      // a rest: rows rounded up to 32 (MMA N); a full tile: 0
};
// A rest of more rows runs as a full tile with empty rows: 32 experts of 192 rows
// (4096 x 7168) take 191 us so and 195 as rests; of 160 rows 190 and 178.
constexpr int kMaxRest = 160;
__device__ __forceinline__ Tile pair_tile(const LinearTable &t, int u) {
  Tile r;
  static_cast<LinearTile &>(r) = tile_at<kTok, 256>(t, u);
  r.n = r.rows > kMaxRest ? 0 : (r.rows + 31) & ~31;
  return r;
}

// A promoting warp.
template <bool kBrief>
struct Promoter {
  const LinearParams &p;
  uint32_t smem, bars;          // shared addresses: the buffers, and accf[0]
  volatile int *abort_flag;
  uint32_t tmem, acce0;         // its lanes of tensor memory; the even CTA's acce[0]
  int quad, cg, rank;           // lane quadrant, column half or first chunk
  uint32_t phase;               // bits 0, 1: of accf; from 2: of sf
  uint32_t slot;                // scale slot in use

  __device__ __forceinline__ int lane() const { return threadIdx.x & 31; }

  __device__ __forceinline__ bool sums_ready(int buf, int u) {
    if (!warp_wait<kBrief>(bars + 8 * buf, (phase >> buf) & 1, abort_flag, p.wait_limit_ns, p.status,
                   W_PROM_ACCF, u))
      return false;
    phase ^= 1u << buf;
    tc_fence_after();
    return true;
  }
  __device__ __forceinline__ void release(int buf) {
    tc_fence_before();
    __syncwarp();
    if (lane() == 0) mbar_arrive_remote(acce0 + 8 * buf);
  }

  // Runs f(address of a k-block's scales) over the tile's k-blocks: block0 for
  // even ones, block1 for odd ones.
  template <class F0, class F1>
  __device__ __forceinline__ bool k_loop(int u, F0 &&block0, F1 &&block1) {
    const int kb = p.kb;
    for (int j = 0; j < kb; j += 4) {
      if (!warp_wait<kBrief>(bars + kToSf + 8 * slot, (phase >> (2 + slot)) & 1, abort_flag, p.wait_limit_ns,
                     p.status, W_PROM_S, u))
        return false;
      phase ^= 4u << slot;
      uint32_t s = smem + OFF_S + slot * kGroupBytes;
      const int end = min(j + 4, kb);
      for (int i = j; i < end; i += 2, s += 8 * kTok) {
        if (!block0(s)) return false;
        if (i + 1 < end && !block1(s + 4 * kTok)) return false;
      }
      __syncwarp();
      if (lane() == 0) mbar_arrive_addr(bars + kToSe + 8 * slot);
      slot = slot + 1 == kGroups ? 0 : slot + 1;
    }
    return true;
  }

  // ---- full tile: this thread's token, columns 128 cg .. 128 cg + 127
  template <int kBuf>
  __device__ __forceinline__ bool full_block(float (&acc)[4][32], uint32_t s, int u) {
    if (!sums_ready(kBuf, u)) return false;
    const uint32_t t0 = tmem + kBuf * kTok + cg * 128;
    uint32_t r[2][16];               // one read in flight while the one before is added
    tmem_ld_32x32b_x16(t0, r[0]);
    const float f = ld_shared_f32(s + 4 * threadIdx.x);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      tmem_wait_ld();
      tmem_reg_fence16(r[c & 1]);
      if (c < 7) tmem_ld_32x32b_x16(t0 + (c + 1) * 16, r[(c + 1) & 1]);
      else release(kBuf);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        acc[c / 2][16 * (c & 1) + i] = fmaf(__uint_as_float(r[c & 1][i]), f, acc[c / 2][16 * (c & 1) + i]);
    }
    return true;
  }
  __device__ __forceinline__ bool full_tile(const Tile &t, int u) {
    float acc[4][32];
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[c][i] = 0.f;
    if (!k_loop(u, [&](uint32_t s) { return full_block<0>(acc, s, u); },
                [&](uint32_t s) { return full_block<1>(acc, s, u); }))
      return false;
    const int ln = lane(), n = t.n0 + cg * 128, tok = rank * 128 + quad * 32, left = t.rows - tok;
    if (left >= 32) {            // 32 tokens of this expert: two stores of 64 columns
      const uint32_t put = staging() + ln * 128;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t m[32];          // rounded while the first half is being read
#pragma unroll
        for (int i = 0; i < 32; ++i)
          m[i] = bf16_pair(acc[2 * h + i / 16][2 * (i & 15)], acc[2 * h + i / 16][2 * (i & 15) + 1]);
        staging_free();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_shared_v4(put + 16 * ((i ^ ln) & 7), m[4 * i], m[4 * i + 1], m[4 * i + 2], m[4 * i + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (ln == 0) {
          if (n + 64 * h < p.N) tma_store_2d(&p.tm_y, staging(), n + 64 * h, t.row + tok);
          bulk_commit();
        }
      }
      return true;
    }
    staging_free();
    const uint32_t put = staging() + ln * kStgPitch;
    __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(p.y) + static_cast<int64_t>(t.row + tok) * p.N + n;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t m[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = bf16_pair(acc[c][8 * i + 2 * k], acc[c][8 * i + 2 * k + 1]);
        st_shared_v4(put + 16 * i, m[0], m[1], m[2], m[3]);
      }
      store_chunk(y + 32 * c, left, p.N - n - 32 * c);
    }
    return true;
  }

  // ---- rest tile: 32 rows of W, this warp's kNC 32-token chunks
  template <int kNC, int kBuf>
  __device__ __forceinline__ bool rest_block(float (&acc)[kNC > 0 ? kNC : 1][32], uint32_t s, int u) {
    if (!sums_ready(kBuf, u)) return false;
    // 16 lanes of a chunk at a time; the next read, and the next chunk's
    // scales, are on their way while one is added
    const uint32_t t0 = tmem + kBuf * kTok + cg * 32;
    uint32_t r[2][16];
    float2 f[2][4];
    if constexpr (kNC > 0) {
      tmem_ld_16x256b_x4(t0, r[0]);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[0][i] = ld_shared_f32x2(s + 32 * i);
    }
#pragma unroll
    for (int c = 0; c < kNC; ++c) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        tmem_wait_ld();
        tmem_reg_fence16(r[h]);
        if (h == 0) tmem_ld_16x256b_x4(t0 + (16u << 16) + c * 64, r[1]);
        else if (c + 1 < kNC) tmem_ld_16x256b_x4(t0 + (c + 1) * 64, r[0]);
        else release(kBuf);
        if (h == 0 && c + 1 < kNC) {
#pragma unroll
          for (int i = 0; i < 4; ++i) f[(c + 1) & 1][i] = ld_shared_f32x2(s + 256 * (c + 1) + 32 * i);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            acc[c][8 * i + 4 * h + k] =
                fmaf(__uint_as_float(r[h][4 * i + k]), (k & 1) ? f[c & 1][i].y : f[c & 1][i].x,
                     acc[c][8 * i + 4 * h + k]);
      }
    }
    if constexpr (kNC == 0) release(kBuf);
    return true;
  }
  // The number of chunks is a constant: with a run-time number the sums moved
  // between registers around every branch.
  template <int kNC>
  __device__ __forceinline__ bool rest_tile(const Tile &t, int u) {
    float acc[kNC > 0 ? kNC : 1][32];              // [chunk][token group, 16-lane half, row, token]
#pragma unroll
    for (int c = 0; c < kNC; ++c)
#pragma unroll
      for (int i = 0; i < 32; ++i) acc[c][i] = 0.f;
    const uint32_t mine = 8 * (threadIdx.x & 3) + 128 * cg;
    if (!k_loop(u, [&](uint32_t s) { return rest_block<kNC, 0>(acc, s + mine, u); },
                [&](uint32_t s) { return rest_block<kNC, 1>(acc, s + mine, u); }))
      return false;
    const int ln = lane(), n = t.n0 + rank * 128 + quad * 32;
    const uint32_t put = staging() + (ln & 7) * kStgPitch + (ln >> 3) * 16;
    staging_free();
    __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(p.y) + static_cast<int64_t>(t.row) * p.N + n;
#pragma unroll
    for (int c = 0; c < kNC; ++c) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {                // tokens 8 i .. 8 i + 7 of the chunk
        uint32_t m[4];                             // rows of W in groups of eight
#pragma unroll
        for (int k = 0; k < 4; ++k) m[k] = bf16_pair(acc[c][8 * i + 2 * k], acc[c][8 * i + 2 * k + 1]);
        stmatrix_x4_trans(put + 8 * i * kStgPitch, m[0], m[1], m[2], m[3]);
      }
      const int tok = (2 * c + cg) * 32;
      store_chunk(y + static_cast<int64_t>(tok) * p.N, t.rows - tok, p.N - n);
    }
    return true;
  }

  // ---- output
  __device__ __forceinline__ uint32_t staging() const { return smem + OFF_STG + (4 * cg + quad) * kStgBytes; }
  static __device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&x);
  }
  // This warp's buffer once its last stores have read it.
  __device__ __forceinline__ void staging_free() const {
    if (lane() == 0) bulk_wait_read<0>();
    __syncwarp();
  }
  // The staged 32 tokens x 32 columns to y (its first element), at most `toks`
  // tokens and `cols` columns (a multiple of 16).
  __device__ __forceinline__ void store_chunk(__nv_bfloat16 *y, int toks, int cols) {
    __syncwarp();
    const int ln = lane(), c = (ln & 3) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = 8 * i + (ln >> 2);
      const uint4 x = ld_shared_v4(staging() + tok * kStgPitch + 2 * c);
      if (tok < toks && c < cols) *reinterpret_cast<uint4 *>(y + static_cast<int64_t>(tok) * p.N + c) = x;
    }
    __syncwarp();
  }
};

template <bool kBrief>
__global__ void __launch_bounds__(kThreads, 1)
    linear_pair_kernel(const __grid_constant__ LinearParams p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int64_t scan[64];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + OFF_BAR);   // even CTA: both CTAs' bytes
  uint64_t *empty = full + kStages;       // consumed by the pair's MMAs
  uint64_t *accf = empty + kStages;       // block sums ready (both CTAs)
  uint64_t *acce = accf + 2;              // even CTA: read by both CTAs' promoting warps
  uint64_t *sf = acce + 2;                // scales of four k-blocks written
  uint64_t *se = sf + kGroups;
  uint64_t *drain = se + kGroups;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + OFF_MISC);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + OFF_MISC + 4);

  // (the broadcast tells the compiler that the number is the warp's)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint64_t lim = p.wait_limit_ns;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pid = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int kb = p.kb;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&accf[i], 1);
      mbar_init(&acce[i], 2 * kPromWarps);
    }
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&sf[i], 2);
      mbar_init(&se[i], kPromWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kPromWarps + 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  const LinearTable tab{reinterpret_cast<int *>(smem + OFF_TAB),
                        reinterpret_cast<int *>(smem + OFF_TAB) + kMaxExperts + 4, p.G, (p.N + 255) / 256};
  kernel_begin();                   // nothing before this reads or writes the caller's memory
  build_table<kTok>(p, tab, scan);
  const int n_tiles = tab.tile0[p.G];
  tc_fence_before();
  cluster_sync();                   // both CTAs' barriers are initialised
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);

  if (warp < kPromWarps) {
    regs_inc<208>();   // 256 x 208 + 128 x 88 = the launch's 384 x 168
    Promoter<kBrief> w{p, smem_u32(smem), smem_u32(accf), abort_flag,
               tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16),
               mapa_shared(smem_u32(&acce[0]), 0), warp & 3, warp >> 2, static_cast<int>(rank), 0, 0};
    bool ok = true;
    for (int u = pid; ok && u < n_tiles; u += pairs) {
      const Tile t = pair_tile(tab, u);
      if (t.n == 0) {
        ok = w.full_tile(t, u);
        continue;
      }
      switch ((t.n / 32 + 1 - (warp >> 2)) / 2) {  // this warp's chunks: every other one
        case 0: ok = w.rest_tile<0>(t, u); break;
        case 1: ok = w.rest_tile<1>(t, u); break;
        case 2: ok = w.rest_tile<2>(t, u); break;
        default: ok = w.rest_tile<3>(t, u); break;
      }
    }
    if (lane == 0) bulk_wait<0>();   // the stores have left shared memory
  } else {
    regs_dec<88>();
    if (warp == kPromWarps) {
      // The whole warp runs the loop and one lane issues.  With one lane in the
      // loop a k-block's loads took 525 cycles to issue whatever their size, and
      // the MMAs of small rests waited for them (617 cycles a block against 503).
      const bool el = elect_one();
      const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0), empty0 = smem_u32(empty);
      if (el) {
        prefetch_tmap(&p.tm_w);
        prefetch_tmap(&p.tm_x);
        prefetch_tmap(&p.tm_y);
      }
      const uint64_t keep = l2_policy_evict_last();
      int s = 0;
      uint32_t ph = 0, armed = 0;
      bool ok = true;
      for (int u = pid; ok && u < n_tiles; u += pairs) {
        const Tile t = pair_tile(tab, u);
        const int share = t.n == 0 ? 128 : t.n / 2;      // this CTA's tokens
        const int boxes = share > kXBox ? 2 : 1;
        const uint32_t tx = 2 * (kWBytes + boxes * kXBox * 128);
        const int row_w = t.expert * p.N + t.n0 + static_cast<int>(rank) * 128;
        const int row_x = t.row + static_cast<int>(rank) * share;
        for (int j = 0; j < kb; ++j) {
          ok = warp_wait<kBrief>(empty0 + 8 * s, ph ^ 1, abort_flag, lim, p.status, W_PROD_EMPTY, u);
          if (!ok) break;
          if (el) {
            if (leader) mbar_arrive_expect_tx(&full[s], tx);
            uint8_t *sx = smem + OFF_X + s * kXBytes;
            tma_load_2d_pair(smem + s * kWBytes, &p.tm_w, full0 + 8 * s, j * 128, row_w, keep);
            tma_load_2d_pair(sx, &p.tm_x, full0 + 8 * s, j * 128, row_x, keep);
            if (boxes == 2)
              tma_load_2d_pair(sx + kXBox * 128, &p.tm_x, full0 + 8 * s, j * 128, row_x + kXBox, keep);
          }
          __syncwarp();
          ++armed;
          if (++s == kStages) { s = 0; ph ^= 1; }
        }
      }
      // Every load of this CTA lands before the pair can exit: the even CTA
      // sees them on `full`, its partner sees the stages released.
      for (uint32_t i = armed > kStages ? armed - kStages : 0; i < armed; ++i) {
        uint64_t *b = leader ? &full[i % kStages] : &empty[i % kStages];
        if (!mbar_wait(b, (i / kStages) & 1, abort_flag, drain_limit_ns(lim), p.status,
                       W_PROD_DRAIN, static_cast<int>(i), false))
          break;
      }
    }
    if (warp == kPromWarps + 1 && leader) {
      const bool el = elect_one();
      const uint64_t w_desc0 = smem_desc(smem_u32(smem), 16, 1024, 2);
      const uint64_t x_desc0 = smem_desc(smem_u32(smem + OFF_X), 16, 1024, 2);
      int s = 0;
      uint32_t ph = 0, aph = 3;                    // phases of full; bits of acce (first pass: free)
      const uint32_t full0 = smem_u32(full), acce0 = smem_u32(acce);
      bool ok = true;
      for (int u = pid; ok && u < n_tiles; u += pairs) {
        const Tile t = pair_tile(tab, u);
        // (the broadcasts tell the compiler that these are the warp's, which
        // keeps them in uniform registers for the MMAs)
        const uint32_t n = t.n == 0 ? 256 : t.n;
        const uint32_t idesc = __shfl_sync(0xffffffffu, idesc_f8(256, 0) | (n >> 3) << 17, 0);
        const bool turned = __shfl_sync(0xffffffffu, t.n, 0) != 0;
        const uint64_t a0 = turned ? w_desc0 : x_desc0, b0 = turned ? x_desc0 : w_desc0;
        // A k-block, its sums into buffer kBuf.  Half of acce's arrivals are the
        // partner's: behind them lie its tensor-memory reads and no memory that
        // anyone writes, so the waits' CTA scope is enough (cluster scope for
        // this wait 723 us against 714, for all of them 766, and with arrivals
        // released at cluster scope too 1716).
        auto block = [&](auto buf_c) {
          constexpr int kBuf = decltype(buf_c)::value;
          if (!warp_wait<kBrief>(full0 + 8 * s, ph, abort_flag, lim, p.status, W_MMA_FULL, u) ||
              !warp_wait<kBrief>(acce0 + 8 * kBuf, (aph >> kBuf) & 1, abort_flag, lim, p.status, W_MMA_ACCE, u))
            return false;
          aph ^= 1u << kBuf;
          tc_fence_after();
          const uint64_t ad = a0 + static_cast<uint64_t>(s * (kWBytes >> 4));
          const uint64_t bd = b0 + static_cast<uint64_t>(s * (kWBytes >> 4));
          if (el) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f8_pair(tmem_base + kBuf * kTok, ad + 2 * k, bd + 2 * k, idesc, k != 0);
            mma_commit_pair(&accf[kBuf], 0x3);
            mma_commit_pair(&empty[s], 0x3);
          }
          __syncwarp();
          if (++s == kStages) { s = 0; ph ^= 1; }
          return true;
        };
        // every tile starts on buffer 0
        for (int j = 0; ok && j < kb; j += 2) {
          ok = block(std::integral_constant<int, 0>{});
          if (ok && j + 1 < kb) ok = block(std::integral_constant<int, 1>{});
        }
      }
      // every MMA completes before tensor memory is released
      if (el) mma_commit_pair(drain, 0x1);
      __syncwarp();
      mbar_wait(drain, 0, abort_flag, drain_limit_ns(lim), p.status, W_MMA_DRAIN, 0, false);
    }
    if (warp >= kPromWarps + 2) {
      // Two loaders; a slot has 256 numbers for each of four k-blocks.  Rest
      // tile: one per token, with the scale of this CTA's rows of W; loader h
      // has tokens 128 h + lane + 32 i.  Full tile: one per token of this CTA
      // for each half of W's rows; loader h has half h, tokens lane + 32 i.  A
      // group's loads are in flight while the one before is written.
      const int h = warp - kPromWarps - 2;
      const int tok0 = h * 128 + lane;
      const bool vec = (kb & 3) == 0;
      int g = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int u = pid; ok && u < n_tiles; u += pairs) {
        const Tile t = pair_tile(tab, u);
        const bool whole = t.n == 0;
        const int nb = min(t.n0 / 128 + (whole ? h : static_cast<int>(rank)), p.nb - 1);
        const int from = whole ? static_cast<int>(rank) * 128 + lane : tok0;
        const float *sw = p.sw + (static_cast<int64_t>(t.expert) * p.nb + nb) * kb;
        const float *sx = p.sx + static_cast<int64_t>(t.row + from) * kb;
        float v[4][4], w[4];
        auto load = [&](int j) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float *src = sx + static_cast<int64_t>(32 * i) * kb + j;
            if (from + 32 * i >= t.rows) {
              v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
            } else if (vec) {
              const float4 q = *reinterpret_cast<const float4 *>(src);
              v[i][0] = q.x; v[i][1] = q.y; v[i][2] = q.z; v[i][3] = q.w;
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) v[i][k] = j + k < kb ? src[k] : 0.f;
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) w[k] = j + k < kb ? sw[j + k] : 0.f;
        };
        load(0);
        for (int j = 0; j < kb; j += 4) {
          ok = warp_wait<kBrief>(smem_u32(&se[g]), ph ^ 1, abort_flag, lim, p.status, W_S_EMPTY, u);
          if (!ok) break;
          float *dst = reinterpret_cast<float *>(smem + OFF_S + g * kGroupBytes) + tok0;
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[k * kTok + 32 * i] = v[i][k] * w[k];
          __syncwarp();
          if (lane == 0) mbar_arrive(&sf[g]);
          if (j + 4 < kb) load(j + 4);
          if (++g == kGroups) { g = 0; ph ^= 1; }
        }
      }
    }
  }
  // The odd CTA's shared and tensor memory stay until the pair is done with
  // them, and the even CTA's barriers until its partner's last arrival.
  tc_fence_before();
  cluster_sync();
  if (warp == kPromWarps + 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

template <bool kBrief>
cudaError_t launch(const LinearParams &p, int sms, cudaStream_t stream) {
  const auto kernel = linear_pair_kernel<kBrief>;
  static PerDevice<int> resident;      // CTA pairs that fit the device
  int max_pairs = 0;
  const cudaError_t err = resident.get(&max_pairs, [&](int *n) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3(2, 1, 1);
    c.blockDim = dim3(kThreads, 1, 1);
    c.dynamicSmemBytes = kSmem;
    c.attrs = attr;
    c.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(n, kernel, &c);
  });
  if (err != cudaSuccess) return err;
  const int64_t tiles = (p.R / kTok + std::min<int64_t>(p.R, p.G)) * ((p.N + 255) / 256);
  int64_t pairs = std::min<int64_t>(sms / 2, tiles);
  if (max_pairs > 0) pairs = std::min<int64_t>(pairs, max_pairs);
  return launch_step(kernel, static_cast<unsigned>(2 * pairs), kThreads, kSmem, stream, 2, p);
}

}  // namespace

int linear_pair_x_box() { return kXBox; }

cudaError_t launch_linear_pair(const LinearParams &p, int sms, cudaStream_t stream) {
  return brief_limit(p.wait_limit_ns) ? launch<true>(p, sms, stream) : launch<false>(p, sms, stream);
}

}  // namespace dg
