/*
 * dg_wgrad.h -- C ABI of the GB300 (sm_103a) K-grouped weight-gradient library.
 *
 * Mixture-of-Experts weight gradient, one GEMM per expert, all experts in one
 * launch:  D[e] (+)= A_e^T B_e  (with the casts that produce its FP8 operands,
 * and the M-grouped data gradient dx_e = dy_e W_e that pairs with it).  The operands are concatenated along tokens:
 * A is [sum_k, M] (upstream gradients dy, M = h_out), B is [sum_k, N] (input
 * activations x, N = h_in), and expert e owns the contiguous rows
 * [off_e, off_e + K_e), off_e = K_0 + ... + K_{e-1}.  The GEMM's reduction
 * axis is the token axis.
 *   Sources: "How to Use DeepGEMM Weight Gradient Kernels for Training
 *   Backward Passes" (sections "API Entry Points", "FP8 Implementation
 *   Example", "BF16 Alternative", "Dispatch and Tensor-Map Handling");
 *   "Is DeepGEMM directly applicable to backward in training?" (qijiaxing,
 *   26 Mar 2025: dw = dy^T x, K = tokens, one scale per 128 tokens along K).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every pointer argument named a, b, w, sfa, sfb, sfw, d, c, x, x_sf, q_in,
 *    sf_in, src_rows, pair_rows, topk_idx, ks, h, da, q_dh, sf_dh, q_a, sf_a,
 *    q, sf, ks_dev, ms_dev, counts, row_of_pair, xs, ye, y, dy, dye, dw, s, sx,
 *    sw, grad_scale, and every pointer in a dg_adamw_tensor, is a DEVICE
 *    pointer on the current CUDA device; ks_host, ms_host and tensors are HOST
 *    pointers.
 *  - All matrices are dense row-major with the last index contiguous (no
 *    padding between rows).  Device pointers must be 16-byte aligned.
 *  - The caller owns every buffer.  The first call on a device allocates one
 *    small status word for that device, kept until process exit.  Each FP8
 *    GEMM call also takes scratch for its packed scale factors (below) from a
 *    memory pool the library creates per device: allocated and freed in
 *    stream order on `stream` (cudaMallocFromPoolAsync / cudaFreeAsync), so
 *    calls on different streams never share it; the pool keeps freed blocks
 *    for reuse.  The data-gradient calls, dg_moe_layout_plan and (above 2^15
 *    pairs) dg_moe_sort take their scratch from the same pool.
 *    The BF16 GEMM, the casts and the other MoE step calls allocate nothing
 *    per call.
 *  - Work is enqueued on `stream` (NULL = legacy default stream) and runs
 *    asynchronously.  ks_host / ms_host are read during the call only;
 *    device buffers must stay valid until the enqueued work completes.
 *  - Argument errors are returned before anything is enqueued; the output is
 *    then untouched.  dg_last_error() gives a message for the calling thread.
 *  - DG_LOG=1 in the environment makes each GEMM call print its plan (tile
 *    orientation and width, tiles, entries split along K, output mode) to
 *    stderr.
 *  - Device-side waits are bounded (default 4 s; environment variable
 *    DG_WAIT_LIMIT_US, a decimal number, else DG_WAIT_LIMIT_MS, read at each
 *    call).  A wait that runs out makes the kernel stop early and record
 *    DG_ERR_TIMEOUT in the device status word, which dg_sync_check() reports;
 *    the output is then unspecified.  Waits for copies already in flight, on the way out, keep a
 *    limit of at least 2 s so that no copy outlives the kernel.
 *  - The MoE step calls launch their kernels as programmatic dependents: a
 *    kernel's CTAs may start while the kernel before it in the stream ends, and
 *    wait there for its completion before they read or write anything.
 *    DG_PDL=0 in the environment (read at each call) turns that off.
 *  - DG_DETERMINISTIC=1 in the environment (read at each call) keeps every
 *    expert of an in-place FP8 or BF16 GEMM in one piece (no split along K;
 *    see c under dg_k_grouped_fp8_wgrad), making in-place results bitwise
 *    reproducible at some cost in balance.
 */
#ifndef DG_WGRAD_H
#define DG_WGRAD_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *dg_stream_t; /* identical to cudaStream_t */

typedef enum {
    DG_OK = 0,
    DG_ERR_INVALID_ARG = 1,  /* bad shape, size, alignment, pointer or option */
    DG_ERR_UNSUPPORTED = 2,  /* device is not sm_103, or a size above a stated limit */
    DG_ERR_CUDA = 3,         /* a CUDA runtime / driver call failed */
    DG_ERR_TIMEOUT = 4       /* a bounded device-side wait ran out (see above) */
} dg_status;

typedef enum { DG_F32 = 0, DG_BF16 = 1 } dg_dtype;

typedef enum {
    DG_TOKEN_MAJOR = 0,   /* q is [T, C]: same layout as x (what the TN GEMM reads) */
    DG_CHANNEL_MAJOR = 1  /* q is [C, T]: the physical transpose of x */
} dg_layout;

/* Largest number of experts per call (one schedule entry per expert). */
#define DG_MAX_GROUPS 1024

/*
 * dg_k_grouped_fp8_wgrad -- K-grouped FP8 weight gradient with 1x1xgran_k
 * block scales.
 *
 *   D[e, m, n] = Cterm[e, m, n] + sum_{k in expert e}
 *                fp8(a[k, m]) * 2^(sfa[k / gran_k, m] - 127)
 *              * fp8(b[k, n]) * 2^(sfb[k / gran_k, n] - 127)
 *
 * Source: "How to Use DeepGEMM Weight Gradient Kernels for Training Backward
 * Passes", sections "API Entry Points" (k_grouped_fp8_gemm_tn_contiguous: the
 * TN form that reads [sum_k, M] / [sum_k, N] operands directly) and "FP8
 * Implementation Example" ((tensor, scale) operand pairs, ks on host and as a
 * device tensor, optional accumulator, recipe (1, 1, 128) with gran_k 32 or
 * 128); the DeepGEMM knowledge-base article "UE8M0 Format in DeepGEMM" (scales
 * are power-of-two UE8M0 bytes consumed by the SM100 tensor core).
 *
 *   a       E4M3 codes [sum_k, M]           sfa  UE8M0 bytes [sum_k / gran_k, M]
 *   b       E4M3 codes [sum_k, N]           sfb  UE8M0 bytes [sum_k / gran_k, N]
 *   d       output [G, M, N], FP32 or BF16 (d_dtype); BF16 is rounded to
 *           nearest-even from the FP32 accumulator.
 *   c       NULL: Cterm = 0.  c == d: accumulate in place (D += ...).  Any other
 *           pointer: a separate FP32 [G, M, N] accumulator (not modified).
 *           Only with d_dtype == DG_F32.  In place, an expert much longer than
 *           the others is split along K into parts that each add into D, so
 *           the order of the FP32 additions (and the last bits of D) may vary
 *           from run to run (unless DG_DETERMINISTIC is set); every other mode
 *           writes each element once and is bitwise reproducible.
 *   G       number of experts, 0 <= G <= DG_MAX_GROUPS.
 *   M, N    positive multiples of 16.
 *   sum_k   total tokens; must equal ks_host[0] + ... + ks_host[G-1].
 *   ks_host, ks_dev  per-expert token counts (host / device copies, same
 *           values).  Each K_e >= 0 and a multiple of 128 (an expert's slice is
 *           whole 128-token blocks).  K_e == 0 experts are skipped: with c == d
 *           their D[e] is untouched, with c == NULL it is zeroed, with a
 *           separate c it is a copy of C[e] ("Dispatch and Tensor-Map
 *           Handling": zero-size groups are skipped).  ks_dev is read by the
 *           kernel to confirm the host copy; a mismatch is recorded as
 *           DG_ERR_INVALID_ARG in the status word (see dg_sync_check).
 *   gran_k  32 or 128: tokens per scale block ("FP8 Implementation Example").
 * Work enqueued: a scale-packing pass, then the GEMM.  The pass rewrites every
 * group of four scale rows (four 128-token blocks at gran_k 128, the four
 * 32-token blocks of one 128-token block at gran_k 32) of each expert into
 * 512-byte records laid out as the tensor core reads scales, so the GEMM loads
 * them with TMA.  Scratch: (scale groups) x (2 * ceil(M' / 256) +
 * ceil(N' / BN) * ceil(BN / 128)) x 512 bytes, where (M', N') = (N, M) when
 * N % 224 != 0 and M % 224 == 0 (the kernel then computes tiles of D^T) and
 * (M, N) otherwise, BN = 224 if N' % 224 == 0 else 128, and the scale groups
 * are ceil(K_e / 512) per expert at gran_k 128 and K_e / 128 at gran_k 32
 * (about four times as many; an in-place expert split along K counts each
 * part's groups) -- about 3.9 MB for G = 32, M = 4096, N = 7168,
 * sum_k = 32768 at gran_k 128.
 * Errors: DG_ERR_INVALID_ARG for any violated condition above (including
 * NULL pointers where data is needed and misaligned pointers),
 * DG_ERR_UNSUPPORTED off sm_103, DG_ERR_CUDA on a failed launch or scratch
 * allocation.
 */
dg_status dg_k_grouped_fp8_wgrad(const void *a, const uint8_t *sfa,
                                 const void *b, const uint8_t *sfb,
                                 void *d, dg_dtype d_dtype, const float *c,
                                 int G, int M, int N, int64_t sum_k,
                                 const int *ks_host, const int *ks_dev,
                                 int gran_k, dg_stream_t stream);

/*
 * dg_k_grouped_fp8_wgrad_nt -- dg_k_grouped_fp8_wgrad with K-major (NT)
 * operands: a is E4M3 [M, sum_k] and b is E4M3 [N, sum_k] (the token axis
 * contiguous: the channel-major output of the casts, q [C, T]).  Everything
 * else -- scales sfa [sum_k / gran_k, M] and sfb [sum_k / gran_k, N], d, c,
 * ks, gran_k, errors, scratch -- is as for dg_k_grouped_fp8_wgrad, and the
 * result is the same sum.
 *
 * Source: "How to Use DeepGEMM Weight Gradient Kernels for Training Backward
 * Passes", section "API Entry Points" (k_grouped_fp8_gemm_nt_contiguous: A
 * non-transposed [M, K], B transposed [N, K]); "Is DeepGEMM directly applicable
 * to backward in training?" (qijiaxing, 26 Mar 2025: dy^T as A [h_out,
 * tokens], x^T as B [h_in, tokens]; 3 Apr 2025: a contiguous K axis is the
 * layout the NT form is built for).
 */
dg_status dg_k_grouped_fp8_wgrad_nt(const void *a, const uint8_t *sfa,
                                    const void *b, const uint8_t *sfb,
                                    void *d, dg_dtype d_dtype, const float *c,
                                    int G, int M, int N, int64_t sum_k,
                                    const int *ks_host, const int *ks_dev,
                                    int gran_k, dg_stream_t stream);

/*
 * dg_k_grouped_bf16_wgrad -- K-grouped weight gradient with BF16 operands and
 * FP32 accumulation, no scales:  D[e] = Cterm[e] + A_e^T B_e.
 *
 * Source: "How to Use DeepGEMM Weight Gradient Kernels for Training Backward
 * Passes", section "BF16 Alternative" (k_grouped_bf16_gemm_tn_contiguous,
 * same call shape as the FP8 form without scales).
 *
 *   a  BF16 [sum_k, M], b  BF16 [sum_k, N]; d, d_dtype, c as for the FP8 call.
 *   M, N positive multiples of 8.  K_e >= 0 arbitrary (no block alignment).
 * Errors as for the FP8 call.
 */
dg_status dg_k_grouped_bf16_wgrad(const void *a, const void *b,
                                  void *d, dg_dtype d_dtype, const float *c,
                                  int G, int M, int N, int64_t sum_k,
                                  const int *ks_host, const int *ks_dev,
                                  dg_stream_t stream);

/*
 * dg_m_grouped_fp8_dgrad -- the other GEMM of a MoE expert's backward, the
 * data (input) gradient, M-grouped over a contiguous token layout:
 *
 *   D[t, n] = sum_{k < K} fp8(A[t, k]) 2^(sfa[t, k / gran_k] - 127)
 *                         * fp8(W[e, k, n]) 2^(sfw[e, k / gran_k, n] - 127)
 *
 * for every token row t of expert e (rows [off_e, off_e + M_e), off_e =
 * M_0 + ... + M_{e-1}): dx_e = dy_e W_e with W_e the expert's [h_out, h_in]
 * weight as a linear layer stores it.
 *
 * Source: "Is DeepGEMM directly applicable to backward in training?"
 * (YouJiacheng, 26 Feb 2025: a GEMM's backward is two GEMMs; LyricZhao, same
 * day: the library ships the data-gradient GEMM, the weight gradient needs
 * the K-grouped kernel and the fused casts).  The pages give no layout or
 * scale recipe for it; this entry point takes the plainest one consistent
 * with the rest of the path: dy as the forward pass stores activations (E4M3,
 * one UE8M0 scale per token per gran_k channels, the 1 x 128 tile) and the
 * weight with one UE8M0 scale per column per gran_k rows of K (a 128 x 128
 * block scale is this with each block's byte repeated over its columns), both
 * scales along the contraction axis as the tensor core's block-scaled MMA
 * consumes them ("UE8M0 Format in DeepGEMM", packed scales on SM100).
 *
 *   a      E4M3 [sum_m, K], row-major (K contiguous): dy, experts' rows contiguous.
 *   sfa    UE8M0 [sum_m, K / gran_k].
 *   w      E4M3 [G, K, N], row-major (N contiguous).
 *   sfw    UE8M0 [G, K / gran_k, N].
 *   d      [sum_m, N] FP32 (d_dtype DG_F32) or BF16 (DG_BF16, round to
 *          nearest even), written (no accumulator).
 *   G      0 <= G <= DG_MAX_GROUPS; K a positive multiple of 128; N a
 *          positive multiple of 16; G * K < 2^31.
 *   ms_host, ms_dev  per-expert token counts (host / device copies, same
 *          values), each >= 0 and a multiple of 128 (the padded MoE layout,
 *          dg_moe_layout_plan); they sum to sum_m.  Experts with no tokens
 *          own no rows.  ms_dev is checked by the kernel as ks_dev is.
 *   gran_k 32 or 128.
 * Work enqueued: two scale-packing passes (dy's scales per 128-token chunk,
 * the weights' per N tile), then the GEMM.  Scratch from the device pool:
 * (ceil(K / 128 / g) x (sum_m / 128 + 1) + E x ceil(K / 128 / g) x
 * ceil(N / BN) x ceil(BN / 128)) x 512 bytes, g = 4 at gran_k 128 and 1 at
 * 32, E the experts with tokens, BN as above.  Errors as for the weight
 * gradient calls; DG_ERR_UNSUPPORTED also for an output of 2^40 bytes or more.
 */
dg_status dg_m_grouped_fp8_dgrad(const void *a, const uint8_t *sfa,
                                 const void *w, const uint8_t *sfw,
                                 void *d, dg_dtype d_dtype,
                                 int G, int K, int N, int64_t sum_m,
                                 const int *ms_host, const int *ms_dev,
                                 int gran_k, dg_stream_t stream);

/*
 * dg_m_grouped_fp8_dgrad_nt -- dg_m_grouped_fp8_dgrad with the weights stored
 * K-major: w is E4M3 [G, N, K] (row n of expert e holds W_e[:, n], K
 * contiguous), the layout of a transposed weight copy.  The scales keep the
 * layout sfw [G, K / gran_k, N] (one per column n per gran_k rows of K), and
 * a, sfa, d, ms, gran_k, the result, errors and scratch are as for
 * dg_m_grouped_fp8_dgrad.  G * N < 2^31.
 *
 * Source: as dg_m_grouped_fp8_dgrad; "How to Use DeepGEMM Weight Gradient
 * Kernels for Training Backward Passes", section "API Entry Points" (the NT
 * operand form: the second operand transposed, K contiguous).
 */
dg_status dg_m_grouped_fp8_dgrad_nt(const void *a, const uint8_t *sfa,
                                    const void *w, const uint8_t *sfw,
                                    void *d, dg_dtype d_dtype,
                                    int G, int K, int N, int64_t sum_m,
                                    const int *ms_host, const int *ms_dev,
                                    int gran_k, dg_stream_t stream);

/*
 * dg_quant_transpose_fp8 -- the cast a weight-gradient GEMM needs: per column,
 * per gran_k-token block, one power-of-two scale, values to E4M3.
 *
 *   amax    = max_{k in block} |x[k, col]|
 *   e       = clamp(ceil(log2(amax / 448)), -127, 127)   (amax == 0 -> -127)
 *   sf      = e + 127                                     (UE8M0 byte)
 *   q[k, col] = E4M3 round-to-nearest-even of x[k, col] * 2^-e
 *
 * Source: "Is DeepGEMM directly applicable to backward in training?"
 * (LyricZhao, 26 Feb 2025: weight gradients need fused transpose + cast
 * kernels; hxdtest quoting the DeepSeek-V3 workflow, 4 May 2025: activations
 * are transposed and re-quantised into 128x1 tiles; qijiaxing, 26 Mar 2025:
 * every 128 elements along the token axis share one scale).  448 is the
 * largest E4M3 magnitude, so the cast never saturates.
 *
 *   x         BF16 [T, C] (tokens x channels).
 *   T         non-negative multiple of gran_k.
 *   C         positive multiple of 16.
 *   q         E4M3 out: [T, C] (DG_TOKEN_MAJOR) or [C, T] (DG_CHANNEL_MAJOR).
 *   sf        UE8M0 out [T / gran_k, C].
 *   gran_k    32 or 128.
 * Inputs must be finite.  Errors: DG_ERR_INVALID_ARG / DG_ERR_UNSUPPORTED /
 * DG_ERR_CUDA as above.
 */
dg_status dg_quant_transpose_fp8(const void *x, int64_t T, int C,
                                 void *q, uint8_t *sf,
                                 dg_layout q_layout, int gran_k,
                                 dg_stream_t stream);

/*
 * dg_requant_transpose_fp8 -- re-quantise stored FP8 activations for the
 * weight gradient: from the forward pass's 1 x 128 tiles (one scale per token
 * per 128 channels) to column blocks (one scale per channel per gran_k
 * tokens), with the same cast as dg_quant_transpose_fp8 applied to the
 * exactly dequantised values:
 *
 *   x[t, c] = E4M3(q_in[t, c]) * 2^(sf_in[t, c / 128] - 127)
 *   (q, sf) = dg_quant_transpose_fp8 of x
 *
 * Source: "Is DeepGEMM directly applicable to backward in training?" (hxdtest,
 * 4 May 2025, quoting the DeepSeek-V3 workflow: forward activations are
 * stored as 1x128 FP8 tiles; the backward pass reads them out, dequantises,
 * transposes and re-quantises them into 128x1 tiles; TheTinyTeddy, 12 Mar
 * 2025: the FP8 weight-gradient GEMM lets activations be stored in FP8).  The
 * pages do not give the stored scales' format; here they are UE8M0 bytes (the
 * SM100 format of "UE8M0 Format in DeepGEMM").
 *
 *   q_in      E4M3 codes [T, C] (token-major, as the forward pass stored them).
 *   sf_in     UE8M0 bytes [T, C / 128]; bytes 0..254 (255 is NaN: unsupported).
 *   T         non-negative multiple of gran_k.
 *   C         positive multiple of 128.
 *   q, sf, q_layout, gran_k   as for dg_quant_transpose_fp8.
 * Every dequantised value is exact in the kernel (it works on x * 2^-8, which
 * is finite and exact in FP32 for every code and scale byte), so the result is
 * bit-identical to the definition above.  Errors as for dg_quant_transpose_fp8.
 */
dg_status dg_requant_transpose_fp8(const void *q_in, const uint8_t *sf_in,
                                   int64_t T, int C,
                                   void *q, uint8_t *sf,
                                   dg_layout q_layout, int gran_k,
                                   dg_stream_t stream);

/*
 * dg_quant_moe_layout_fp8 -- the column-block cast fused with the MoE token
 * layout: output row t is source row src_rows[t], or a row of zeros where
 * src_rows[t] == -1 (padding an expert's slice up to whole 128-token blocks),
 * then cast as by dg_quant_transpose_fp8 (BF16 source) or
 * dg_requant_transpose_fp8 (stored FP8 source).
 *
 * Source: "Is DeepGEMM directly applicable to backward in training?"
 * (LyricZhao, 26 Feb 2025: weight-gradient support needs utility kernels with
 * the cast fused with the MoE layout; NiuMa, 18 Mar 2025: the FP8 weight
 * gradient needs each expert's token count to be a multiple of 128).
 *
 *   x         x_sf == NULL: BF16 [T_src, C].  Otherwise E4M3 codes [T_src, C]
 *             with x_sf UE8M0 [T_src, C / 128] (1 x 128 tiles, as for
 *             dg_requant_transpose_fp8; C then a multiple of 128).
 *   T_src     source rows (>= 0, < 2^31).
 *   src_rows  device int32 [T]: source row of each output row, or -1.  An
 *             entry outside [-1, T_src) gives a zero row and is recorded as
 *             DG_ERR_INVALID_ARG in the device status word (dg_sync_check).
 *   T         output rows: a non-negative multiple of gran_k (each expert's
 *             slice is a whole number of blocks).
 *   q, sf, q_layout, gran_k   as for dg_quant_transpose_fp8, over the T output
 *             rows.
 * Errors as for dg_quant_transpose_fp8.
 */
dg_status dg_quant_moe_layout_fp8(const void *x, const uint8_t *x_sf,
                                  int64_t T_src, int C,
                                  const int *src_rows, int64_t T,
                                  void *q, uint8_t *sf,
                                  dg_layout q_layout, int gran_k,
                                  dg_stream_t stream);

/*
 * dg_moe_layout_plan -- the MoE token layout that dg_quant_moe_layout_fp8 and
 * the K-grouped GEMMs consume, built on the device from top-k routing.
 *
 * Expert e's slice holds its routing pairs (t, j) (topk_idx[t, j] == e) in the
 * order of the pair index t * topk + j, then -1 padding rows up to a multiple
 * of `align`; the slices follow in expert order.  ks[e] is the slice's padded
 * length, so ks feeds the GEMM's ks_dev directly (and, copied to the host, its
 * ks_host).  Deterministic: the same routing always gives the same layout.
 *
 * Source: "Is DeepGEMM directly applicable to backward in training?"
 * (LyricZhao, 26 Feb 2025: casts fused with the MoE layout; NiuMa, 18 Mar
 * 2025: the FP8 weight gradient needs each expert's token count to be a
 * multiple of 128, which padding provides).
 *
 *   topk_idx   device int32 [T_tok, topk]: the expert of each (token, slot),
 *              or -1 for an unused slot.  An entry outside [-1, G) is skipped
 *              and recorded as DG_ERR_INVALID_ARG in the device status word
 *              (dg_sync_check).
 *   T_tok      tokens (>= 0);  topk >= 1;  T_tok * topk + G * (align - 1) < 2^31.
 *   G          experts, 1 <= G <= DG_MAX_GROUPS.
 *   align      slice length multiple, 1..65536 (128 for the FP8 GEMM).
 *   ks         device int32 [G] out.
 *   src_rows   device int32 [cap] out: the source token t of each row, -1 on
 *              padding and on every row past the layout's end.
 *   pair_rows  device int32 [cap] out, or NULL: the pair index t * topk + j of
 *              each row (for operands stored per routed pair), -1 likewise.
 *   cap        rows of src_rows / pair_rows; at least T_tok * topk +
 *              G * (align - 1), the largest layout any routing can give.
 * Scratch: (ceil(T_tok * topk / 4096) + 1) * G int32 counters from the
 * library's stream-ordered pool.  Errors: DG_ERR_INVALID_ARG (arguments,
 * cap too small, NULL or misaligned pointers), DG_ERR_UNSUPPORTED (G above
 * DG_MAX_GROUPS, sizes above the limit), DG_ERR_CUDA.
 */
dg_status dg_moe_layout_plan(const int *topk_idx, int64_t T_tok, int topk,
                             int G, int align,
                             int *ks, int *src_rows, int *pair_rows,
                             int64_t cap, dg_stream_t stream);

/*
 * dg_swiglu_backward_quant_fp8 -- the SwiGLU backward of a MoE expert fused
 * with the column-block cast of its outputs, token-major:
 *
 *   h = [g | u] (gate half first), s = 1 / (1 + e^-g), silu(g) = g * s
 *   dg = da * u * s * (1 + g * (1 - s)),  du = da * silu(g),  a = silu(g) * u
 *   (q_dh, sf_dh) = cast of dh = [dg | du]   (the up/gate weight gradient's A)
 *   (q_a, sf_a)   = cast of a                 (the down-projection's B)
 * with the cast of dg_quant_transpose_fp8 (one UE8M0 scale per column per
 * gran_k tokens).
 *
 * Source: "Is DeepGEMM directly applicable to backward in training?"
 * (LyricZhao, 26 Feb 2025: weight-gradient support needs utility kernels,
 * among them casting fused with SwiGLU).  The pages give no formula; this is
 * the standard SwiGLU.
 *
 *   h       BF16 [T, 2I];  da  BF16 [T, I].
 *   T       non-negative multiple of gran_k.   I  positive multiple of 16.
 *   q_dh    E4M3 [T, 2I];  sf_dh  UE8M0 [T / gran_k, 2I].
 *   q_a     E4M3 [T, I] and sf_a UE8M0 [T / gran_k, I], or both NULL.
 *   gran_k  32 or 128.
 * Arithmetic: FP32 with explicitly rounded operations, e^-|g| from expf and
 * 1 / (1 + e^-|g|) from the hardware reciprocal (within 1 ulp); dg, du and a must stay finite in FP32
 * (non-finite values are unsupported).  Each quantised code and scale is the
 * one of a value within a few FP32 ulp of the exact result (the tests bound
 * it).  Errors as for dg_quant_transpose_fp8.
 */
dg_status dg_swiglu_backward_quant_fp8(const void *h, const void *da,
                                       int64_t T, int I,
                                       void *q_dh, uint8_t *sf_dh,
                                       void *q_a, uint8_t *sf_a,
                                       int gran_k, dg_stream_t stream);

/*
 * dg_k_grouped_fp8_wgrad_noalloc -- dg_k_grouped_fp8_wgrad for callers that
 * cannot allocate device memory.  The pages have no counterpart: this is an
 * addition of this library.
 *
 * The ordinary call allocates a 16-byte status record per device (cudaMalloc)
 * on its first use and takes stream-ordered scratch for the packed scale
 * factors on every call.  A caller whose device memory is owned by its own
 * caching allocator, or that must not take the device synchronisation
 * cudaMalloc can cause, cannot accept that.  This entry point computes exactly
 * what dg_k_grouped_fp8_wgrad computes, with the same arguments and errors,
 * by the same host steps (validation, schedule with its tile orientation and
 * split along K, tensor maps, scale packing, launch), and allocates nothing:
 * the status record and the packed scale records live in one file-scope
 * device array of the library, 256 bytes + 32 MiB (every GPU that loads this
 * part of the library holds it until the process exits).
 *  - The first call on a device does the set-up (device queries, the
 *    array's device address via cudaGetSymbolAddress); make that first call
 *    before any stream capture.
 *  - Each call clears the record and rewrites the scale records on `stream`
 *    before its GEMM; calls that overlap on the GPU (on different streams)
 *    share the array and race on it.
 *  - It never synchronises.  dg_sync_check() reads and clears this entry
 *    point's record as well as the ordinary one, so device-side timeouts and
 *    ks_dev mismatches are reported there.
 *  - Limits: the packed scale records must fit 32 MiB (their size is given
 *    under dg_k_grouped_fp8_wgrad; G = 64, M = 4096, N = 7168,
 *    sum_k = 131072 needs 14 MB at gran_k 128 and about four times that,
 *    above the limit, at gran_k 32); larger problems, and sizes above the kernel's own limits
 *    (G > DG_MAX_GROUPS, sum_k > 2^31 - 256), are rejected with
 *    DG_ERR_UNSUPPORTED and a message before any CUDA call.
 */
dg_status dg_k_grouped_fp8_wgrad_noalloc(const void *a, const uint8_t *sfa,
                                         const void *b, const uint8_t *sfb,
                                         void *d, dg_dtype d_dtype, const float *c,
                                         int G, int M, int N, int64_t sum_k,
                                         const int *ks_host, const int *ks_dev,
                                         int gran_k, dg_stream_t stream);

/*
 * The rest of a MoE layer's training or serving step around the GEMMs above:
 * tokens sorted by expert and back with their weights, the row cast and the
 * experts' forward FP8 product, and the optimizer that takes the weight
 * gradients.  Their formulas are the standard ones; the layouts and formats
 * are this library's.  Every call works on device counts and maps, waits for
 * nothing on the host and can be captured in a CUDA graph: a replay is the same
 * call again, on what its tensors hold then.  (A captured dg_moe_sort of more
 * than 2^15 pairs takes its scratch from an allocation that the graph owns.)
 * For dg_adamw_step that means the captured step number, rates and seed: an
 * optimizer whose steps count on is called, or captured anew, at each step.
 *
 * dg_moe_sort -- token rows in expert order, from top-k routing.
 *
 *   row(t, j) = off_e + #{pairs before t * topk + j routed to e},  e = topk_idx[t, j]
 *
 * off_e is the sum over the experts before e of their pair counts, each
 * rounded up to a multiple of `align`.  The layout (counts, pair_rows,
 * src_rows) is that of dg_moe_layout_plan; row_of_pair is its inverse, which
 * the calls below read.  Deterministic.
 *
 *   topk_idx     device int32 [T, topk]: the expert of each (token, slot), -1
 *                for an unused slot.  An entry outside [-1, G) is treated as
 *                unused and recorded (dg_sync_check: DG_ERR_INVALID_ARG).
 *   G            1 .. DG_MAX_GROUPS;  align 1 .. 65536.
 *   counts       device int32 [G] out: rows of each expert's slice.
 *   row_of_pair  device int32 [T, topk] out: row(t, j), -1 for an unused slot.
 *   pair_rows    device int32 [cap] out: pair t * topk + j of each row, -1 for
 *                padding rows and rows past the layout's end.
 *   src_rows     device int32 [cap] out or NULL: token t of each row, -1 likewise.
 *   cap          at least T * topk + G * (align - 1), below 2^31 - 256.
 * Scratch above 2^15 pairs: (chunks + 1) * G int32 of the device's pool (in a
 * captured call, of the graph), chunks the 512-pair (at most 2048) pieces of the
 * pairs.
 */
dg_status dg_moe_sort(const int *topk_idx, int64_t T, int topk, int G, int align, int *counts,
                      int *row_of_pair, int *pair_rows, int *src_rows, int64_t cap,
                      dg_stream_t stream);

/*
 * dg_moe_dispatch -- xs[row(t, j)] = x[t] for every used slot; rows whose
 * pair_rows entry is negative become zeros, so every row of xs is written.
 *
 *   x   [T, C], xs [R, C], both BF16 or both FP32 (dtype); C a positive
 *       multiple of 8.
 *   row_of_pair [T, topk], pair_rows [R] as dg_moe_sort wrote them (any leading
 *       R rows that hold the whole layout).  A row_of_pair entry at or past R
 *       is skipped and recorded (dg_sync_check: DG_ERR_INVALID_ARG).
 * Its gradient is dg_moe_combine with w NULL.
 */
dg_status dg_moe_dispatch(const void *x, dg_dtype dtype, int64_t T, int C, int topk,
                          const int *row_of_pair, const int *pair_rows, int64_t R, void *xs,
                          dg_stream_t stream);

/*
 * dg_moe_combine -- y[t] = sum_j w[t, j] ye[row(t, j)], the sum in FP32 in the
 * order of j, rounded once.  An unused slot gives nothing: its weight and any
 * padding row may hold anything, NaN included.  A token without used slots
 * gets zeros.  w NULL: plain sum (the gradient of dg_moe_dispatch).
 *
 *   ye [R, C], y [T, C] as for dg_moe_dispatch; w FP32 [T, topk].
 */
dg_status dg_moe_combine(const void *ye, dg_dtype dtype, int64_t R, int C, int64_t T, int topk,
                         const int *row_of_pair, const float *w, void *y, dg_stream_t stream);

/*
 * dg_moe_combine_backward -- gradient of dg_moe_combine:
 *
 *   dye[row(t, j)] = w[t, j] dy[t],   dw[t, j] = sum_c dy[t, c] ye[row(t, j), c]
 *
 * dw is summed in FP32 in a fixed order; an unused slot's is 0, and rows that
 * no pair owns get zeros in dye.
 *
 *   dy [T, C], ye and dye [R, C] as above; w, dw FP32 [T, topk].
 */
dg_status dg_moe_combine_backward(const void *dy, const void *ye, dg_dtype dtype, int64_t T, int C,
                                  int topk, const int *row_of_pair, const int *pair_rows,
                                  int64_t R, const float *w, void *dye, float *dw,
                                  dg_stream_t stream);

/*
 * dg_quant_rows_fp8 -- BF16 rows to E4M3 with one FP32 scale for each 128
 * columns, optionally sent to the experts' rows as by dg_moe_dispatch: the
 * left operand of dg_m_grouped_fp8_linear.
 *
 *   s[t, b] = max(amax_b, 2^-100) * fl(1 / 448)
 *   q[t, c] = E4M3 round-to-nearest-even of x[t, c] * fl(1 / s), |.| <= 448
 *
 * each step one correctly rounded FP32 operation; the last block of a row may
 * be shorter than 128.
 *
 *   x   BF16 [T, C], finite; C a positive multiple of 16.
 *   row_of_pair, pair_rows  both NULL (then R = T, topk = 1 and row t is row
 *       t), or as for dg_moe_dispatch (one that has no entries may be NULL);
 *       rows that no pair owns get codes 0 and the smallest scale, 2^-100 *
 *       fl(1 / 448).
 *   q   E4M3 [R, C];  s  FP32 [R, ceil(C / 128)].
 */
dg_status dg_quant_rows_fp8(const void *x, int64_t T, int C, int topk, const int *row_of_pair,
                            const int *pair_rows, int64_t R, void *q, float *s,
                            dg_stream_t stream);

/*
 * dg_m_grouped_fp8_linear -- the experts' forward product with FP32 block
 * scales and counts on the device only:
 *
 *   y[t, n] = sum_b sx[t, b] sw[e, n / 128, b] sum_{k in b} x[t, k] w[e, n, k]
 *
 * over the blocks b of 128 k (the last may be shorter), for the rows t of
 * expert e: [off_e, off_e + ms_dev[e]), off_e the sum of the counts before.
 * Any counts, zero included; rows past their sum are not written.  Block sums
 * are formed in the tensor core, scaled and added in FP32, and rounded once.
 * The two scales of a block are multiplied first, in FP32: a product below
 * 2^-126 loses bits, and one that overflows makes the row infinite or NaN.
 *
 *   x    E4M3 [R, K];  sx FP32 [R, ceil(K / 128)].
 *   w    E4M3 [G, N, K] (a linear layer's weight);
 *   sw   FP32 [G, ceil(N / 128), ceil(K / 128)].
 *   y    BF16 [R, N].
 *   K, N positive multiples of 16;  0 <= G <= DG_MAX_GROUPS;  R and G * N below
 *        2^31 - 256, and (R / 16 + min(R, G)) * ceil(N / 128) below 2^28.
 *   ms_dev  device int32 [G].  A negative count (taken as zero) and counts that
 *        sum past R (the rows past R are left out) are recorded
 *        (dg_sync_check: DG_ERR_INVALID_ARG).
 */
dg_status dg_m_grouped_fp8_linear(const void *x, const float *sx, const void *w, const float *sw,
                                  void *y, int G, int K, int N, int64_t R, const int *ms_dev,
                                  dg_stream_t stream);

/* One tensor of an optimizer step (device pointers, 16-byte aligned but for
 * the scales). */
typedef struct dg_adamw_tensor {
    float *p;          /* parameters, updated in place */
    const void *g;     /* gradients, FP32 or BF16 */
    void *m, *v;       /* moments: FP32 m and v, or E4M3 codes of m and of r = sqrt(v) */
    uint8_t *sm, *sv;  /* 8 bits: UE8M0 scales, one per 128 elements; else NULL */
    void *copy;        /* BF16 copy of the new parameters, or NULL */
    int64_t n;         /* elements, any number up to 2^40 */
} dg_adamw_tensor;

/*
 * dg_adamw_step -- AdamW over many tensors at once.
 *
 *   g' = g * grad_scale,  m' = b1 m + (1 - b1) g',  v' = b2 v + (1 - b2) g'^2
 *   p' = p (1 - lr wd) - lr / (1 - b1^t) m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
 *
 * 32-bit states hold m and v.  8-bit states hold m and r = sqrt(v) in blocks
 * of 128 elements of the flattened tensor as E4M3 codes times 2^(scale - 127),
 * the scale the smallest that brings the block's maximum to 448 or below;
 * zeros everywhere is the state before the first step.  The update takes the
 * new moments unrounded.  They are then rounded up to the next E4M3 number
 * with the probability of the part cut off, decided by 16 bits of a hash of
 * (seed, place of the tensor in the list, element): give each step its own
 * seed.  r above zero never becomes zero.  The same call gives the same bits.
 * Each code is right on average, m over many steps too; v, the square of a
 * rounded r, settles 3 to 6 % high and r spreads by 12 to 17 % (rms) under
 * steady gradients, whatever b2.
 *
 *   tensors     HOST array of n entries, read during the call only.
 *   grad_dtype  of every g;  state_bits 8 or 32, of every tensor.
 *   step        t, from 1.  betas in [0, 1).
 *   grad_scale  device FP32 scalar, or NULL for 1.  If it is not finite,
 *               nothing is written.
 * A code of m has m's sign, zeros included.  A non-finite gradient makes its
 * element's moments and parameter non-finite, one whose square overflows makes
 * v infinite; with 8 bits a non-finite moment is code 0x7F (NaN), without
 * effect on its block's scale.
 */
dg_status dg_adamw_step(const dg_adamw_tensor *tensors, int n, dg_dtype grad_dtype,
                        int state_bits, int64_t step, double lr, double beta1, double beta2,
                        double eps, double weight_decay, const float *grad_scale, uint64_t seed,
                        dg_stream_t stream);

/* Message describing the calling thread's last non-OK status ("" if none). */
const char *dg_last_error(void);

/*
 * Synchronise `stream`, then read and clear the current device's status words
 * (the ordinary entry points' record and dg_k_grouped_fp8_wgrad_noalloc's).
 * Allocates nothing.  Returns DG_ERR_TIMEOUT if a kernel gave up on a bounded
 * wait,
 * DG_ERR_INVALID_ARG if a kernel found ks_dev different from ks_host, a
 * src_rows, topk_idx or row_of_pair entry or an expert's row count out of range,
 * DG_ERR_CUDA if the synchronisation failed, else DG_OK.
 */
dg_status dg_sync_check(dg_stream_t stream);

/* Library version, major * 10000 + minor * 100 + patch. */
int dg_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DG_WGRAD_H */
