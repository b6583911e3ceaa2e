/*
 * jetfp8.h -- C ABI of the MI355X (gfx950) FP8 group-quantize + block-scaled GEMM library.
 *
 * The operations are those of the Jet-RL unified FP8 precision flow ("Jet-RL: Enabling On-Policy FP8
 * Reinforcement Learning with Unified Training and Rollout Precision Flow", gist.science explainers,
 * sections "Architecture Centrale" and "Schema de Quantification" / "Esquema de Quantizacao"):
 * the same FP8 linear layers serve rollout and the training forward; activations are quantized in 1x128
 * groups, weights in 128x128 blocks; gradients between operators stay BF16 and are quantized inside the
 * DGrad and WGrad GEMMs, which run in FP8 ("1x128 and 128x1" groupings for WGrad).
 *
 * Numerics (readings of what the pages leave open):
 *   FP8 format ... OCP E4M3 (bias 7, largest finite 448, NaN never produced).
 *   scale ........ s = fl32(amax / 448) per group, computed on every call (no calibration state).
 *   code ......... nearest E4M3 value to x / s (exact quotient), ties to the even code, |x/s| > 448
 *                  saturates to 448; an all-zero group has s = 0 and signed-zero codes.
 *   GEMMs ........ per output element: acc = +0; for each 128-wide group g of the contraction axis in
 *                  ascending order: acc = fma(p_g, fl32(sa_g * sb_g), acc), where p_g is the fp32 group
 *                  dot product formed by one gfx950 FP8 matrix instruction; out = bf16(acc), round to
 *                  nearest even.  The contraction is never split, so an output row is bitwise the same
 *                  whatever the number of rows in the call (decode M=1 and a training batch agree).
 *
 * Conventions for every entry point:
 *   - Matrices are dense, row-major, last index contiguous; bf16 tensors are passed as raw 16-bit
 *     patterns (void*), FP8 codes as uint8_t, scales as float.  No strides, but for the row pitches (ldq, ldk, ldv) of
 *     the key/value cache's calls and those (ldx, ldd) of the rotary positions.
 *   - Every pointer is a DEVICE pointer owned by the caller; the library never allocates, frees or
 *     synchronizes.  Work is enqueued on `stream` (a hipStream_t; NULL = the default stream) and runs
 *     asynchronously; outputs are valid once the stream has reached that point.
 *   - Arguments are validated on the host before anything is launched.  Return value: JETFP8_OK, or a
 *     negative jetfp8_status; on error nothing has been enqueued and outputs are untouched
 *     (JETFP8_ERR_HIP: a launch was rejected by the runtime; earlier kernels of the same call may have
 *     been enqueued).  No exception ever crosses this interface.
 *   - All pointers must be 16-byte aligned (JETFP8_ERR_ALIGN otherwise).  Buffers must not overlap, but where a call
 *     says that an output may be one of its inputs.
 *   - Sizes: every dimension >= 1; every grouped or contraction axis a multiple of 128, plus the
 *     per-mode rules below (JETFP8_ERR_SHAPE otherwise); every dimension < 2^31.  Kernels address their
 *     tiles with 32-bit offsets and launch one-dimensional grids, so each call also rejects, with
 *     JETFP8_ERR_SHAPE and before any launch:
 *       GEMMs ............... 256 * (contraction length) >= 2^31, or (contraction length / 128) * (rows of
 *                             either operand) * 4 >= 2^31 (bytes of a scale array);
 *       ROWS_1x128 .......... ceil(cols / 512) * ceil(rows / 32) > 2^31 - 1;
 *       COLS_128x1_T ........ ceil(cols / 128) * (rows / 128) > 2^31 - 1;
 *       BLOCKS_128x128 ...... rows / 128 > 65535;
 *       quantize_dual ....... (cols / 128) * (rows / 128) > 2^31 - 1, 64 * cols + 256 >= 2^31, or
 *                             128 * rows + 128 >= 2^31;
 *       requantize_cols_t ... (cols / 128) * (rows / 128) > 2^31 - 1, 32 * cols + 128 >= 2^31, or
 *                             128 * rows + 128 >= 2^31;
 *       swiglu_quantize ..... ceil(cols / 512) * ceil(rows / 32) >= 2^31, or 128 * cols >= 2^31 (32 rows of
 *                             gate_up in bytes);
 *       kv_append, attention  2 * kv_heads * num_units >= 2^24, and attention also grids of its own kernels of
 *                             2^24 thread blocks or more (a launch holds fewer than 2^32 threads);
 *       rotary .............. tokens >= 2^24 - 1024, or heads >= 2^20;
 *       kv_prefix, kv_fork,
 *       kv_sweep ............ requests > 4096, 64 * max_blocks >= 2^31, or requests * max_blocks >= 2^31;
 *       kv_fork_recent,
 *       kv_move ............. requests (moves) * kv_heads >= 2^24.
 *   - Thread safety: calls are independent; concurrent calls on different streams are allowed.
 */
#ifndef JETFP8_H
#define JETFP8_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    JETFP8_OK = 0,
    JETFP8_ERR_NULL = -1,   /* a required pointer is NULL */
    JETFP8_ERR_SHAPE = -2,  /* a dimension < 1, >= 2^31, or a grouped/contraction axis not a multiple of 128 */
    JETFP8_ERR_ALIGN = -3,  /* a pointer is not 16-byte aligned */
    JETFP8_ERR_MODE = -4,   /* unknown grouping mode, or dst_codes_t given for a mode without it */
    JETFP8_ERR_HIP = -5,    /* the HIP runtime rejected a launch */
    JETFP8_ERR_VALUE = -6   /* a scalar argument is outside its domain (e.g. eps <= 0) */
} jetfp8_status;

typedef enum {
    /* 1x128 groups along the contiguous axis (activations X for the forward, dY for DGrad).
     * src [rows][cols] -> dst_codes [rows][cols], dst_scales [cols/128][rows].  cols % 128 == 0. */
    JETFP8_ROWS_1x128 = 0,
    /* 128x1 groups along the row axis, codes written transposed (dY and X for WGrad, grouped along
     * the token axis).  src [rows][cols] -> dst_codes [cols][rows], dst_scales [rows/128][cols].
     * rows % 128 == 0, cols % 64 == 0. */
    JETFP8_COLS_128x1_T = 1,
    /* 128x128 blocks (weights).  src [rows][cols] -> dst_codes [rows][cols],
     * dst_scales [rows/128][cols/128], and when dst_codes_t != NULL the same codes transposed,
     * dst_codes_t [cols][rows] (the B operand of DGrad).  rows % 128 == 0 and cols % 128 == 0. */
    JETFP8_BLOCKS_128x128 = 2,
    /* As JETFP8_BLOCKS_128x128 (same codes, scales and optional row-major transposed copy), with dst_codes written
     * in the fragment order that jetfp8_gemm_fwd_frag reads: the byte of row n, column k goes to
     *   ((n / 16) * (cols / 128) + k / 128) * 2048 + ((k % 32) / 16) * 1024 + 16 * (n % 16 + 16 * ((k % 128) / 32))
     *   + k % 16.
     * A pure permutation of the row-major codes (same size); rows % 128 == 0 and cols % 128 == 0. */
    JETFP8_BLOCKS_128x128_FRAG = 3
} jetfp8_grouping;

/* Group quantization of a bf16 matrix to E4M3 codes plus fp32 scales (Jet-RL explainers,
 * "Schema de Quantification": 1x128 per-group for activations, 128x128 per-block for weights;
 * 1x128 and 128x1 for WGrad).  dst_codes_t is only accepted (and optional) for BLOCKS_128x128;
 * pass NULL for the other modes. */
int jetfp8_quantize(const void* src_bf16, int64_t rows, int64_t cols, int mode,
                    uint8_t* dst_codes, float* dst_scales, uint8_t* dst_codes_t, void* stream);

/* Both groupings of one bf16 matrix from a single read of it: the 1x128 codes and scales of
 * JETFP8_ROWS_1x128 and the transposed 128x1 codes and scales of JETFP8_COLS_128x1_T, bit for bit the
 * outputs of those two modes.  This serves a tensor that feeds a GEMM along its contiguous axis and the
 * WGrad GEMM along its token axis (Jet-RL explainers, "Schema de Quantification" / "Passage Arriere": dY
 * is quantized for DGrad and for WGrad; X for the forward and for WGrad): 4 bytes of codes written per
 * 2 bytes read, instead of reading the matrix twice.
 * src [rows][cols] -> dst_codes [rows][cols], dst_scales [cols/128][rows], dst_codes_t [cols][rows],
 * dst_scales_t [rows/128][cols].  rows % 128 == 0 and cols % 128 == 0; all four outputs are required. */
int jetfp8_quantize_dual(const void* src_bf16, int64_t rows, int64_t cols, uint8_t* dst_codes,
                         float* dst_scales, uint8_t* dst_codes_t, float* dst_scales_t, void* stream);

/* WGrad operand from a saved FP8 activation.  The pages keep the activations saved for the backward pass in
 * FP8 (Jet-RL explainers, "Schema de Quantification"); WGrad needs X grouped along the token axis.  This
 * takes the 1x128 codes of X and their scales (the JETFP8_ROWS_1x128 outputs), dequantizes each element as
 * one fp32 product decode(code) * scale, and quantizes those values in 128x1 groups along the rows with the
 * same scale and rounding rules as JETFP8_COLS_128x1_T, codes written transposed.  Reads 1 byte per element
 * instead of the 2 of the bf16 matrix.  Finite codes only (0x7F / 0xFF are E4M3 NaN).
 * codes [rows][cols], scales [cols/128][rows] -> dst_codes_t [cols][rows], dst_scales_t [rows/128][cols].
 * rows % 128 == 0 and cols % 128 == 0. */
int jetfp8_requantize_cols_t(const uint8_t* codes, const float* scales, int64_t rows, int64_t cols,
                             uint8_t* dst_codes_t, float* dst_scales_t, void* stream);

/* Fused RMSNorm -> 1x128 quantization.  The activation quantization is fused with the operator that produces
 * the activation (Jet-RL explainers, "Schema de Quantification"), here the RMSNorm in front of a linear layer:
 *   r[i]    = fp32 nearest to 1 / sqrt(mean_k x[i][k]^2 + eps)      (formed in fp64; see below)
 *   y[i][k] = bf16( fl32( fl32(x[i][k] * r[i]) * weight[k] ) )       (round to nearest even)
 *   dst_codes, dst_scales = the JETFP8_ROWS_1x128 quantization of y, bit for bit.
 * x [rows][cols] bf16, weight [cols] bf16 -> dst_codes [rows][cols], dst_scales [cols/128][rows];
 * optional (NULL = not written): dst_rstd [rows] fp32 (r, for the backward), dst_y_bf16 [rows][cols] (y).
 * r is the correctly rounded value unless the exact value lies within about 2^-47 (relative) of a point
 * where its fp32 rounding changes; there either neighbour may be returned.  cols % 128 == 0 and
 * cols <= 8192 (a row is held in registers); 0 < eps <= FLT_MAX (JETFP8_ERR_VALUE otherwise).
 * Finite inputs whose y overflows bf16 give unspecified codes for that group. */
int jetfp8_rmsnorm_quantize(const void* x_bf16, const void* weight_bf16, int64_t rows, int64_t cols, float eps,
                            uint8_t* dst_codes, float* dst_scales, float* dst_rstd, void* dst_y_bf16, void* stream);

/* The same behind a residual connection: h = bf16(fl32(x + residual)), the residual stream's next value, is written to
 * dst_h_bf16 [rows][cols], and codes, scales, rstd and y are those of jetfp8_rmsnorm_quantize of h, bit for bit.  dst_h_bf16
 * may be x_bf16 or residual_bf16 (an update in place).  x + residual must not overflow bf16. */
int jetfp8_rmsnorm_add_quantize(const void* x_bf16, const void* residual_bf16, const void* weight_bf16, int64_t rows,
                                int64_t cols, float eps, void* dst_h_bf16, uint8_t* dst_codes, float* dst_scales,
                                float* dst_rstd, void* dst_y_bf16, void* stream);

/* Backward pass of both.  Gradients between operators stay in bf16 (Jet-RL explainers, "Schema de Quantification"); with
 * dy that of y (from DGrad), dres that of h by way of the residual stream (NULL: none), the roundings taken as the identity
 * and g = dy * weight:
 *   dx[i][k] = rstd[i] * (g[i][k] - h[i][k] * rstd[i]^2 * mean_k(g[i] h[i])) + dres[i][k]
 *   dw[k]    = sum_i dy[i][k] * h[i][k] * rstd[i]
 * dx is the gradient of h, so of x and of the residual alike.  dy, h, dres [rows][cols] bf16, weight [cols] bf16, rstd
 * [rows] fp32 -> dst_dx_bf16 [rows][cols] (fp32, rounded once; it may be dy_bf16 or dres_bf16), dst_dw [cols] fp32
 * (NULL: not written; then no workspace is needed).  Column sums are fp32 in one fixed order over at most 512 parts of the
 * rows and fp64 over the parts: a call's results are the same every time.  cols % 128 == 0 and cols <= 8192.
 * workspace: jetfp8_rmsnorm_backward_workspace() bytes; calls that may run at the same time need one each;
 * JETFP8_ERR_SHAPE if workspace_bytes is less. */
int jetfp8_rmsnorm_backward(const void* dy_bf16, const void* h_bf16, const void* weight_bf16, const float* rstd,
                            const void* dres_bf16, int64_t rows, int64_t cols, void* dst_dx_bf16, float* dst_dw,
                            void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that jetfp8_rmsnorm_backward needs for dst_dw; JETFP8_ERR_SHAPE if it would refuse the sizes. */
int64_t jetfp8_rmsnorm_backward_workspace(int64_t rows, int64_t cols);

/* Fused SwiGLU -> 1x128 quantization (the activation in front of the down projection, quantized by the
 * operator that produces it; Jet-RL explainers, "Schema de Quantification"):
 *   h[i][j] = bf16 nearest to silu(g) * u = g * u / (1 + exp(-g)) of the exact real value, with
 *             g = gate_up[i][j] (gate: columns 0 .. cols-1) and u = gate_up[i][cols + j] (up: cols .. 2cols-1);
 *   dst_codes, dst_scales = the JETFP8_ROWS_1x128 quantization of h, bit for bit.
 * gate_up [rows][2 cols] bf16 -> dst_codes [rows][cols], dst_scales [cols/128][rows]; optional
 * dst_h_bf16 [rows][cols] (h; NULL = not written).  cols % 128 == 0.  Finite inputs; inputs whose h
 * overflows bf16 give unspecified codes for that group. */
int jetfp8_swiglu_quantize(const void* gate_up_bf16, int64_t rows, int64_t cols, uint8_t* dst_codes,
                           float* dst_scales, void* dst_h_bf16, void* stream);

/* Forward FP8 linear (rollout decode, prefill, training forward).  Jet-RL explainers, "Architecture Centrale":
 * rollout runs the same FP8 linear layers, with the same quantization, as the training forward pass;
 * "Schema de Quantification": activations in 1x128 groups, weights in 128x128 blocks, FP8 GEMM.
 *   Y[m][n] = sum_g xs[g][m] * ws[n/128][g] * sum_{k in g} xq[m][k] * wq[n][k]
 * xq [M][K], xs [K/128][M] (JETFP8_ROWS_1x128 of X); wq [N][K], ws [N/128][K/128]
 * (JETFP8_BLOCKS_128x128 of W); y [M][N] bf16.  K % 128 == 0, N % 128 == 0, any M >= 1. */
int jetfp8_gemm_fwd(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws,
                    void* y_bf16, int64_t M, int64_t N, int64_t K, void* stream);

/* Forward FP8 linear for rollout decode over weights in the fragment order of JETFP8_BLOCKS_128x128_FRAG: the
 * same operation, and bitwise the same result, as jetfp8_gemm_fwd on the row-major codes.  Jet-RL explainers,
 * "Enonce du Probleme": rollout takes over 70 % of RL training time; at decode token counts the GEMM streams the
 * FP8 weights once per step, and this layout lets every weight load read whole 128-byte lines.
 * xq [M][K], xs [K/128][M]; wq_frag (N * K bytes, fragment order), ws [N/128][K/128]; y [M][N] bf16.
 * K % 128 == 0, N % 128 == 0, 1 <= M <= 64 and (K / 128) * M <= 8192 (JETFP8_ERR_SHAPE otherwise). */
int jetfp8_gemm_fwd_frag(const uint8_t* xq, const float* xs, const uint8_t* wq_frag, const float* ws,
                         void* y_bf16, int64_t M, int64_t N, int64_t K, void* stream);

/* DGrad FP8 GEMM (Jet-RL explainers, "Schema de Quantification", backward-pass items: gradients between
 * operators stay BF16, and the DGrad GEMM runs in FP8 with the gradient quantized on entry):
 *   dX[m][k] = sum_g dys[g][m] * ws[g][k/128] * sum_{n in g} dyq[m][n] * wqT[k][n]
 * dyq [M][N], dys [N/128][M] (JETFP8_ROWS_1x128 of dY); wqT [K][N] (the transposed block codes of W
 * from JETFP8_BLOCKS_128x128), ws [N/128][K/128] (the forward block scales, unchanged);
 * dx [M][K] bf16.  N % 128 == 0, K % 128 == 0, any M >= 1. */
int jetfp8_gemm_dgrad(const uint8_t* dyq, const float* dys, const uint8_t* wqT, const float* ws,
                      void* dx_bf16, int64_t M, int64_t N, int64_t K, void* stream);

/* WGrad FP8 GEMM.  Jet-RL explainers, "Schema de Quantification" / "Esquema de Quantizacao": the weight
 * gradient GEMM runs in FP8 with the "1x128 and 128x1" configuration, read as both operands grouped along the
 * token axis, which is the contraction axis; gradients reach it in BF16 and are quantized on entry:
 *   dW[n][k] = sum_g dysT[g][n] * xsT[g][k] * sum_{m in g} dyqT[n][m] * xqT[k][m]
 * dyqT [N][M], dysT [M/128][N] (JETFP8_COLS_128x1_T of dY); xqT [K][M], xsT [M/128][K]
 * (JETFP8_COLS_128x1_T of X); dw [N][K] bf16, overwritten.  M % 128 == 0, N % 128 == 0,
 * K % 128 == 0. */
int jetfp8_gemm_wgrad(const uint8_t* dyqT, const float* dysT, const uint8_t* xqT, const float* xsT,
                      void* dw_bf16, int64_t M, int64_t N, int64_t K, void* stream);

/* ---- Rollout's FP8 key/value cache ---------------------------------------------------------------------------
 *
 * Rollout takes most of RL training time, and more of it the longer the generations (Jet-RL explainers, "Enonce du
 * Probleme"); next to the weights each decode step streams the keys and values of every token so far.  Here they are
 * kept in the flow's own precision, E4M3 with scale amax / 448 formed when they are written, and by a definition that
 * does not depend on how a sequence was cut into calls ("Architecture Centrale": rollout and the training forward
 * share one graph and one quantization):
 *   - a BLOCK is JETFP8_KV_BLOCK = 64 consecutive tokens of a request (positions 64 j .. 64 j + 63).  A complete block
 *     is quantized once, from bf16: per kv head one scale for the 64 x D keys and one for the 64 x D values;
 *   - until it is complete a block is kept in bf16 (a RECENT block);
 *   - a query at position t reads blocks 0 .. t/64 - 1 as E4M3 and positions 64 (t/64) .. t as bf16.
 * No token is quantized twice, and no query reads a scale that later tokens had a part in.
 *
 * Buffers (kv_heads H, head_dim D = 64 or 128):
 *   codes  uint8 [num_blocks][H][2][64 D], scales float [num_blocks][H][2]: keys (0) and values (1) of the physical
 *          blocks.  Complete blocks are never written again, so requests may share them (a prompt that several
 *          rollouts start from: the same physical ids in several rows of the block table);
 *   recent bf16 [recent_blocks][H][2][64 D], recent_blocks >= 2 requests + tokens / 64 for the largest call
 *          (jetfp8_attention refuses less): blocks 2 r and 2 r + 1 belong to request r and keep its unfinished block from
 *          call to call; those from 2 requests on hold the blocks that a call's prompts pass through.  So every step
 *          is planned for the same number of requests (one that is idle has no new tokens);
 *   block_table int32 [requests][max_blocks]: physical block of each complete block of each request.
 * Inside a block the 64 D values are in the order in which the attention kernel's waves read them.  For key n and
 * channel d:
 *   codes, keys     ((n/16 * D/64 + d/64) * 64 + d%32/8 * 16 + n%16) * 16 + d%64/32 * 8 + d%8
 *   codes, values   (d/16 * 64 + n%16/4 * 16 + d%16) * 16 + n/32 * 8 + n%32/16 * 4 + n%4
 *   recent, keys    ((n/16 * D/32 + d/32) * 64 + d%32/8 * 16 + n%16) * 8 + d%8
 *   recent, values  ((d/16 * 2 + n/32) * 64 + n%16/4 * 16 + d%16) * 8 + n%32/16 * 4 + n%4
 *
 * A step (decode, prefill, or both in one batch) is: plan once, then for every layer append and attention with that
 * layer's codes, scales and recent.  Every call reads its lengths on the device, so a step can be captured in a graph
 * and replayed; max_new and max_seq only bound them.
 */
#define JETFP8_KV_BLOCK 64
#define JETFP8_KV_UNIT_WORDS 8

typedef enum {                  /* per-request outcome of jetfp8_kv_plan */
    JETFP8_KV_OK = 0,
    JETFP8_KV_BAD_LENGTH = 1,   /* a negative length, more new tokens than max_new, more tokens than the table's row
                                 * holds, or a recent block other than 0 or 1 */
    JETFP8_KV_NO_ROWS = 2,      /* its new tokens end behind the call's rows */
    JETFP8_KV_NO_BLOCK = 4      /* it completes more blocks than the free list has left, or one whose id is no block of
                                 * the cache.  Blocks are handed out in request order: after a request that is refused
                                 * for them no later one gets any in this step, so that a request that needs many is not
                                 * passed by for ever.  Who would rather let them pass plans it without new tokens */
} jetfp8_kv_status;

/* Units that a plan of this many rows and requests may have: min(tokens, (tokens + 62 requests) / 64 + requests). */
int64_t jetfp8_kv_max_units(int64_t tokens, int64_t requests);

/* Block tables, slot map and work units of a step, on the device, from the requests' lengths.
 *   state [requests][2] int32: tokens so far, and which of the request's two recent blocks (0 or 1) is being filled;
 *                              (0, 0) for a new request;
 *   new_lens [requests] int32: new tokens of each request, 0 .. max_new (0: it has no part in the step).  Their rows
 *                              follow one another in the call's q, k, v ([tokens] rows; rows behind the last
 *                              request's are padding and stay untouched);
 *   free_blocks [num_free] int32 (may be NULL if num_free is 0), free_head [1] int32: ids of unused physical blocks, of
 *                              which the first *free_head have been handed out.  A negative id ends the list;
 * Writes
 *   block_table [requests][max_blocks] int32: only the entries of blocks that the step completes, taken from the free
 *                              list in request order;
 *   next_state, next_free:     state and free_head after the step (other buffers than the inputs, so that a step can
 *                              be planned again);
 *   status [requests] int32:   jetfp8_kv_status.  A request that is refused has no units, its rows stay untouched in
 *                              later calls, and its state does not change; the others go ahead (but for
 *                              those that complete a block, after one with JETFP8_KV_NO_BLOCK);
 *   units [jetfp8_kv_max_units(tokens, requests)][JETFP8_KV_UNIT_WORDS] int32, in request and block order: request,
 *                              block index, recent block, first row, rows, place of the first row in the block,
 *                              physical block (-1: not complete after this step), 0; unused records are all -1;
 *   slots [tokens] int64 (NULL: not written): 64 * physical block + place of every new token whose block the step
 *                              completes, -1 for the others.
 * requests <= 4096, tokens <= 2^19, 64 * max_blocks < 2^31. */
int jetfp8_kv_plan(const int32_t* state, const int32_t* new_lens, const int32_t* free_blocks, int64_t num_free,
                   const int32_t* free_head, int32_t* block_table, int64_t max_blocks, int64_t requests,
                   int64_t tokens, int64_t max_new, int32_t* next_state, int32_t* next_free, int32_t* status,
                   int32_t* units, int64_t* slots, void* stream);

/* The same for a cache of num_blocks blocks and recent_blocks recent blocks (every layer's, as given to append and
 * attention).  The free list ends at its first id that is not in 0 .. num_blocks - 1, and recent_blocks
 * < 2 requests + tokens / 64 is refused (JETFP8_ERR_SHAPE), so that the units of every request with status
 * JETFP8_KV_OK fit the cache and none of its tokens is left out.  jetfp8_kv_plan cannot see ids that are too large:
 * append and attention leave out units that have one. */
int jetfp8_kv_plan_cache(const int32_t* state, const int32_t* new_lens, const int32_t* free_blocks, int64_t num_free,
                         const int32_t* free_head, int32_t* block_table, int64_t max_blocks, int64_t requests,
                         int64_t tokens, int64_t max_new, int64_t num_blocks, int64_t recent_blocks,
                         int32_t* next_state, int32_t* next_free, int32_t* status, int32_t* units, int64_t* slots,
                         void* stream);

/* New keys and values into a layer's cache: into the recent blocks, and for each block that the step completes its
 * codes and scales.  k, v: bf16, row t at k + t * ldk elements, [kv_heads][head_dim] contiguous within a row (so they
 * may be columns of a fused projection); ldk, ldv >= kv_heads * head_dim and multiples of 8.  Repeating the call
 * writes the same values again.  A unit whose fields do not fit the buffers is left out (units of
 * jetfp8_kv_plan_cache fit).  Finite inputs (others give unspecified codes of their block and head). */
int jetfp8_kv_append(const void* k_bf16, int64_t ldk, const void* v_bf16, int64_t ldv, int64_t tokens,
                     const int32_t* units, int64_t num_units, int64_t kv_heads, int64_t head_dim, uint8_t* codes,
                     float* scales, int64_t num_blocks, void* recent_bf16, int64_t recent_blocks, void* stream);

/* Causal attention of the step's new tokens over the cache, after jetfp8_kv_append of the same step:
 *   o[t][h] = sum_n p_n v_n,  p = softmax_n(softmax_scale * q[t][h] . k_n),  n over the positions up to t's,
 * k_n and v_n being those of kv head h / (q_heads / kv_heads).  q: bf16, row t at q + t * ldq elements,
 * [q_heads][head_dim] contiguous within a row.
 *   dst_o_bf16 [tokens][q_heads][head_dim] (NULL: not written);
 *   dst_codes, dst_scales (both or neither; head_dim 128 only): the JETFP8_ROWS_1x128 quantization of that bf16
 *   matrix [tokens][q_heads * 128], bit for bit: the activation of the output projection, quantized by the operator
 *   that produces it (Jet-RL explainers, "Schema de Quantification").
 * fp32 scores, softmax and sums.  For the second product the probabilities are rounded: over the own block to 16 bits; over
 * the cache, each together with its block's value scale s_n, to 11 bits where p_n s_n is above 2^-20 of the row's largest
 * such product, and by at most 2^-31 of that largest below (so a block of small values keeps its bits beside one of large
 * values that has no weight).  Where values are near 2^-126 and below, an error of 2^-134 or less (half a bf16 there) is
 * added.  A row's sums have one fixed order (spans of 8 blocks, joined in ascending order, then its own block), so a
 * token's result is bitwise the same decoded alone, in a batch, or within a prompt.
 * max_new: no request has more new tokens; max_seq: nor more tokens after the step.  A unit beyond either, or whose
 * fields do not fit the buffers, is left out (its rows stay as they were); a block id outside 0 .. num_blocks - 1
 * reads as a block without keys.  Infinities and NaN reach only the rows that may see them.  Values below 2^90 (sums over
 * the keys are taken before they are divided by the denominator), queries below 2^104 (scores over the cache are those of
 * its codes until their scale comes in; at -infinity a key has no weight, at infinity the row is NaN).
 * 0 < softmax_scale <= FLT_MAX / 2 (JETFP8_ERR_VALUE otherwise).
 * workspace: jetfp8_attention_workspace() bytes (its content is not kept between calls; calls that may run at the same
 * time need one each); JETFP8_ERR_SHAPE if workspace_bytes is less. */
int jetfp8_attention(const void* q_bf16, int64_t ldq, int64_t tokens, const int32_t* units, int64_t num_units,
                     const int32_t* block_table, int64_t requests, int64_t max_blocks, const uint8_t* codes,
                     const float* scales, int64_t num_blocks, const void* recent_bf16, int64_t recent_blocks,
                     int64_t max_new, int64_t max_seq, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                     float softmax_scale, void* dst_o_bf16, uint8_t* dst_codes, float* dst_scales, void* workspace,
                     int64_t workspace_bytes, void* stream);

/* Bytes of workspace that jetfp8_attention needs for these sizes (0: none); JETFP8_ERR_SHAPE if it would refuse them.
 * A call lays its work and workspace out by max_new and max_seq for every unit alike (the rows of up to 64 new tokens,
 * the partial results of a request of max_seq tokens).  So a step with a prompt's chunk beside many single tokens takes
 * less of both as two calls, each with a part of the plan's units (any part, in any order) and its own max_new. */
int64_t jetfp8_attention_workspace(int64_t num_units, int64_t max_new, int64_t max_seq, int64_t q_heads,
                                   int64_t kv_heads, int64_t head_dim);

/* ---- Samples that share a prompt, and the cache's pages between steps ------------------------------------------
 *
 * Reinforcement learning rolls out several samples of each prompt (Jet-RL explainers, "Enonce du Probleme": rollout is
 * most of the time).  Their requests hold the prompt's complete blocks in common: the same ids at the head of their rows
 * of the block table.  A request holds what the first tokens / 64 entries of its row name, and nothing else says so:
 * blocks need no counts, and a request that is done gives up its own by having 0 tokens in its state.
 * The calls that take a state stand between two steps and take that after the last one (jetfp8_kv_plan's next_state): by the
 * state before a step, the blocks that the step filled would count as free.
 */

/* Which units of a step share blocks, from jetfp8_kv_plan's units in their order: once for a step, for all layers.
 *   groups [requests] int32: consecutive requests with the same id, 0 or above, make a group (those with the same id
 *                              further on another one); a negative id: no group;
 *   prefix [num_units][4] int32: for the units of a group of which two requests or more have new tokens, and whose tables
 *                              agree in 8 blocks or more before the earliest of the units: the first unit of the group,
 *                              the number of its units, the blocks that they share (a multiple of 8), 0.  Other units:
 *                              itself, 1, 0, 0; unused ones -1, 0, 0, 0.
 * The tables are compared, so a group whose requests turn out to share less is no error. */
int jetfp8_kv_prefix(const int32_t* units, int64_t num_units, const int32_t* block_table, int64_t requests,
                     int64_t max_blocks, const int32_t* groups, int32_t* prefix, void* stream);

/* jetfp8_attention, with the blocks that the units of a group share read once for all their rows.  prefix: of
 * jetfp8_kv_prefix for these units and tables (others give unspecified results of the units concerned, within the buffers).
 * The results are those of jetfp8_attention, bit for bit.  Calls that may read little (by num_units and max_seq), and those
 * with more than 32 rows (new tokens times query heads of a kv head) a unit, are made as jetfp8_attention makes them; where
 * one span of long contexts is all that is shared, a call without records is faster.  workspace:
 * jetfp8_attention_prefix_workspace() bytes: as jetfp8_attention, but for 17 to 32 rows a unit a partial result of each 8
 * blocks, where jetfp8_attention keeps one of each 64 or none. */
int jetfp8_attention_prefix(const void* q_bf16, int64_t ldq, int64_t tokens, const int32_t* units, int64_t num_units,
                            const int32_t* prefix, const int32_t* block_table, int64_t requests, int64_t max_blocks,
                            const uint8_t* codes, const float* scales, int64_t num_blocks, const void* recent_bf16,
                            int64_t recent_blocks, int64_t max_new, int64_t max_seq, int64_t q_heads, int64_t kv_heads,
                            int64_t head_dim, float softmax_scale, void* dst_o_bf16, uint8_t* dst_codes, float* dst_scales,
                            void* workspace, int64_t workspace_bytes, void* stream);

int64_t jetfp8_attention_prefix_workspace(int64_t num_units, int64_t max_new, int64_t max_seq, int64_t q_heads,
                                          int64_t kv_heads, int64_t head_dim);

/* Requests that go on from others: samples of one prompt, beams, resampled rollouts.  parents [requests] int32: request r
 * becomes a copy of request parents[r] as it is now; it stays as it is if that is r or no request, or if one of the two has
 * a recent block other than 0 or 1.  Any map will do, also one in which requests change places.  Writes, to other
 * buffers than the inputs (JETFP8_ERR_SHAPE if next_state overlaps state, or next_table block_table),
 *   next_state [requests][2]: a copy has its parent's tokens, and the one of its own recent blocks that was not in use;
 *   next_table [requests][max_blocks]: the parent's row (the request's own if it stays), -1 behind its complete blocks.
 * Per layer, jetfp8_kv_fork_recent copies the unfinished blocks.  A copy's former blocks are free after the next sweep. */
int jetfp8_kv_fork(const int32_t* state, const int32_t* block_table, int64_t max_blocks, int64_t requests,
                   const int32_t* parents, int32_t* next_state, int32_t* next_table, void* stream);

/* The recent blocks of one layer for the same parents and (former) state.  Repeating the call writes the same values. */
int jetfp8_kv_fork_recent(const int32_t* parents, const int32_t* state, int64_t requests, int64_t kv_heads,
                          int64_t head_dim, void* recent_bf16, int64_t recent_blocks, void* stream);

/* The free list anew, from what the requests hold (entries that are no block of the cache do not count):
 *   free_blocks [num_blocks] int32: the blocks that nobody holds, ascending, and -1 behind them, which ends the list for
 *                              jetfp8_kv_plan; free_head [1] int32: 0;  live [1] int32: the number L of held blocks.
 * With next_table and moves (both or neither) the cache is compacted: held blocks with ids of L and above, ascending, move
 * to the free ids below L, ascending, and the free list begins with L:
 *   next_table [requests][max_blocks] int32: the tables with the new ids, -1 behind the complete blocks; JETFP8_ERR_SHAPE
 *                              if it overlaps block_table;
 *   moves [max(1, num_blocks / 2)][2] int32: from, to; unused ones -1, -1.  Per layer, jetfp8_kv_move carries them out.
 * num_blocks <= 2^18.  workspace: jetfp8_kv_sweep_workspace() bytes (0: none). */
int jetfp8_kv_sweep(const int32_t* state, const int32_t* block_table, int64_t max_blocks, int64_t requests,
                    int64_t num_blocks, int32_t* free_blocks, int32_t* free_head, int32_t* live, int32_t* next_table,
                    int32_t* moves, void* workspace, int64_t workspace_bytes, void* stream);

int64_t jetfp8_kv_sweep_workspace(int64_t requests, int64_t max_blocks, int64_t num_blocks);

/* Copies of blocks in one layer's cache, codes and scales: moves [num_moves][2] int32, from and to.  No block may be the
 * target of two moves or both a source and a target (jetfp8_kv_sweep's are in order); moves with an id outside 0 ..
 * num_blocks - 1 are left out. */
int jetfp8_kv_move(const int32_t* moves, int64_t num_moves, int64_t kv_heads, int64_t head_dim, uint8_t* codes,
                   float* scales, int64_t num_blocks, void* stream);

/* ---- Rotary positions ---------------------------------------------------------------------------------------- */

typedef enum {                  /* the channels of pair i of a head's first 2 pairs channels */
    JETFP8_ROTARY_HALVES = 0,       /* i and pairs + i */
    JETFP8_ROTARY_INTERLEAVED = 1   /* 2 i and 2 i + 1 */
} jetfp8_rotary_layout;

/* Queries and keys turned by their tokens' positions, between the projection and jetfp8_kv_append.  Pair (a, b) number i
 * of row t turns by the angle f = positions[t] * freqs[i]:
 *   a' = amplitude * (a cos f - b sin f),   b' = amplitude * (b cos f + a sin f);
 * inverse = 1: by -f, with the same amplitude, which is the backward pass.  Channels behind the pairs stay as they are, and
 * so do rows whose position is negative (they are not written).  The angle is formed in fp64, the rest in fp32, rounded
 * once.  x: bf16, row t at x + t * ldx elements, [heads][head_dim] contiguous within a row (queries and keys of a fused
 * projection are one call); dst likewise at ldd.  dst may be x (ldd = ldx then).  head_dim % 16 == 0, at most 512;
 * pairs % 8 == 0, 2 * pairs <= head_dim; ldx, ldd >= heads * head_dim and multiples of 8.  freqs [pairs] fp64, radians for
 * each position.  0 < amplitude <= FLT_MAX (JETFP8_ERR_VALUE otherwise); an unknown layout is JETFP8_ERR_MODE. */
int jetfp8_rotary(const void* x_bf16, int64_t ldx, int64_t tokens, int64_t heads, int64_t head_dim,
                  const int32_t* positions, const double* freqs, int64_t pairs, int layout, float amplitude, int inverse,
                  void* dst_bf16, int64_t ldd, void* stream);

/* The positions of a step's rows from jetfp8_kv_plan's units in their order: positions [tokens] int32, -1 for rows of no
 * unit.  tokens <= 2^19. */
int jetfp8_kv_positions(const int32_t* units, int64_t num_units, int64_t tokens, int32_t* positions, void* stream);

/* Static, NUL-terminated description of a status code (never NULL). */
const char* jetfp8_status_string(int status);

/* Library version, major*10000 + minor*100 + patch. */
int jetfp8_version(void);

#ifdef __cplusplus
}
#endif

#endif /* JETFP8_H */
