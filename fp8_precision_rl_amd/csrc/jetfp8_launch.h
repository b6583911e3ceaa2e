// Host-side launchers of the libjetfp8 kernels (shapes are validated by the C ABI layer before these run).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace jetfp8 {

// The GEMM kernels address a block's operand band (256 rows x contraction bytes) and a scale array
// (groups x rows x 4 bytes) through 32-bit buffer offsets; the C ABI rejects shapes beyond this.
constexpr int64_t kMaxGemmBand = ((int64_t)1 << 31) - 1;

// Size limits of each kernel's launch grid and of its 32-bit buffer offsets.  The C ABI checks these on the host
// (JETFP8_ERR_SHAPE) before calling a launcher; the launchers assume them.
bool quant_rows_fits(int64_t R, int64_t C);
bool quant_cols_t_fits(int64_t R, int64_t C);
bool quant_dual_fits(int64_t R, int64_t C);
bool quant_requant_cols_fits(int64_t R, int64_t C);
bool quant_blocks_fits(int64_t R, int64_t C);
bool swiglu_quant_fits(int64_t R, int64_t F);

hipError_t launch_quant_rows(const uint16_t* x, int64_t R, int64_t C, uint8_t* q, float* s, hipStream_t st);
hipError_t launch_quant_cols_t(const uint16_t* x, int64_t R, int64_t C, uint8_t* qT, float* sT, hipStream_t st);
hipError_t launch_quant_dual(const uint16_t* x, int64_t R, int64_t C, uint8_t* q, float* s, uint8_t* qT, float* sT,
                             hipStream_t st);
hipError_t launch_quant_requant_cols(const uint8_t* q, const float* s, int64_t R, int64_t C, uint8_t* qT,
                                     float* sT, hipStream_t st);
// Fused producers (1x128 codes of the produced bf16 activation).  RMSNorm holds a row in registers: at most
// kRmsNormMaxCols columns.
constexpr int64_t kRmsNormMaxCols = 8192;
hipError_t launch_rmsnorm_quant(const uint16_t* x, const uint16_t* w, int64_t R, int64_t C, float eps, uint8_t* q,
                                float* s, float* rstd, uint16_t* y, hipStream_t st);
hipError_t launch_rmsnorm_add_quant(const uint16_t* x, const uint16_t* res, const uint16_t* w, int64_t R, int64_t C,
                                    float eps, uint16_t* h, uint8_t* q, float* s, float* rstd, uint16_t* y,
                                    hipStream_t st);
int64_t rmsnorm_backward_workspace(int64_t R, int64_t C);
hipError_t launch_rmsnorm_backward(const uint16_t* dy, const uint16_t* h, const uint16_t* w, const float* rstd,
                                   const uint16_t* dres, int64_t R, int64_t C, uint16_t* dx, float* dw, float* workspace,
                                   hipStream_t st);
hipError_t launch_swiglu_quant(const uint16_t* gu, int64_t R, int64_t F, uint8_t* q, float* s, uint16_t* h,
                               hipStream_t st);
// frag = true: q in the fragment order of JETFP8_BLOCKS_128x128_FRAG instead of row-major.
hipError_t launch_quant_blocks(const uint16_t* x, int64_t R, int64_t C, uint8_t* q, float* s, uint8_t* qT, bool frag,
                               hipStream_t st);

// C[i][j] = sum_g As[g][i] * sb(j, g) * sum_{k in g} A[i][k] * B[j][k], A [I][Kc], B [J][Kc].
// Block-scaled B: sb(j, g) = Bs[(j / 128) * sbj + g * sbg].  Row-scaled B: sb(j, g) = Bs[g * J + j].
hipError_t launch_gemm_block_scaled_b(const uint8_t* A, const float* As, const uint8_t* B, const float* Bs,
                                      uint16_t* C, int64_t I, int64_t J, int64_t Kc, int64_t sbj, int64_t sbg,
                                      hipStream_t st);
// Rows r0 .. r0 + rows - 1 of a block-scaled-B GEMM with I rows on the small-M kernel (decode_rows_fit(rows, Kc)).
bool decode_rows_fit(int64_t rows, int64_t Kc);
hipError_t launch_decode_rows(const uint8_t* A, const float* As, const uint8_t* B, const float* Bs, uint16_t* C,
                              int64_t I, int64_t r0, int64_t rows, int64_t J, int64_t Kc, int64_t sbj, int64_t sbg,
                              hipStream_t st);
// Forward GEMM with the weight codes in the fragment order of JETFP8_BLOCKS_128x128_FRAG (small-M kernel only:
// M <= 64 and (K / 128) * M <= 8192, checked by gemm_fwd_frag_fits).
bool gemm_fwd_frag_fits(int64_t M, int64_t K);
hipError_t launch_gemm_fwd_frag(const uint8_t* xq, const float* xs, const uint8_t* wqf, const float* ws, uint16_t* y,
                                int64_t M, int64_t N, int64_t K, hipStream_t st);
// The FP8 key/value cache: a step's plan, the append of its keys and values, and the attention over the cache.
constexpr int64_t kKvMaxRequests = 4096;            // three prefix sums of a request are kept in LDS
constexpr int64_t kKvMaxGrid = (int64_t)1 << 24;    // a launch holds fewer than 2^32 threads, 256 to a thread block
constexpr int64_t kKvMaxTokens = (int64_t)1 << 19;  // sums over 4096 requests stay below 2^32
int64_t kv_max_units(int64_t tokens, int64_t requests);
hipError_t launch_kv_plan(const int32_t* state, const int32_t* new_lens, const int32_t* free_blocks, int64_t num_free,
                          const int32_t* free_head, int32_t* table, int64_t width, int64_t requests, int64_t tokens,
                          int64_t max_new, int32_t* next_state, int32_t* next_free, int32_t* status, int32_t* units,
                          int64_t* slots, int64_t num_blocks, hipStream_t st);
hipError_t launch_kv_append(const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv, int64_t tokens,
                            const int32_t* units, int64_t num_units, int64_t heads, int64_t D, uint8_t* codes,
                            float* scales, int64_t num_blocks, uint16_t* recent, int64_t recent_blocks, hipStream_t st);
// Bytes of workspace, and whether the launch grids hold the call.  prefix: with records of the blocks that units share.
int64_t attention_workspace(int64_t num_units, int64_t max_new, int64_t max_seq, int64_t q_heads, int64_t kv_heads,
                            int64_t D, bool prefix);
bool attention_fits(int64_t num_units, int64_t max_new, int64_t max_seq, int64_t q_heads, int64_t kv_heads, int64_t D,
                    bool prefix);
hipError_t launch_attention(const uint16_t* q, int64_t ldq, int64_t tokens, const int32_t* units, int64_t num_units,
                            const int32_t* prefix, const int32_t* table, int64_t requests, int64_t width,
                            const uint8_t* codes, const float* scales, int64_t num_blocks, const uint16_t* recent,
                            int64_t recent_blocks, int64_t max_new, int64_t max_seq, int64_t q_heads, int64_t kv_heads,
                            int64_t D, float softmax_scale, uint16_t* o, uint8_t* oq, float* os, float* workspace,
                            hipStream_t st);
// Page operations of the cache (jetfp8_pages.hip).
constexpr int64_t kKvMaxSweepBlocks = (int64_t)1 << 18;      // marks and counts of that many blocks fit 64 KB of LDS
hipError_t launch_kv_positions(const int32_t* units, int64_t num_units, int64_t tokens, int32_t* positions, hipStream_t st);
hipError_t launch_kv_prefix(const int32_t* units, int64_t num_units, const int32_t* table, int64_t requests, int64_t width,
                            const int32_t* groups, int32_t* prefix, hipStream_t st);
hipError_t launch_kv_fork(const int32_t* state, const int32_t* table, int64_t width, int64_t requests,
                          const int32_t* parents, int32_t* next_state, int32_t* next_table, hipStream_t st);
hipError_t launch_kv_fork_recent(const int32_t* parents, const int32_t* state, int64_t requests, int64_t heads, int64_t D,
                                 uint16_t* recent, hipStream_t st);
int64_t kv_sweep_workspace(int64_t requests, int64_t width, int64_t num_blocks);
hipError_t launch_kv_sweep(const int32_t* state, const int32_t* table, int64_t width, int64_t requests, int64_t num_blocks,
                           int32_t* free_blocks, int32_t* free_head, int32_t* live, int32_t* next_table, int32_t* moves,
                           uint64_t* workspace, hipStream_t st);
hipError_t launch_kv_move(const int32_t* moves, int64_t num_moves, int64_t heads, int64_t D, uint8_t* codes, float* scales,
                          int64_t num_blocks, hipStream_t st);
// Rotary positions: P = pairs of a head's first 2 P channels; a head has at most kRotaryMaxDim channels.
constexpr int64_t kRotaryMaxDim = 512;
bool rotary_fits(int64_t tokens, int64_t heads);      // the launch grid
hipError_t launch_rotary(const uint16_t* x, int64_t ldx, int64_t tokens, int64_t heads, int64_t D, const int32_t* positions,
                         const double* freqs, int64_t pairs, bool interleaved, float amplitude, bool inverse,
                         uint16_t* out, int64_t ldo, hipStream_t st);
hipError_t launch_gemm_row_scaled_b(const uint8_t* A, const float* As, const uint8_t* B, const float* Bs,
                                    uint16_t* C, int64_t I, int64_t J, int64_t Kc, hipStream_t st);

}  // namespace jetfp8
