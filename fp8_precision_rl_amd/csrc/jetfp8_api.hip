// C ABI of libjetfp8: host-side validation, then kernel launches on the caller's stream.
// Validation touches no HIP API, so every error path can be exercised without a GPU.
#include <float.h>
#include <stdint.h>

#include "../../include/jetfp8.h"
#include "jetfp8_launch.h"

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 31;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool dim_ok(int64_t d) { return d >= 1 && d < kMaxDim; }
int hip_status(hipError_t e) { return e == hipSuccess ? JETFP8_OK : JETFP8_ERR_HIP; }

// Shared checks of the three GEMMs: pointers, alignment, dims, and the axes that must be multiples of 128.
int check_gemm(const void* a, const void* as, const void* b, const void* bs, const void* out, int64_t d0,
               int64_t d1, int64_t d2, bool d0_grouped) {
    if (!a || !as || !b || !bs || !out) return JETFP8_ERR_NULL;
    if (!dim_ok(d0) || !dim_ok(d1) || !dim_ok(d2)) return JETFP8_ERR_SHAPE;
    if (d1 % 128 || d2 % 128 || (d0_grouped && d0 % 128)) return JETFP8_ERR_SHAPE;
    if (!aligned16(a) || !aligned16(as) || !aligned16(b) || !aligned16(bs) || !aligned16(out)) return JETFP8_ERR_ALIGN;
    return JETFP8_OK;
}

// 32-bit offset limits of the GEMM kernels (I rows and J rows of the two operands, contraction Kc): a
// block's 256-row operand band and each scale array must stay below 2^31 bytes.
int check_gemm_extent(int64_t I, int64_t J, int64_t Kc) {
    const int64_t G = Kc / 128;
    if (256 * Kc > jetfp8::kMaxGemmBand || G * I * 4 > jetfp8::kMaxGemmBand || G * J * 4 > jetfp8::kMaxGemmBand)
        return JETFP8_ERR_SHAPE;
    return JETFP8_OK;
}

// Sizes of the key/value cache that append and attention share.
bool kv_dims_ok(int64_t tokens, int64_t num_units, int64_t kv_heads, int64_t head_dim, int64_t num_blocks,
                int64_t recent_blocks) {
    return dim_ok(tokens) && dim_ok(num_units) && dim_ok(kv_heads) && (head_dim == 64 || head_dim == 128) &&
           dim_ok(num_blocks) && dim_ok(recent_blocks) && 2 * kv_heads * num_units < jetfp8::kKvMaxGrid;
}

bool row_pitch_ok(int64_t ld, int64_t heads, int64_t head_dim) {
    return dim_ok(ld) && ld % 8 == 0 && heads <= ld / head_dim;
}

bool attention_dims_ok(int64_t num_units, int64_t max_new, int64_t max_seq, int64_t q_heads, int64_t kv_heads,
                       int64_t head_dim) {
    return dim_ok(num_units) && dim_ok(max_new) && dim_ok(max_seq) && dim_ok(q_heads) && dim_ok(kv_heads) &&
           q_heads % kv_heads == 0 && q_heads <= 65536 && (head_dim == 64 || head_dim == 128) &&
           jetfp8::attention_fits(num_units, max_new, max_seq, q_heads, kv_heads);
}

}  // namespace

extern "C" {

int jetfp8_version(void) { return 401; }

const char* jetfp8_status_string(int status) {
    switch (status) {
        case JETFP8_OK: return "ok";
        case JETFP8_ERR_NULL: return "a required pointer is NULL";
        case JETFP8_ERR_SHAPE: return "bad shape: a dimension is < 1 or >= 2^31, or a grouped/contraction axis is not a multiple of 128";
        case JETFP8_ERR_ALIGN: return "a pointer is not 16-byte aligned";
        case JETFP8_ERR_MODE: return "unknown grouping mode, or a transposed-code output given for a mode without one";
        case JETFP8_ERR_HIP: return "the HIP runtime rejected a kernel launch";
        case JETFP8_ERR_VALUE: return "a scalar argument is outside its domain";
        default: return "unknown status";
    }
}

int jetfp8_quantize(const void* src_bf16, int64_t rows, int64_t cols, int mode, uint8_t* dst_codes,
                    float* dst_scales, uint8_t* dst_codes_t, void* stream) {
    if (mode != JETFP8_ROWS_1x128 && mode != JETFP8_COLS_128x1_T && mode != JETFP8_BLOCKS_128x128 &&
        mode != JETFP8_BLOCKS_128x128_FRAG)
        return JETFP8_ERR_MODE;
    if (dst_codes_t && mode != JETFP8_BLOCKS_128x128 && mode != JETFP8_BLOCKS_128x128_FRAG) return JETFP8_ERR_MODE;
    if (!src_bf16 || !dst_codes || !dst_scales) return JETFP8_ERR_NULL;
    if (!dim_ok(rows) || !dim_ok(cols)) return JETFP8_ERR_SHAPE;
    switch (mode) {
        case JETFP8_ROWS_1x128: if (cols % 128) return JETFP8_ERR_SHAPE; break;
        case JETFP8_COLS_128x1_T: if (rows % 128 || cols % 64) return JETFP8_ERR_SHAPE; break;
        default: if (rows % 128 || cols % 128) return JETFP8_ERR_SHAPE; break;
    }
    const bool fits = mode == JETFP8_ROWS_1x128 ? jetfp8::quant_rows_fits(rows, cols)
                      : mode == JETFP8_COLS_128x1_T ? jetfp8::quant_cols_t_fits(rows, cols)
                                                    : jetfp8::quant_blocks_fits(rows, cols);
    if (!fits) return JETFP8_ERR_SHAPE;
    if (!aligned16(src_bf16) || !aligned16(dst_codes) || !aligned16(dst_scales) ||
        (dst_codes_t && !aligned16(dst_codes_t)))
        return JETFP8_ERR_ALIGN;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const uint16_t* x = static_cast<const uint16_t*>(src_bf16);
    switch (mode) {
        case JETFP8_ROWS_1x128: return hip_status(jetfp8::launch_quant_rows(x, rows, cols, dst_codes, dst_scales, st));
        case JETFP8_COLS_128x1_T: return hip_status(jetfp8::launch_quant_cols_t(x, rows, cols, dst_codes, dst_scales, st));
        default: return hip_status(jetfp8::launch_quant_blocks(x, rows, cols, dst_codes, dst_scales, dst_codes_t,
                                                               mode == JETFP8_BLOCKS_128x128_FRAG, st));
    }
}

int jetfp8_quantize_dual(const void* src_bf16, int64_t rows, int64_t cols, uint8_t* dst_codes, float* dst_scales,
                         uint8_t* dst_codes_t, float* dst_scales_t, void* stream) {
    if (!src_bf16 || !dst_codes || !dst_scales || !dst_codes_t || !dst_scales_t) return JETFP8_ERR_NULL;
    if (!dim_ok(rows) || !dim_ok(cols) || rows % 128 || cols % 128) return JETFP8_ERR_SHAPE;
    if (!jetfp8::quant_dual_fits(rows, cols)) return JETFP8_ERR_SHAPE;
    if (!aligned16(src_bf16) || !aligned16(dst_codes) || !aligned16(dst_scales) || !aligned16(dst_codes_t) ||
        !aligned16(dst_scales_t))
        return JETFP8_ERR_ALIGN;
    return hip_status(jetfp8::launch_quant_dual(static_cast<const uint16_t*>(src_bf16), rows, cols, dst_codes,
                                                dst_scales, dst_codes_t, dst_scales_t,
                                                static_cast<hipStream_t>(stream)));
}

int jetfp8_requantize_cols_t(const uint8_t* codes, const float* scales, int64_t rows, int64_t cols,
                             uint8_t* dst_codes_t, float* dst_scales_t, void* stream) {
    if (!codes || !scales || !dst_codes_t || !dst_scales_t) return JETFP8_ERR_NULL;
    if (!dim_ok(rows) || !dim_ok(cols) || rows % 128 || cols % 128) return JETFP8_ERR_SHAPE;
    if (!jetfp8::quant_requant_cols_fits(rows, cols)) return JETFP8_ERR_SHAPE;
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(dst_codes_t) || !aligned16(dst_scales_t))
        return JETFP8_ERR_ALIGN;
    return hip_status(jetfp8::launch_quant_requant_cols(codes, scales, rows, cols, dst_codes_t, dst_scales_t,
                                                        static_cast<hipStream_t>(stream)));
}

int jetfp8_rmsnorm_quantize(const void* x_bf16, const void* weight_bf16, int64_t rows, int64_t cols, float eps,
                            uint8_t* dst_codes, float* dst_scales, float* dst_rstd, void* dst_y_bf16, void* stream) {
    if (!x_bf16 || !weight_bf16 || !dst_codes || !dst_scales) return JETFP8_ERR_NULL;
    if (!dim_ok(rows) || !dim_ok(cols) || cols % 128 || cols > jetfp8::kRmsNormMaxCols) return JETFP8_ERR_SHAPE;
    if (!(eps > 0.0f && eps <= FLT_MAX)) return JETFP8_ERR_VALUE;
    if (!aligned16(x_bf16) || !aligned16(weight_bf16) || !aligned16(dst_codes) || !aligned16(dst_scales) ||
        (dst_rstd && !aligned16(dst_rstd)) || (dst_y_bf16 && !aligned16(dst_y_bf16)))
        return JETFP8_ERR_ALIGN;
    return hip_status(jetfp8::launch_rmsnorm_quant(static_cast<const uint16_t*>(x_bf16),
                                                   static_cast<const uint16_t*>(weight_bf16), rows, cols, eps,
                                                   dst_codes, dst_scales, dst_rstd, static_cast<uint16_t*>(dst_y_bf16),
                                                   static_cast<hipStream_t>(stream)));
}

int jetfp8_swiglu_quantize(const void* gate_up_bf16, int64_t rows, int64_t cols, uint8_t* dst_codes,
                           float* dst_scales, void* dst_h_bf16, void* stream) {
    if (!gate_up_bf16 || !dst_codes || !dst_scales) return JETFP8_ERR_NULL;
    if (!dim_ok(rows) || !dim_ok(cols) || !dim_ok(2 * cols) || cols % 128) return JETFP8_ERR_SHAPE;
    if (!jetfp8::swiglu_quant_fits(rows, cols)) return JETFP8_ERR_SHAPE;
    if (!aligned16(gate_up_bf16) || !aligned16(dst_codes) || !aligned16(dst_scales) ||
        (dst_h_bf16 && !aligned16(dst_h_bf16)))
        return JETFP8_ERR_ALIGN;
    return hip_status(jetfp8::launch_swiglu_quant(static_cast<const uint16_t*>(gate_up_bf16), rows, cols, dst_codes,
                                                  dst_scales, static_cast<uint16_t*>(dst_h_bf16),
                                                  static_cast<hipStream_t>(stream)));
}

int jetfp8_gemm_fwd(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, void* y_bf16, int64_t M,
                    int64_t N, int64_t K, void* stream) {
    int rc = check_gemm(xq, xs, wq, ws, y_bf16, M, N, K, false);
    if (rc == JETFP8_OK) rc = check_gemm_extent(M, N, K);
    if (rc != JETFP8_OK) return rc;
    return hip_status(jetfp8::launch_gemm_block_scaled_b(xq, xs, wq, ws, static_cast<uint16_t*>(y_bf16), M, N, K,
                                                         K / 128, 1, static_cast<hipStream_t>(stream)));
}

int jetfp8_gemm_fwd_frag(const uint8_t* xq, const float* xs, const uint8_t* wq_frag, const float* ws, void* y_bf16,
                         int64_t M, int64_t N, int64_t K, void* stream) {
    int rc = check_gemm(xq, xs, wq_frag, ws, y_bf16, M, N, K, false);
    if (rc == JETFP8_OK) rc = check_gemm_extent(M, N, K);
    if (rc != JETFP8_OK) return rc;
    if (!jetfp8::gemm_fwd_frag_fits(M, K)) return JETFP8_ERR_SHAPE;
    return hip_status(jetfp8::launch_gemm_fwd_frag(xq, xs, wq_frag, ws, static_cast<uint16_t*>(y_bf16), M, N, K,
                                                   static_cast<hipStream_t>(stream)));
}

int jetfp8_gemm_dgrad(const uint8_t* dyq, const float* dys, const uint8_t* wqT, const float* ws, void* dx_bf16,
                      int64_t M, int64_t N, int64_t K, void* stream) {
    int rc = check_gemm(dyq, dys, wqT, ws, dx_bf16, M, N, K, false);
    if (rc == JETFP8_OK) rc = check_gemm_extent(M, K, N);
    if (rc != JETFP8_OK) return rc;
    return hip_status(jetfp8::launch_gemm_block_scaled_b(dyq, dys, wqT, ws, static_cast<uint16_t*>(dx_bf16), M, K, N,
                                                         1, K / 128, static_cast<hipStream_t>(stream)));
}

int jetfp8_gemm_wgrad(const uint8_t* dyqT, const float* dysT, const uint8_t* xqT, const float* xsT, void* dw_bf16,
                      int64_t M, int64_t N, int64_t K, void* stream) {
    int rc = check_gemm(dyqT, dysT, xqT, xsT, dw_bf16, M, N, K, true);
    if (rc == JETFP8_OK) rc = check_gemm_extent(N, K, M);
    if (rc != JETFP8_OK) return rc;
    return hip_status(jetfp8::launch_gemm_row_scaled_b(dyqT, dysT, xqT, xsT, static_cast<uint16_t*>(dw_bf16), N, K, M,
                                                       static_cast<hipStream_t>(stream)));
}

int64_t jetfp8_kv_max_units(int64_t tokens, int64_t requests) {
    if (tokens < 1 || tokens > jetfp8::kKvMaxTokens || requests < 1 || requests > jetfp8::kKvMaxRequests)
        return JETFP8_ERR_SHAPE;
    return jetfp8::kv_max_units(tokens, requests);
}

int jetfp8_kv_plan(const int32_t* state, const int32_t* new_lens, const int32_t* free_blocks, int64_t num_free,
                   const int32_t* free_head, int32_t* block_table, int64_t max_blocks, int64_t requests, int64_t tokens,
                   int64_t max_new, int32_t* next_state, int32_t* next_free, int32_t* status, int32_t* units,
                   int64_t* slots, void* stream) {
    // no size of a cache to go by: ids up to the type's largest, and as many recent blocks as the step may need
    return jetfp8_kv_plan_cache(state, new_lens, free_blocks, num_free, free_head, block_table, max_blocks, requests, tokens,
                                max_new, kMaxDim - 1, kMaxDim - 1, next_state, next_free, status, units, slots, stream);
}

int jetfp8_kv_plan_cache(const int32_t* state, const int32_t* new_lens, const int32_t* free_blocks, int64_t num_free,
                         const int32_t* free_head, int32_t* block_table, int64_t max_blocks, int64_t requests,
                         int64_t tokens, int64_t max_new, int64_t num_blocks, int64_t recent_blocks, int32_t* next_state,
                         int32_t* next_free, int32_t* status, int32_t* units, int64_t* slots, void* stream) {
    if (!state || !new_lens || !free_head || !block_table || !next_state || !next_free || !status || !units ||
        (!free_blocks && num_free != 0))
        return JETFP8_ERR_NULL;
    if (requests < 1 || requests > jetfp8::kKvMaxRequests || tokens < 1 || tokens > jetfp8::kKvMaxTokens ||
        !dim_ok(max_new) || !dim_ok(max_blocks) || !dim_ok(JETFP8_KV_BLOCK * max_blocks) || num_free < 0 ||
        num_free >= kMaxDim || !dim_ok(num_blocks) || !dim_ok(recent_blocks) ||
        recent_blocks < 2 * requests + tokens / JETFP8_KV_BLOCK)
        return JETFP8_ERR_SHAPE;
    if (!aligned16(state) || !aligned16(new_lens) || !aligned16(free_blocks) || !aligned16(free_head) ||
        !aligned16(block_table) || !aligned16(next_state) || !aligned16(next_free) || !aligned16(status) ||
        !aligned16(units) || !aligned16(slots))
        return JETFP8_ERR_ALIGN;
    return hip_status(jetfp8::launch_kv_plan(state, new_lens, free_blocks, num_free, free_head, block_table, max_blocks,
                                             requests, tokens, max_new, next_state, next_free, status, units, slots,
                                             num_blocks, static_cast<hipStream_t>(stream)));
}

int jetfp8_kv_append(const void* k_bf16, int64_t ldk, const void* v_bf16, int64_t ldv, int64_t tokens,
                     const int32_t* units, int64_t num_units, int64_t kv_heads, int64_t head_dim, uint8_t* codes,
                     float* scales, int64_t num_blocks, void* recent_bf16, int64_t recent_blocks, void* stream) {
    if (!k_bf16 || !v_bf16 || !units || !codes || !scales || !recent_bf16) return JETFP8_ERR_NULL;
    if (!kv_dims_ok(tokens, num_units, kv_heads, head_dim, num_blocks, recent_blocks) ||
        !row_pitch_ok(ldk, kv_heads, head_dim) || !row_pitch_ok(ldv, kv_heads, head_dim))
        return JETFP8_ERR_SHAPE;
    if (!aligned16(k_bf16) || !aligned16(v_bf16) || !aligned16(units) || !aligned16(codes) || !aligned16(scales) ||
        !aligned16(recent_bf16))
        return JETFP8_ERR_ALIGN;
    return hip_status(jetfp8::launch_kv_append(static_cast<const uint16_t*>(k_bf16), ldk,
                                               static_cast<const uint16_t*>(v_bf16), ldv, tokens, units, num_units,
                                               kv_heads, head_dim, codes, scales, num_blocks,
                                               static_cast<uint16_t*>(recent_bf16), recent_blocks,
                                               static_cast<hipStream_t>(stream)));
}

int64_t jetfp8_attention_workspace(int64_t num_units, int64_t max_new, int64_t max_seq, int64_t q_heads,
                                   int64_t kv_heads, int64_t head_dim) {
    if (!attention_dims_ok(num_units, max_new, max_seq, q_heads, kv_heads, head_dim)) return JETFP8_ERR_SHAPE;
    return jetfp8::attention_workspace(num_units, max_new, max_seq, q_heads, kv_heads, head_dim);
}

int jetfp8_attention(const void* q_bf16, int64_t ldq, int64_t tokens, const int32_t* units, int64_t num_units,
                     const int32_t* block_table, int64_t requests, int64_t max_blocks, const uint8_t* codes,
                     const float* scales, int64_t num_blocks, const void* recent_bf16, int64_t recent_blocks,
                     int64_t max_new, int64_t max_seq, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                     float softmax_scale, void* dst_o_bf16, uint8_t* dst_codes, float* dst_scales, void* workspace,
                     int64_t workspace_bytes, void* stream) {
    if (!q_bf16 || !units || !block_table || !codes || !scales || !recent_bf16 || (!dst_o_bf16 && !dst_codes) ||
        !dst_codes != !dst_scales)
        return JETFP8_ERR_NULL;
    if (!attention_dims_ok(num_units, max_new, max_seq, q_heads, kv_heads, head_dim) ||
        !kv_dims_ok(tokens, num_units, kv_heads, head_dim, num_blocks, recent_blocks) || !dim_ok(requests) ||
        !dim_ok(max_blocks) || !row_pitch_ok(ldq, q_heads, head_dim) || (dst_codes && head_dim != 128) ||
        recent_blocks < 2 * requests + tokens / JETFP8_KV_BLOCK)
        return JETFP8_ERR_SHAPE;
    if (!(softmax_scale > 0.0f && softmax_scale <= FLT_MAX / 2)) return JETFP8_ERR_VALUE;
    const int64_t need = jetfp8::attention_workspace(num_units, max_new, max_seq, q_heads, kv_heads, head_dim);
    if (need > 0 && !workspace) return JETFP8_ERR_NULL;
    if (need > workspace_bytes) return JETFP8_ERR_SHAPE;
    if (!aligned16(q_bf16) || !aligned16(units) || !aligned16(block_table) || !aligned16(codes) || !aligned16(scales) ||
        !aligned16(recent_bf16) || !aligned16(dst_o_bf16) || !aligned16(dst_codes) || !aligned16(dst_scales) ||
        !aligned16(workspace))
        return JETFP8_ERR_ALIGN;
    return hip_status(jetfp8::launch_attention(
        static_cast<const uint16_t*>(q_bf16), ldq, tokens, units, num_units, block_table, requests, max_blocks, codes,
        scales, num_blocks, static_cast<const uint16_t*>(recent_bf16), recent_blocks, max_new, max_seq, q_heads,
        kv_heads, head_dim, softmax_scale, static_cast<uint16_t*>(dst_o_bf16), dst_codes, dst_scales,
        static_cast<float*>(workspace), static_cast<hipStream_t>(stream)));
}

}  // extern "C"
