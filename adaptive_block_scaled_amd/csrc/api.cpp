// C-ABI front end of libif4: host-side validation, then one launch.
// Validation runs before any HIP call, so a bad argument never enqueues work.
#include "../../include/if4.h"

#include <math.h>
#include <stdint.h>

#include "../../include/if4_kv.h"
#include "if4_internal.h"
#include "kv_internal.h"

namespace {

constexpr int kMaxExp = 64;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

int elem_size(int dtype) { return dtype == IF4_F32 ? 4 : 2; }

int hip_status(hipError_t e) { return e == hipSuccess ? IF4_OK : IF4_ERR_HIP; }

int check_quantize(const void* x, int x_dtype, int64_t rows, int64_t cols,
                   int64_t ld_x, const uint8_t* codes, const uint8_t* scales,
                   int32_t scale_exp, int mode) {
    if (x_dtype != IF4_F32 && x_dtype != IF4_BF16) return IF4_ERR_DTYPE;
    if (mode < IF4_MODE_ADAPTIVE || mode > IF4_MODE_FORCE_INT4) return IF4_ERR_DTYPE;
    if (rows < 0 || cols < 0 || cols % 16 != 0 || ld_x < cols) return IF4_ERR_SHAPE;
    if (scale_exp < -kMaxExp || scale_exp > kMaxExp) return IF4_ERR_RANGE;
    if (rows == 0 || cols == 0) return IF4_OK;
    if (!x || !codes || !scales) return IF4_ERR_NULL;
    if (!aligned(x, 16) || (ld_x * elem_size(x_dtype)) % 16 != 0 || !aligned(codes, 8))
        return IF4_ERR_ALIGN;
    return IF4_OK;
}

// x^T quantize: groups run along dim 0, so rows (not cols) must be whole
// groups; x needs only element alignment (each lane loads single elements).
int check_quantize_t(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x,
                     const uint8_t* codes, const uint8_t* scales, int32_t scale_exp, int mode) {
    if (x_dtype != IF4_F32 && x_dtype != IF4_BF16) return IF4_ERR_DTYPE;
    if (mode < IF4_MODE_ADAPTIVE || mode > IF4_MODE_FORCE_INT4) return IF4_ERR_DTYPE;
    if (rows < 0 || cols < 0 || rows % 16 != 0 || ld_x < cols) return IF4_ERR_SHAPE;
    if (scale_exp < -kMaxExp || scale_exp > kMaxExp) return IF4_ERR_RANGE;
    if (rows == 0 || cols == 0) return IF4_OK;
    if (!x || !codes || !scales) return IF4_ERR_NULL;
    if (!aligned(x, elem_size(x_dtype)) || !aligned(codes, 8)) return IF4_ERR_ALIGN;
    return IF4_OK;
}

// Largest sizes of the KV cache's entry points: row and key indices are 32-bit
// in the kernels, kv heads are a grid dimension.
constexpr int64_t kMaxIndex = (int64_t)1 << 30;
constexpr int64_t kMaxKvHeads = 65535;

int check_cache(const if4_kv_cache& c) {
    if (c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return IF4_ERR_SHAPE;
    if (c.page_size <= 0 || c.page_size % 16 != 0 || c.page_size > kMaxIndex) return IF4_ERR_SHAPE;
    if (c.pages < 0 || c.pages > kMaxIndex) return IF4_ERR_SHAPE;
    if (c.kv_heads <= 0 || c.kv_heads > kMaxKvHeads) return IF4_ERR_SHAPE;
    // tiles of 16 tokens and one kv head: their index is 31 bits in the kernels
    if (c.pages > 0 && c.page_size / 16 * c.kv_heads > 0x7FFFFFFF / c.pages) return IF4_ERR_SHAPE;
    if (c.k_exp < -kMaxExp || c.k_exp > kMaxExp || c.v_exp < -kMaxExp || c.v_exp > kMaxExp)
        return IF4_ERR_RANGE;
    return IF4_OK;
}

int check_cache_pointers(const if4_kv_cache& c) {
    if (c.pages == 0) return IF4_OK;
    if (!c.k_codes || !c.k_scales || !c.v_codes || !c.v_scales) return IF4_ERR_NULL;
    if (!aligned(c.k_codes, 16) || !aligned(c.k_scales, 16) || !aligned(c.v_codes, 16) ||
        !aligned(c.v_scales, 16))
        return IF4_ERR_ALIGN;
    return IF4_OK;
}

int check_attention(const if4_kv_cache* cache, const if4_kv_attention_args* a) {
    if (!cache || !a) return IF4_ERR_NULL;
    const int st = check_cache(*cache);
    if (st != IF4_OK) return st;
    if (a->batch < 0 || a->total_q < 0 || a->max_q < 0 || a->max_len < 0 || a->table_stride < 0)
        return IF4_ERR_SHAPE;
    if (a->heads <= 0 || a->heads % cache->kv_heads != 0) return IF4_ERR_SHAPE;
    const int64_t group = a->heads / cache->kv_heads;
    if (a->total_q > kMaxIndex / group || a->batch > kMaxIndex / cache->kv_heads ||
        a->table_stride > kMaxIndex)
        return IF4_ERR_SHAPE;
    if (a->window < 0 || a->sinks < 0 || (!a->causal && (a->window || a->sinks)))
        return IF4_ERR_RANGE;
    if (!isfinite(a->scale) || a->scale < 0.0f) return IF4_ERR_RANGE;
    return IF4_OK;
}

// No sequence can have more rows than there are.
if4_kv_attention_args bounded(const if4_kv_attention_args& a) {
    if4_kv_attention_args r = a;
    if (r.max_q > r.total_q) r.max_q = r.total_q;
    return r;
}

}  // namespace

extern "C" {

int if4_version(void) { return 100; }

const char* if4_status_string(int status) {
    switch (status) {
        case IF4_OK: return "ok";
        case IF4_ERR_NULL: return "null pointer";
        case IF4_ERR_SHAPE: return "bad shape (negative size, cols/K not a multiple of 16, or leading dimension too small)";
        case IF4_ERR_ALIGN: return "misaligned pointer or leading dimension";
        case IF4_ERR_DTYPE: return "unknown dtype or mode";
        case IF4_ERR_RANGE: return "scale exponent outside [-64, 64]";
        case IF4_ERR_HIP: return "HIP launch failed";
        default: return "unknown status";
    }
}

int if4_quantize_mode(const void* x, int x_dtype, int64_t rows, int64_t cols,
                      int64_t ld_x, uint8_t* codes, uint8_t* scales,
                      int32_t scale_exp, int mode, void* stream) {
    int st = check_quantize(x, x_dtype, rows, cols, ld_x, codes, scales, scale_exp, mode);
    if (st != IF4_OK || rows == 0 || cols == 0) return st;
    return hip_status(if4::launch_quantize(x, x_dtype == IF4_BF16, rows, cols, ld_x, codes,
                                           scales, scale_exp, mode, (hipStream_t)stream));
}

int if4_quantize_rht(const void* x, int x_dtype, int64_t rows, int64_t cols,
                     int64_t ld_x, uint32_t sign_mask, uint8_t* codes, uint8_t* scales,
                     int32_t scale_exp, int mode, void* stream) {
    if (sign_mask > 0xFFFFu) return IF4_ERR_RANGE;
    int st = check_quantize(x, x_dtype, rows, cols, ld_x, codes, scales, scale_exp, mode);
    if (st != IF4_OK || rows == 0 || cols == 0) return st;
    return hip_status(if4::launch_quantize_rht(x, x_dtype == IF4_BF16, rows, cols, ld_x,
                                               sign_mask, codes, scales, scale_exp, mode,
                                               (hipStream_t)stream));
}

int if4_quantize_t(const void* x, int x_dtype, int64_t rows, int64_t cols,
                   int64_t ld_x, uint8_t* codes, uint8_t* scales,
                   int32_t scale_exp, int mode, void* stream) {
    int st = check_quantize_t(x, x_dtype, rows, cols, ld_x, codes, scales, scale_exp, mode);
    if (st != IF4_OK || rows == 0 || cols == 0) return st;
    return hip_status(if4::launch_quantize_t(x, x_dtype == IF4_BF16, rows, cols, ld_x, codes,
                                             scales, scale_exp, mode, (hipStream_t)stream));
}

int if4_quantize(const void* x, int x_dtype, int64_t rows, int64_t cols,
                 int64_t ld_x, uint8_t* codes, uint8_t* scales,
                 int32_t scale_exp, void* stream) {
    return if4_quantize_mode(x, x_dtype, rows, cols, ld_x, codes, scales, scale_exp,
                             IF4_MODE_ADAPTIVE, stream);
}

int if4_quantize_ifn(int bits, const void* x, int x_dtype, int64_t rows, int64_t cols,
                     int64_t ld_x, uint8_t* codes, uint8_t* scales, int32_t scale_exp, int mode,
                     void* stream) {
    if (bits != 3 && bits != 6) return IF4_ERR_DTYPE;
    int st = check_quantize(x, x_dtype, rows, cols, ld_x, codes, scales, scale_exp, mode);
    if (st != IF4_OK || rows == 0 || cols == 0) return st;
    return hip_status(if4::launch_quantize_ifn(bits, x, x_dtype == IF4_BF16, rows, cols, ld_x,
                                               codes, scales, scale_exp, mode,
                                               (hipStream_t)stream));
}

int if4_dequantize_ifn(int bits, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                       int64_t cols, int32_t scale_exp, void* y, int y_dtype, int64_t ld_y,
                       void* stream) {
    if (bits != 3 && bits != 6) return IF4_ERR_DTYPE;
    if (y_dtype != IF4_F32 && y_dtype != IF4_BF16) return IF4_ERR_DTYPE;
    if (rows < 0 || cols < 0 || cols % 16 != 0 || ld_y < cols) return IF4_ERR_SHAPE;
    if (scale_exp < -kMaxExp || scale_exp > kMaxExp) return IF4_ERR_RANGE;
    if (rows == 0 || cols == 0) return IF4_OK;
    if (!codes || !scales || !y) return IF4_ERR_NULL;
    if (!aligned(y, 16) || (ld_y * elem_size(y_dtype)) % 16 != 0 || !aligned(codes, 8))
        return IF4_ERR_ALIGN;
    return hip_status(if4::launch_dequantize_ifn(bits, codes, scales, rows, cols, scale_exp, y,
                                                 y_dtype == IF4_BF16, ld_y, (hipStream_t)stream));
}

int if4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                   int64_t cols, int32_t scale_exp, void* y, int y_dtype,
                   int64_t ld_y, void* stream) {
    if (y_dtype != IF4_F32 && y_dtype != IF4_BF16) return IF4_ERR_DTYPE;
    if (rows < 0 || cols < 0 || cols % 16 != 0 || ld_y < cols) return IF4_ERR_SHAPE;
    if (scale_exp < -kMaxExp || scale_exp > kMaxExp) return IF4_ERR_RANGE;
    if (rows == 0 || cols == 0) return IF4_OK;
    if (!codes || !scales || !y) return IF4_ERR_NULL;
    if (!aligned(y, 16) || (ld_y * elem_size(y_dtype)) % 16 != 0 || !aligned(codes, 8))
        return IF4_ERR_ALIGN;
    return hip_status(if4::launch_dequantize(codes, scales, rows, cols, scale_exp, y,
                                             y_dtype == IF4_BF16, ld_y, (hipStream_t)stream));
}

int if4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, int32_t a_exp,
             const uint8_t* w_codes, const uint8_t* w_scales, int32_t w_exp,
             int64_t M, int64_t N, int64_t K, float* c, int64_t ldc,
             void* stream) {
    if (M < 0 || N < 0 || K < 0 || K % 16 != 0 || ldc < N) return IF4_ERR_SHAPE;
    if (a_exp < -kMaxExp || a_exp > kMaxExp || w_exp < -kMaxExp || w_exp > kMaxExp)
        return IF4_ERR_RANGE;
    if (M == 0 || N == 0) return IF4_OK;
    if (!c) return IF4_ERR_NULL;
    if (K > 0 && (!a_codes || !a_scales || !w_codes || !w_scales)) return IF4_ERR_NULL;
    if (!aligned(c, 4) || (K > 0 && (!aligned(a_codes, 8) || !aligned(w_codes, 8))))
        return IF4_ERR_ALIGN;
    return hip_status(if4::launch_gemm(a_codes, a_scales, a_exp, w_codes, w_scales, w_exp, M,
                                       N, K, c, ldc, (hipStream_t)stream));
}

int if4_kv_append(const if4_kv_cache* cache, const void* k, const void* v, int dtype,
                  int64_t tokens, int64_t k_stride_token, int64_t k_stride_head,
                  int64_t v_stride_token, int64_t v_stride_head, const int64_t* slots, int mode,
                  void* stream) {
    if (!cache) return IF4_ERR_NULL;
    if (dtype != IF4_F32 && dtype != IF4_BF16) return IF4_ERR_DTYPE;
    if (mode < IF4_MODE_ADAPTIVE || mode > IF4_MODE_FORCE_INT4) return IF4_ERR_DTYPE;
    int st = check_cache(*cache);
    if (st != IF4_OK) return st;
    if (tokens < 0) return IF4_ERR_SHAPE;
    if (tokens == 0) return IF4_OK;
    if (!k || !v || !slots) return IF4_ERR_NULL;
    st = check_cache_pointers(*cache);
    if (st != IF4_OK) return st;
    const int64_t strides[4] = {k_stride_token, k_stride_head, v_stride_token, v_stride_head};
    for (int64_t s : strides)
        if (s * elem_size(dtype) % 16 != 0) return IF4_ERR_ALIGN;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return IF4_ERR_ALIGN;
    if (cache->pages == 0) return IF4_OK;
    return hip_status(if4::launch_kv_append(*cache, k, v, dtype == IF4_BF16, tokens, strides, slots,
                                            mode, (hipStream_t)stream));
}

int if4_kv_read(const if4_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k, void* v,
                int dtype, void* stream) {
    if (!cache) return IF4_ERR_NULL;
    if (dtype != IF4_F32 && dtype != IF4_BF16) return IF4_ERR_DTYPE;
    int st = check_cache(*cache);
    if (st != IF4_OK) return st;
    if (tokens < 0) return IF4_ERR_SHAPE;
    if (tokens == 0) return IF4_OK;
    if (!k || !v || !slots) return IF4_ERR_NULL;
    st = check_cache_pointers(*cache);
    if (st != IF4_OK) return st;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return IF4_ERR_ALIGN;
    return hip_status(if4::launch_kv_read(*cache, slots, tokens, k, v, dtype == IF4_BF16,
                                          (hipStream_t)stream));
}

int64_t if4_kv_attention_workspace(const if4_kv_cache* cache, const if4_kv_attention_args* args) {
    const int st = check_attention(cache, args);
    if (st != IF4_OK) return -st;
    const if4_kv_attention_args a = bounded(*args);
    if (a.batch == 0 || a.max_q == 0) return 0;
    return if4::kv_attention_workspace(*cache, a);
}

int64_t if4_kv_attention_workspace_most(const if4_kv_cache* cache, const if4_kv_attention_args* args) {
    const int st = check_attention(cache, args);
    if (st != IF4_OK) return -st;
    const if4_kv_attention_args a = bounded(*args);
    if (a.batch == 0 || a.max_q == 0) return 0;
    return if4::kv_attention_workspace_most(*cache, a);
}

int if4_kv_attention(const if4_kv_cache* cache, const if4_kv_attention_args* args, void* workspace,
                     int64_t workspace_bytes, void* stream) {
    int st = check_attention(cache, args);
    if (st != IF4_OK) return st;
    const if4_kv_attention_args a = bounded(*args);
    if (a.batch == 0 || a.max_q == 0) return IF4_OK;
    if (!a.q || !a.out || !a.seq_lens || !a.q_starts) return IF4_ERR_NULL;
    if (a.table_stride > 0 && !a.page_table) return IF4_ERR_NULL;
    st = check_cache_pointers(*cache);
    if (st != IF4_OK) return st;
    if (!aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.page_table, 4) ||
        !aligned(a.seq_lens, 4) || !aligned(a.q_starts, 4))
        return IF4_ERR_ALIGN;
    if (a.q_stride_token % 8 || a.q_stride_head % 8 || a.out_stride_token % 8 ||
        a.out_stride_head % 8)
        return IF4_ERR_ALIGN;
    const int64_t need = if4::kv_attention_workspace(*cache, a);
    if (need > 0 && !workspace) return IF4_ERR_NULL;
    if (need > workspace_bytes) return IF4_ERR_SHAPE;
    if (!aligned(workspace, 16)) return IF4_ERR_ALIGN;
    return hip_status(if4::launch_kv_attention(*cache, a, workspace, (hipStream_t)stream));
}

}  // extern "C"
