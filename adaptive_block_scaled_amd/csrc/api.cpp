// C-ABI front end of libif4: host-side validation, then one launch.
// Validation runs before any HIP call, so a bad argument never enqueues work.
#include "../../include/if4.h"

#include <math.h>
#include <stdint.h>

#include "../../include/if4_fp8.h"
#include "../../include/if4_kv.h"
#include "../../include/if4_kv_evict.h"
#include "fp8_internal.h"
#include "if4_internal.h"
#include "kv_evict_internal.h"
#include "kv_internal.h"
#include "qk_internal.h"

namespace {

constexpr int kMaxExp = 64;

// Largest sizes of the FP8 entry points and of if4_norm_rotate.
constexpr int64_t kMaxSize = (int64_t)1 << 31, kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxK = (int64_t)1 << 22;
// Most heads of one kind that if4_norm_rotate takes.
constexpr int64_t kMaxHeads = 65535;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

int elem_size(int dtype) { return dtype == IF4_F32 ? 4 : 2; }

// (an invalid configuration: more workgroups than one launch holds, see launch_limit.h)
int hip_status(hipError_t e) {
    return e == hipSuccess ? IF4_OK : e == hipErrorInvalidConfiguration ? IF4_ERR_SHAPE : IF4_ERR_HIP;
}

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

// The contraction dimension, `along`, holds whole groups of 16; blocks (of one row or
// square) are a grid dimension.
int check_fp8_quantize(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x,
                       int64_t along, int64_t others, int square, const uint8_t* codes,
                       const uint8_t* scales) {
    if (x_dtype != IF4_F32 && x_dtype != IF4_BF16) return IF4_ERR_DTYPE;
    if (square != 0 && square != 1) return IF4_ERR_DTYPE;
    if (rows < 0 || cols < 0 || along % 16 != 0 || ld_x < cols) return IF4_ERR_SHAPE;
    if (rows > kMaxSize || cols > kMaxSize || ld_x > kMaxStride) return IF4_ERR_SHAPE;
    if (rows == 0 || cols == 0) return IF4_OK;
    const int64_t blocks = (along + IF4_FP8_BLOCK - 1) / IF4_FP8_BLOCK;
    if (others > 0x7FFFFFFF / blocks) return IF4_ERR_SHAPE;
    if (!x || !codes || !scales) return IF4_ERR_NULL;
    if (!aligned(x, 16) || (ld_x * elem_size(x_dtype)) % 16 != 0 || !aligned(codes, 16))
        return IF4_ERR_ALIGN;
    return IF4_OK;
}

int check_qk_part(const if4_qk_part& p, int64_t tokens, int size, int out_size, bool backward) {
    if (p.heads == 0) return IF4_OK;
    if (tokens > 0 && (!p.x || !p.y || (backward && !p.g))) return IF4_ERR_NULL;
    if (!p.weight || (backward && !p.d_weight)) return IF4_ERR_NULL;
    const int y_size = backward ? size : out_size;
    if (!aligned(p.x, 16) || !aligned(p.y, 16) || !aligned(p.weight, 16)) return IF4_ERR_ALIGN;
    if (backward && (!aligned(p.g, 16) || !aligned(p.d_weight, 4))) return IF4_ERR_ALIGN;
    if (p.x_stride_token * size % 16 || p.x_stride_head * size % 16 ||
        p.y_stride_token * y_size % 16 || p.y_stride_head * y_size % 16)
        return IF4_ERR_ALIGN;
    if (backward && (p.g_stride_token * out_size % 16 || p.g_stride_head * out_size % 16))
        return IF4_ERR_ALIGN;
    return IF4_OK;
}

int check_qk_sizes(const if4_qk_args& a) {
    for (int t : {a.dtype, a.out_dtype})
        if (t != IF4_F32 && t != IF4_BF16) return IF4_ERR_DTYPE;
    if (a.interleaved != 0 && a.interleaved != 1) return IF4_ERR_DTYPE;
    if (a.head_dim < 8 || a.head_dim > 256 || a.head_dim % 8) return IF4_ERR_SHAPE;
    if (a.rotary < 0 || a.rotary > a.head_dim || a.rotary % (a.interleaved ? 8 : 16))
        return IF4_ERR_SHAPE;
    if (a.tokens < 0 || a.tokens > kMaxSize || a.table_rows < 0 || a.table_rows > kMaxSize)
        return IF4_ERR_SHAPE;
    for (int64_t h : {a.q.heads, a.k.heads})
        if (h < 0 || h > kMaxHeads) return IF4_ERR_SHAPE;
    if (!isfinite(a.eps) || a.eps < 0.0f) return IF4_ERR_RANGE;
    return IF4_OK;
}

int check_qk(const if4_qk_args& a, bool backward) {
    int st = check_qk_sizes(a);
    if (st != IF4_OK) return st;
    const int size = elem_size(a.dtype), out_size = elem_size(a.out_dtype);
    for (const if4_qk_part* p : {&a.q, &a.k})
        if ((st = check_qk_part(*p, a.tokens, size, out_size, backward)) != IF4_OK) return st;
    if (a.tokens > 0 && a.q.heads + a.k.heads > 0) {
        if (!a.positions || (a.rotary > 0 && a.table_rows > 0 && !a.table)) return IF4_ERR_NULL;
        if (!aligned(a.positions, 8) || !aligned(a.table, 16)) return IF4_ERR_ALIGN;
    }
    return IF4_OK;
}

// Sizes that the FP8 product's kernels index: rows of a tile by K in 31 bits.
int check_fp8_gemm_sizes(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0 || K % 16 != 0) return IF4_ERR_SHAPE;
    if (M > kMaxSize || N > kMaxSize || K > kMaxK) return IF4_ERR_SHAPE;
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

// The sums of a call: `in` is read, `out` written where it is not NULL.
int check_mass(const if4_kv_mass& m, int64_t batch, bool out_needed) {
    if (m.mass_rows < 0 || m.mass_rows > kMaxIndex || m.width < 0 || m.width > kMaxIndex)
        return IF4_ERR_SHAPE;
    if (!m.rows && m.mass_rows < batch) return IF4_ERR_SHAPE;
    if (m.mass_rows == 0 || m.width == 0) return IF4_OK;
    if (!m.in || (out_needed && !m.out)) return IF4_ERR_NULL;
    if (!aligned(m.in, 4) || !aligned(m.out, 4) || !aligned(m.rows, 4)) return IF4_ERR_ALIGN;
    return IF4_OK;
}

int check_select(const if4_kv_mass& m, int64_t batch, int64_t kv_heads, int64_t keep) {
    if (m.mass_rows < 0 || m.mass_rows > kMaxIndex || m.width < 0 || m.width > kMaxIndex)
        return IF4_ERR_SHAPE;
    if (batch < 0 || kv_heads <= 0 || kv_heads > kMaxKvHeads || batch > 0x7FFFFFFF / kv_heads)
        return IF4_ERR_SHAPE;
    return keep < 0 || keep > kMaxIndex ? IF4_ERR_SHAPE : IF4_OK;
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
        case IF4_ERR_SHAPE: return "bad shape (negative size, cols/K not a multiple of 16, or leading dimension too small, or more than one launch holds)";
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

int if4_fp8_quantize(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x,
                     int square, uint8_t* codes, uint8_t* scales, void* stream) {
    const int st = check_fp8_quantize(x, x_dtype, rows, cols, ld_x, cols, rows, square, codes, scales);
    if (st != IF4_OK || rows == 0 || cols == 0) return st;
    return hip_status(if4::launch_fp8_quantize(x, x_dtype == IF4_BF16, rows, cols, ld_x, square,
                                               codes, scales, (hipStream_t)stream));
}

int if4_fp8_quantize_t(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ld_x,
                       int square, uint8_t* codes, uint8_t* scales, void* stream) {
    const int st = check_fp8_quantize(x, x_dtype, rows, cols, ld_x, rows, cols, square, codes, scales);
    if (st != IF4_OK || rows == 0 || cols == 0) return st;
    return hip_status(if4::launch_fp8_quantize_t(x, x_dtype == IF4_BF16, rows, cols, ld_x, square,
                                                 codes, scales, (hipStream_t)stream));
}

int64_t if4_fp8_gemm_workspace(int64_t M, int64_t N, int64_t K) {
    const int st = check_fp8_gemm_sizes(M, N, K);
    if (st != IF4_OK) return -st;
    return M == 0 || N == 0 || K == 0 ? 0 : if4::fp8_gemm_workspace(M, N, K);
}

int if4_fp8_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* w_codes,
                 const uint8_t* w_scales, int w_square, int64_t M, int64_t N, int64_t K, void* c,
                 int c_dtype, int64_t ldc, void* workspace, int64_t workspace_bytes,
                 void* stream) {
    if (c_dtype != IF4_F32 && c_dtype != IF4_BF16) return IF4_ERR_DTYPE;
    if (w_square != 0 && w_square != 1) return IF4_ERR_DTYPE;
    const int st = check_fp8_gemm_sizes(M, N, K);
    if (st != IF4_OK) return st;
    if (ldc < N || ldc > kMaxStride) return IF4_ERR_SHAPE;
    if (M == 0 || N == 0) return IF4_OK;
    if (!c || (K > 0 && (!a_codes || !a_scales || !w_codes || !w_scales))) return IF4_ERR_NULL;
    if (!aligned(c, elem_size(c_dtype)) ||
        (K > 0 && (!aligned(a_codes, 16) || !aligned(w_codes, 16))))
        return IF4_ERR_ALIGN;
    const int64_t need = K > 0 ? if4::fp8_gemm_workspace(M, N, K) : 0;
    if (need > 0 && !workspace) return IF4_ERR_NULL;
    if (need > workspace_bytes) return IF4_ERR_SHAPE;
    if (need > 0 && !aligned(workspace, 16)) return IF4_ERR_ALIGN;
    return hip_status(if4::launch_fp8_gemm({a_codes, a_scales, w_codes, w_scales, w_square, M, N, K,
                                            c, c_dtype == IF4_BF16, ldc, workspace},
                                           (hipStream_t)stream));
}

int if4_norm_rotate(const if4_qk_args* args, void* stream) {
    if (!args) return IF4_ERR_NULL;
    const int st = check_qk(*args, false);
    if (st != IF4_OK || args->tokens == 0 || args->q.heads + args->k.heads == 0) return st;
    return hip_status(if4::launch_norm_rotate(*args, (hipStream_t)stream));
}

int64_t if4_norm_rotate_backward_workspace(const if4_qk_args* args) {
    if (!args) return -IF4_ERR_NULL;
    const int st = check_qk_sizes(*args);
    return st != IF4_OK ? -st : if4::norm_rotate_backward_workspace(*args);
}

int if4_norm_rotate_backward(const if4_qk_args* args, void* workspace, int64_t workspace_bytes,
                             void* stream) {
    if (!args) return IF4_ERR_NULL;
    const int st = check_qk(*args, true);
    if (st != IF4_OK || args->q.heads + args->k.heads == 0) return st;
    if (!workspace) return IF4_ERR_NULL;
    if (workspace_bytes < if4::norm_rotate_backward_workspace(*args)) return IF4_ERR_SHAPE;
    if (!aligned(workspace, 16)) return IF4_ERR_ALIGN;
    return hip_status(if4::launch_norm_rotate_backward(*args, workspace, (hipStream_t)stream));
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

int64_t if4_kv_weights_workspace(const if4_kv_cache* cache, const if4_kv_attention_args* args) {
    const int st = check_attention(cache, args);
    if (st != IF4_OK) return -st;
    const if4_kv_attention_args a = bounded(*args);
    return a.batch == 0 || a.max_q == 0 ? 0 : if4::kv_weights_workspace(*cache, a);
}

int64_t if4_kv_weights_workspace_most(const if4_kv_cache* cache, const if4_kv_attention_args* args) {
    const int st = check_attention(cache, args);
    if (st != IF4_OK) return -st;
    const if4_kv_attention_args a = bounded(*args);
    return a.batch == 0 || a.max_q == 0 ? 0 : if4::kv_weights_workspace_most(*cache, a);
}

int if4_kv_weights(const if4_kv_cache* cache, const if4_kv_attention_args* args,
                   const if4_kv_mass* mass, void* workspace, int64_t workspace_bytes,
                   void* stream) {
    int st = check_attention(cache, args);
    if (st != IF4_OK) return st;
    if (!mass) return IF4_ERR_NULL;
    const if4_kv_attention_args a = bounded(*args);
    st = check_mass(*mass, a.batch, true);
    if (st != IF4_OK) return st;
    if (a.batch == 0 || a.max_q == 0) return IF4_OK;
    if (!a.q || !a.seq_lens || !a.q_starts) return IF4_ERR_NULL;
    if (a.table_stride > 0 && !a.page_table) return IF4_ERR_NULL;
    st = check_cache_pointers(*cache);
    if (st != IF4_OK) return st;
    if (!aligned(a.q, 16) || !aligned(a.page_table, 4) || !aligned(a.seq_lens, 4) ||
        !aligned(a.q_starts, 4) || a.q_stride_token % 8 || a.q_stride_head % 8)
        return IF4_ERR_ALIGN;
    const int64_t need = if4::kv_weights_workspace(*cache, a);
    if (!workspace) return IF4_ERR_NULL;
    if (need > workspace_bytes) return IF4_ERR_SHAPE;
    if (!aligned(workspace, 16)) return IF4_ERR_ALIGN;
    // no token has a place
    if (cache->pages == 0 || a.table_stride == 0 || mass->mass_rows == 0 || mass->width == 0)
        return IF4_OK;
    return hip_status(if4::launch_kv_weights(*cache, a, *mass, workspace, (hipStream_t)stream));
}

int64_t if4_kv_select_workspace(const if4_kv_mass* mass, int64_t batch, int64_t kv_heads,
                                int64_t keep) {
    if (!mass) return -IF4_ERR_NULL;
    const int st = check_select(*mass, batch, kv_heads, keep);
    if (st != IF4_OK) return -st;
    return batch == 0 || keep == 0 ? 0 : if4::kv_select_workspace(*mass, batch, kv_heads, keep);
}

int if4_kv_select(const if4_kv_mass* mass, const int32_t* seq_lens, int64_t batch,
                  int64_t kv_heads, int64_t keep, int64_t recent, int64_t sinks, int32_t* kept,
                  void* workspace, int64_t workspace_bytes, void* stream) {
    if (!mass) return IF4_ERR_NULL;
    int st = check_select(*mass, batch, kv_heads, keep);
    if (st != IF4_OK) return st;
    if (recent < 0 || sinks < 0 || recent > keep || sinks > keep - recent) return IF4_ERR_RANGE;
    st = check_mass(*mass, batch, false);
    if (st != IF4_OK) return st;
    if (batch == 0 || keep == 0) return IF4_OK;
    if (!seq_lens || !kept) return IF4_ERR_NULL;
    if (!aligned(seq_lens, 4) || !aligned(kept, 4)) return IF4_ERR_ALIGN;
    const int64_t need = if4::kv_select_workspace(*mass, batch, kv_heads, keep);
    if (need > 0 && !workspace) return IF4_ERR_NULL;
    if (need > workspace_bytes) return IF4_ERR_SHAPE;
    if (need > 0 && !aligned(workspace, 16)) return IF4_ERR_ALIGN;
    return hip_status(if4::launch_kv_select(*mass, seq_lens, batch, kv_heads, keep, recent, sinks,
                                            kept, workspace, (hipStream_t)stream));
}

int if4_kv_compact(const if4_kv_cache* cache, const int32_t* page_table, int64_t table_stride,
                   const int32_t* kept, int64_t batch, int64_t keep, const int32_t* new_table,
                   int64_t new_stride, void* stream) {
    if (!cache) return IF4_ERR_NULL;
    int st = check_cache(*cache);
    if (st != IF4_OK) return st;
    if (batch < 0 || keep < 0 || keep > kMaxIndex || table_stride < 0 || table_stride > kMaxIndex ||
        new_stride < 0 || new_stride > kMaxIndex)
        return IF4_ERR_SHAPE;
    // workgroups, one for 16 tokens of a kv head, are a grid dimension
    if (batch > 0x7FFFFFFF / cache->kv_heads ||
        (batch > 0 && (keep + 15) / 16 > 0x7FFFFFFF / (batch * cache->kv_heads)))
        return IF4_ERR_SHAPE;
    if (batch == 0 || keep == 0 || table_stride == 0 || new_stride == 0 || cache->pages == 0)
        return IF4_OK;
    if (!page_table || !kept || !new_table) return IF4_ERR_NULL;
    st = check_cache_pointers(*cache);
    if (st != IF4_OK) return st;
    if (!aligned(page_table, 4) || !aligned(kept, 4) || !aligned(new_table, 4)) return IF4_ERR_ALIGN;
    return hip_status(if4::launch_kv_compact(*cache, page_table, table_stride, kept, batch, keep,
                                             new_table, new_stride, (hipStream_t)stream));
}

}  // extern "C"
