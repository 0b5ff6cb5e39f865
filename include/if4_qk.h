/*
 * libif4 -- norms of queries and keys for each head with the position rotation in the
 * same pass, and its gradients (C ABI): what a decoder does between its projection
 * and the cache (if4_kv.h).
 *
 * Each vector x of head_dim D values (one token, one head) becomes
 *     z = x / sqrt(mean(x^2) + eps) * weight,
 *     y = z with its first `rotary` values turned in pairs: (a, b) to
 *         (a cos - b sin, a sin + b cos),
 * pair i being values i and i + rotary/2, or 2i and 2i + 1 (interleaved), and its cosine
 * and sine `table`[position of the token][i] and [i + rotary/2].  Everything is computed
 * in fp32 and rounded once, to the output's type.
 *
 * Conventions, status codes and streams are those of if4.h: device pointers, nothing
 * allocated, arguments checked on the host, work only enqueued.  A position outside the
 * table (-1 in a padded batch) is a token that is skipped: its outputs keep what they
 * hold, its input gradients are zeros, and it adds nothing to the weights' gradients.
 */
#ifndef IF4_QK_H
#define IF4_QK_H

#include "if4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The vectors of one kind, queries or keys: element (t, h, d) at t * stride_token + h *
 * stride_head + d.  16-byte aligned, strides multiples of 16 bytes. */
typedef struct if4_qk_part {
    const void* x; /* input, of `dtype` */
    int64_t x_stride_token, x_stride_head;
    const void* g; /* backward: gradient of the output, of `out_dtype` */
    int64_t g_stride_token, g_stride_head;
    void* y; /* forward: output, of `out_dtype`; backward: gradient of x, of `dtype` */
    int64_t y_stride_token, y_stride_head;
    const float* weight; /* [head_dim], 16-byte aligned */
    float* d_weight;     /* backward: [head_dim] */
    int64_t heads;       /* 0: nothing of this kind, and no pointer is looked at */
} if4_qk_part;

typedef struct if4_qk_args {
    if4_qk_part q, k;
    const float* table;       /* device [table_rows, rotary], 16-byte aligned */
    const int64_t* positions; /* device [tokens] */
    int64_t tokens, head_dim; /* head_dim a multiple of 8 in [8, 256] */
    int64_t rotary;           /* a multiple of 16, or of 8 where interleaved, in [0, head_dim] */
    int64_t table_rows;
    float eps; /* finite, >= 0 */
    int32_t interleaved;
    int32_t dtype, out_dtype; /* IF4_F32 or IF4_BF16 */
} if4_qk_args;

/* A part's y may be its x where their types and strides are the same; otherwise no y may
 * overlap an x or the other y. */
int if4_norm_rotate(const if4_qk_args* args, void* stream);

/*
 * Gradients of x (into y) and of the weights (into d_weight, sums over tokens and heads
 * in fp32, in a fixed order) for the gradient g of the output.  y may be g or x under the
 * same condition.
 *   workspace  device, 16-byte aligned, of if4_norm_rotate_backward_workspace() bytes;
 *              holds nothing between calls
 */
int if4_norm_rotate_backward(const if4_qk_args* args, void* workspace, int64_t workspace_bytes,
                             void* stream);

/* Bytes of workspace for these sizes (pointers are not looked at), or a negative status
 * code.  No more tokens or heads need no more. */
int64_t if4_norm_rotate_backward_workspace(const if4_qk_args* args);

#ifdef __cplusplus
}
#endif

#endif /* IF4_QK_H */
