/*
 * libif4 -- paged KV cache in IF4 and the attention that reads it (C ABI).
 *
 * The cache holds the keys and values of a decoder's layer as IF4 (the format
 * of if4.h: groups of 16 along the head dimension D, one E4M3 scale byte
 * with the format flag per group, 4.5 bits per value).  It is made of `pages`
 * pages of `page_size` tokens each; slot = page * page_size + offset names
 * one token's place.  A sequence's token j lives in the slot that its row of
 * the page table gives for page j / page_size and offset j % page_size.
 *
 * Layouts (uint8, contiguous):
 *   k_codes  [pages, kv_heads, page_size, D/2]   each row as if4_quantize
 *   k_scales [pages, kv_heads, page_size, D/16]  writes it
 *   v_codes  [pages, kv_heads, page_size/16, 16, 16, D/32]
 *            (tile of 16 tokens, piece of D/16 consecutive dims, token,
 *            bytes of the piece; element 2j of the piece in the low nibble of
 *            its byte j)
 *   v_scales [pages, kv_heads, page_size/16, D/16, 16]  (tile, group, token)
 * V is tiled because the product with the probabilities contracts over tokens:
 * a matrix-core operand lane needs one piece of several consecutive tokens,
 * which this order makes one load.
 *
 * D is 64, 128 or 256 and page_size a multiple of 16 (else IF4_ERR_SHAPE).
 * Conventions, status codes and streams are those of if4.h: device pointers,
 * nothing allocated, arguments checked on the host, work only enqueued.
 * A cache's tiles of 16 tokens, pages * kv_heads * page_size / 16, fit 31 bits
 * (else IF4_ERR_SHAPE): 2^35 tokens of one head.
 * Indices that live in device memory (slots, page table, lengths) cannot be
 * checked on the host; the kernels check them as stated at each call, so that
 * no value of theirs makes an access outside the buffers.
 */
#ifndef IF4_KV_H
#define IF4_KV_H

#include "if4.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct if4_kv_cache {
    uint8_t* k_codes;  /* 16-byte aligned */
    uint8_t* k_scales; /* 16-byte aligned */
    uint8_t* v_codes;  /* 16-byte aligned */
    uint8_t* v_scales; /* 16-byte aligned */
    int64_t pages, page_size, kv_heads, head_dim;
    int32_t k_exp, v_exp; /* per-tensor powers of two E of if4_quantize, in [-64, 64] */
} if4_kv_cache;

/*
 * Write n tokens: k[t, h, :] and v[t, h, :] are quantized (rules and modes of
 * if4_quantize_mode) into slot slots[t] of every head.
 *   k, v    device, IF4_F32 or IF4_BF16, element (t, h, d) at
 *           t * stride_token + h * stride_head + d elements; 16-byte aligned
 *           and both strides multiples of 16 bytes
 *   slots   device int64 [tokens]; a slot outside [0, pages * page_size) is
 *           skipped.  Slots must differ: of two tokens written to one slot by
 *           one call, some mixture stays.
 */
int if4_kv_append(const if4_kv_cache* cache, const void* k, const void* v, int dtype,
                  int64_t tokens, int64_t k_stride_token, int64_t k_stride_head,
                  int64_t v_stride_token, int64_t v_stride_head, const int64_t* slots, int mode,
                  void* stream);

/*
 * Read n tokens back: k[t, h, :] and v[t, h, :], each [tokens, kv_heads, D]
 * contiguous, 16-byte aligned, get the values of slot slots[t] as
 * if4_dequantize gives them (fp32, or bf16 rounded to nearest even).  A slot
 * outside [0, pages * page_size) reads as zeros.
 */
int if4_kv_read(const if4_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k, void* v,
                int dtype, void* stream);

/*
 * Attention of the newest tokens of `batch` sequences over their cached keys
 * and values.  Sequence b has seq_lens[b] tokens in the cache, and its rows of
 * q are q_starts[b] .. q_starts[b + 1] - 1: T_b = their number, row i at
 * position p_i = seq_lens[b] - T_b + i (its own token is in the cache
 * already, so the last row sits at the last position).  Query head m reads
 * kv head m / (heads / kv_heads).  With S_ij = scale * <q_i, K_j> and row i
 * seeing key j iff
 *     0 <= j < seq_lens[b],
 *     not causal, or j <= p_i,
 *     window == 0, or j > p_i - window, or j < sinks,
 * out_i = sum_j softmax_j(S_ij) V_j over the keys it sees, and zeros where it
 * sees none.  Keys that a row does not see have no influence on it, NaN and
 * infinities included.
 *   q, out   device bf16, element (row, head, d) at row * stride_token +
 *            head * stride_head + d; 16-byte aligned, strides multiples of 8
 *   page_table  device int32 [batch, table_stride], entries outside
 *            [0, pages) are read as the nearest valid page;
 *            seq_lens above table_stride * page_size count as that
 *   q_starts device int32 [batch + 1], ascending, 0 .. total_q
 *   seq_lens device int32 [batch]; a length below zero counts as zero, one above
 *            2^30 - 256 as that
 *   max_q    no sequence has more rows of q than this.  Rows of out past a sequence's
 *            first max_q, before q_starts[0] and from q_starts[batch] on keep what
 *            they hold (a batch may be padded)
 *   max_len  about how long the longest sequence is (only the speed depends on it)
 *   workspace  device, 16-byte aligned, of if4_kv_attention_workspace() bytes
 *            (NULL where that is 0); holds nothing between calls
 * Arithmetic: K and V are decoded to fp16 with 2^-9 as if4_gemm decodes its
 * operands, q is taken as fp16 after an exact power of two per row and head,
 * products are summed in fp32, probabilities are rounded to fp16 for the
 * second product (their sum is that of the rounded ones; the largest of a row in a split
 * of its keys is 1 or more, and what is below 2^-25 of that counts for nothing), the
 * maximum, the sum and the output are fp32 up to the one rounding of out to bf16.
 * Results do not depend on timing.
 */
typedef struct if4_kv_attention_args {
    const void* q;
    void* out;
    int64_t q_stride_token, q_stride_head, out_stride_token, out_stride_head;
    const int32_t* page_table;
    int64_t table_stride;
    const int32_t* seq_lens;
    const int32_t* q_starts;
    int64_t batch, total_q, heads, max_q, max_len;
    int64_t window, sinks; /* >= 0; both only with causal */
    float scale;           /* finite, >= 0 */
    int32_t causal;
} if4_kv_attention_args;

int if4_kv_attention(const if4_kv_cache* cache, const if4_kv_attention_args* args, void* workspace,
                     int64_t workspace_bytes, void* stream);

/* Bytes of workspace that if4_kv_attention needs for these arguments (pointers
 * are not looked at), or a negative status code.  The keys are split to fill the
 * chip, so a smaller batch or shorter contexts can need more. */
int64_t if4_kv_attention_workspace(const if4_kv_cache* cache, const if4_kv_attention_args* args);

/* Bytes that are enough for every call with this cache's heads and head_dim, these query
 * heads, and no more of batch, total_q, max_q and max_len than here, whatever the
 * window: for a workspace that is allocated once.  A negative status code as above. */
int64_t if4_kv_attention_workspace_most(const if4_kv_cache* cache, const if4_kv_attention_args* args);

#ifdef __cplusplus
}
#endif

#endif /* IF4_KV_H */
