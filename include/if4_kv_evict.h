/*
 * libif4 -- eviction from the paged IF4 KV cache (if4_kv.h) by accumulated attention weight
 * (C ABI): how much each cached token has been attended to, which tokens to keep for that,
 * and the tokens kept moved together.
 *
 * The sums ("mass") are fp32, element (row, head, j) at row * stride_row + head * stride_head
 * + j of a buffer [mass_rows, kv_heads, width]: one row per sequence, one sum per kv head
 * and token.  Sequence b of a call has row rows[b], or row b where rows is NULL; a row
 * outside [0, mass_rows) leaves the sequence out.  Sequences of one call have different
 * rows (of two with one row, the sums of either stay).  Every kv head keeps tokens of its
 * own: heads have nothing in common but their number of tokens.
 *
 * Conventions, status codes and streams are those of if4.h; what device memory holds (page
 * tables, lengths, rows, kept) is checked in the kernels as if4_kv_attention does, so that
 * no value of it makes an access outside the buffers.
 */
#ifndef IF4_KV_EVICT_H
#define IF4_KV_EVICT_H

#include "if4_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The sums, and where they go: `out` may be `in` (with its strides), and must not overlap it
 * otherwise. */
typedef struct if4_kv_mass {
    const float* in;
    int64_t in_stride_row, in_stride_head;
    float* out;
    int64_t out_stride_row, out_stride_head;
    const int32_t* rows; /* device [batch], or NULL */
    int64_t mass_rows, width;
} if4_kv_mass;

/*
 * Add the attention weights of the newest tokens of `batch` sequences.  `args` is that of
 * if4_kv_attention (out and its strides are not looked at), and P its softmax: for sequence
 * b with T_b rows of q, kv head g and key j < min(seq_lens[b], width),
 *     out[row, g, j] = (j < seq_lens[b] - T_b ? in[row, g, j] : 0) + sum_i sum_m P_imj
 * over the first max_q rows i and the query heads m of g.  The newest tokens start
 * from nothing: a slot that is used again needs no clearing.  Rows of q that see no
 * key add nothing.  A row that is NaN, or sees a key that is, makes the sums of the keys that
 * it sees NaN and no others.  Sequences without rows of q are left as they are, and so is what lies
 * at and past a sequence's length.
 * Arithmetic: the cache's values enter exactly (as 7 times theirs, in fp16), q as in
 * if4_kv_attention; scores, maxima, sums and weights are fp32, in an order that does not
 * depend on timing.
 *   workspace  device, 16-byte aligned, of if4_kv_weights_workspace() bytes; holds nothing
 *              between calls
 */
int if4_kv_weights(const if4_kv_cache* cache, const if4_kv_attention_args* args,
                   const if4_kv_mass* mass, void* workspace, int64_t workspace_bytes,
                   void* stream);

/* Bytes of workspace for these arguments (pointers are not looked at), or a negative
 * status code. */
int64_t if4_kv_weights_workspace(const if4_kv_cache* cache, const if4_kv_attention_args* args);

/* Bytes that are enough for every call with this cache's heads and no more of batch,
 * total_q, max_q and max_len than here. */
int64_t if4_kv_weights_workspace_most(const if4_kv_cache* cache, const if4_kv_attention_args* args);

/*
 * Which tokens to keep: of n = min(seq_lens[b], width) tokens the first `sinks`, the last
 * `recent`, and of those between the ones with the largest sums, `keep` in all (all n
 * where there are no more).  Equal sums go to the earlier token; NaN counts as the largest.
 *   kept     device int32 [batch, kv_heads, keep] contiguous: their positions,
 *            ascending, then -1
 *   mass     out (NULL: not wanted) gets their sums at 0, 1, ..; its width is keep or more;
 *            what lies behind stays.  It may be `in` (sequences that have one row then
 *            get any positions, or unset ones).
 *   recent + sinks <= keep
 *   workspace  device, 16-byte aligned, of if4_kv_select_workspace() bytes (NULL where that
 *              is 0); holds nothing between calls
 */
int if4_kv_select(const if4_kv_mass* mass, const int32_t* seq_lens, int64_t batch,
                  int64_t kv_heads, int64_t keep, int64_t recent, int64_t sinks, int32_t* kept,
                  void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace for these arguments (of `mass` the sizes count, no pointer), or a
 * negative status code. */
int64_t if4_kv_select_workspace(const if4_kv_mass* mass, int64_t batch, int64_t kv_heads,
                                int64_t keep);

/*
 * Copy K and V of the kept tokens: position kept[b, h, i] of sequence b and kv head h, by
 * page_table, to position i by new_table (device int32 [batch, new_stride]).  The bytes
 * are not decoded.  Pages that are written must not be read in the same call: the kept
 * tokens go to other pages, and the old ones are free afterwards.
 *   kept  device int32 [batch, kv_heads, keep]; positions outside [0, table_stride *
 *         page_size) and entries of new_table outside [0, pages) are skipped, entries of
 *         page_table outside are read as the nearest valid page
 */
int if4_kv_compact(const if4_kv_cache* cache, const int32_t* page_table, int64_t table_stride,
                   const int32_t* kept, int64_t batch, int64_t keep, const int32_t* new_table,
                   int64_t new_stride, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* IF4_KV_EVICT_H */
