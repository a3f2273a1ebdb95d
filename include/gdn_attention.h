/*
 * gdn_attention.h -- the operators of the full-attention layers of a hybrid model, in libgdn.so
 * beside gdn.h and gdn_layer.h.
 *
 * Between the recurrent layers stand attention layers over a paged key/value cache.  They
 * take the maps that gdn_step_plan makes (token_position, token_kv_slot, and the block
 * tables it was given) and the same packed sequences and decode rows:
 *
 *   gdn_rotary              rotary positions of q and k
 *   gdn_kv_cache_write,
 *   gdn_kv_cache_read       keys and values into cache rows, in the activations' dtype or
 *                           quantised to 8 bits for each head of a token, and back
 *   gdn_attention_prefill   causal attention of packed prompts over their cached keys
 *   gdn_attention_decode    attention of one token, a chain or a tree of drafted tokens of
 *                           each cached row
 *
 * A step writes its tokens' keys and values into the cache first; the attention reads all
 * keys there, the step's own among them.
 *
 * The conventions of gdn.h and gdn_layer.h hold here too (caller-owned device memory, nothing
 * allocated, work only enqueued on `stream`, no synchronisation, capturable, host arguments
 * validated before anything is enqueued, gdn_last_error() for the message, row strides in
 * elements, at most 2^32 - 1 threads a launch).  Differences and additions:
 *   Slots       A cache row outside [0, num_rows), or a page that has a negative entry, lies
 *               past its table or reaches past the cache, is absent: never read or written, and
 *               seen by no token.  Within one call no cache row may be written twice.
 *   Arithmetic  Scores, softmax statistics, sums and scales are fp32.  With bf16 activations
 *               the softmax's weights, times the value's scale where there is one, are rounded
 *               to bf16 on their way into the matrix cores, by at most 2^-8 of each; 8-bit
 *               codes are exact there.  Over a plain cache the rounded weights are summed, so
 *               that the rounding of a key that has nearly all of the weight cancels.  With fp32
 *               activations nothing is rounded below fp32.
 *               Values are summed before the sum is divided, with weights of up to 2^8: their
 *               sum over the keys has to stay below 2^119.
 *               A row's results are bitwise the same whatever shares its call, and a prompt
 *               token's do not depend on how its prompt is cut into calls.
 *   Non-finite  A key or value that a token does not see leaves it untouched, whatever it
 *               holds: stale cache rows may hold infinities and NaN.  One that it sees counts
 *               as in the formula, an infinite value whose weight underflowed to zero as NaN,
 *               a head of values with an infinite scale (the write makes none) as NaN too.
 */
#ifndef GDN_ATTENTION_H
#define GDN_ATTENTION_H

#include "gdn_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a cache holds its values: in the activations' dtype, or as 8-bit codes with an fp32
 * scale for each head of a row: 8-bit floating point (4 exponent, 3 mantissa bits, largest
 * value 448), or integers from -127 to 127. */
typedef enum { GDN_CACHE_PLAIN = 0, GDN_CACHE_E4M3 = 1, GDN_CACHE_INT8 = 2 } gdn_cache_format;

/* A cache of keys and values: k, v device [num_rows, num_heads, head_dim] of the format's type,
 * k_scale, v_scale device fp32 [num_rows, num_heads] (not read for GDN_CACHE_PLAIN).  Row
 * page * kv_block + i is token i of a page, as in gdn_step_plan's token_kv_slot.  dtype is that
 * of the activations.  head_dim is a multiple of 8 up to 512 (the attention: 64, 128 or 256),
 * num_heads * head_dim at most 2^20, num_rows at most 2^31 - 1. */
typedef struct {
    int32_t num_heads;
    int32_t head_dim;
    int32_t dtype;       /* a gdn_dtype value */
    int32_t format;      /* a gdn_cache_format value */
    int64_t num_rows;
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
} gdn_kv_cache;

/* rotary_dim (even, 2..head_dim) is the part of each head that turns; the rest stays as it is.
 * Pairs are dims (i, i + rotary_dim / 2), or (2 i, 2 i + 1) with interleaved.  factor multiplies
 * the turned part (1, or the attention factor of a scaled context).  head_dim is at most 512. */
typedef struct {
    int32_t num_q_heads;   /* 0: no q */
    int32_t num_k_heads;   /* 0: no k */
    int32_t head_dim;
    int32_t rotary_dim;
    int32_t dtype;         /* a gdn_dtype value */
    int32_t interleaved;
    float factor;
} gdn_rotary_shape;

/*
 * Rotary positions: pair (a, b) number i of a token at position p becomes
 *     factor (a cos(p f_i) - b sin(p f_i)),   factor (b cos(p f_i) + a sin(p f_i)).
 * The angle is formed in 64 bits from the fp32 frequency and reduced to a part of a turn
 * before it is rounded, so positions up to 2^31 - 1 lose nothing.
 *   positions  device [num_tokens] int32; a token with a negative one is padding: its rows are
 *              left as they are (in q_out and k_out too)
 *   inv_freq   device fp32 [rotary_dim / 2], radians for each position
 *   q, q_out   device [num_tokens, num_q_heads, head_dim] (dtype), row strides q_stride,
 *              q_out_stride;  k, k_out likewise.  q_out may be q itself with the same stride
 *              (in place); otherwise outputs overlap no input.
 * Any alignment to an element; rows and parts of whole 16-byte vectors are the fastest.
 */
gdn_status gdn_rotary(const gdn_rotary_shape* shape, int64_t num_tokens, const int32_t* positions,
                      const float* inv_freq, const void* q, int64_t q_stride, const void* k,
                      int64_t k_stride, void* q_out, int64_t q_out_stride, void* k_out,
                      int64_t k_out_stride, hipStream_t stream);

/*
 * Writes the keys and values of num_tokens tokens into cache rows slots[t].
 *   k, v    device [num_tokens, num_heads, head_dim] (dtype), row strides k_stride, v_stride
 *           (multiples of 8), 16-byte aligned
 *   slots   device [num_tokens] int64; a token whose slot is outside [0, num_rows) is skipped
 * In 8 bits each head x of a token gets the scale max(|x|, 2^-100) / M in fp32, M = 448 or 127,
 * and the codes are x / scale, a division rounded to fp32, rounded to the nearest code (ties
 * to even).  A head with an infinity or a NaN gets a NaN scale and codes of zero: all of it
 * reads back as NaN.
 */
gdn_status gdn_kv_cache_write(const gdn_kv_cache* cache, int64_t num_tokens, const void* k,
                              int64_t k_stride, const void* v, int64_t v_stride,
                              const int64_t* slots, hipStream_t stream);

/* The values of cache rows slots[t] (code times scale in fp32, rounded to dtype) into k_out,
 * v_out, device [num_tokens, num_heads, head_dim] (dtype), dense; zeros where the slot is
 * outside [0, num_rows). */
gdn_status gdn_kv_cache_read(const gdn_kv_cache* cache, int64_t num_tokens, const int64_t* slots,
                             void* k_out, void* v_out, hipStream_t stream);

/*
 * Causal attention of packed prompts over a paged cache: token j of sequence i, at position
 * t = start_pos[i] + j, sees the keys of positions 0..t of its sequence,
 *     o = sum_p w_p v_p / sum_p w_p,   w_p = exp(scale q.k_p),
 * where query head h reads cache head h / (num_q_heads / num_heads).
 *   cu_seqlens  device [num_seqs + 1] int32, as for gdn_chunk_prefill; tokens behind the last
 *               sequence are left as they were
 *   start_pos   device [num_seqs] int32 or NULL (= all 0): tokens cached before these (negative
 *               counts as 0)
 *   q           device [total_tokens, num_q_heads, head_dim] (dtype), row stride q_stride (a
 *               multiple of 8), 16-byte aligned
 *   kv_table    device [num_seqs, kv_table_width] int32: the pages of each sequence; position p
 *               is cache row kv_table[i][p / kv_block] * kv_block + p % kv_block
 *   o           device [total_tokens, num_q_heads, head_dim] (dtype), dense, written; a token
 *               that sees no key (all absent) gets zeros
 * The keys of a row are not split over workgroups here: a few tokens behind a long context are far faster as a
 * chain of gdn_attention_decode (16 tokens behind 32768, 8 heads: 41 us for 704).
 */
gdn_status gdn_attention_prefill(const gdn_kv_cache* cache, int32_t num_q_heads, float scale,
                                 int32_t num_seqs, int64_t total_tokens, const int32_t* cu_seqlens,
                                 const int32_t* start_pos, const void* q, int64_t q_stride,
                                 const int32_t* kv_table, int32_t kv_table_width, int32_t kv_block,
                                 void* o, hipStream_t stream);

/* Bytes of device workspace that gdn_attention_decode needs for at most num_rows rows,
 * tokens_per_row tokens of each and max_keys keys (0 for an unsupported shape or size): a workspace of
 * this size serves every smaller call too. */
size_t gdn_attention_decode_workspace_size(const gdn_kv_cache* cache, int32_t num_q_heads,
                                           int32_t num_rows, int32_t tokens_per_row,
                                           int64_t max_keys);

/*
 * The same for tokens_per_row (1 to 64) tokens of each of num_rows cached rows: one token each is
 * an ordinary decode step, more are drafted tokens, a chain or a tree.
 *   computed    device [num_rows] int32: keys of row b in the cache before these tokens, which
 *               all of them see; the key of its token i is at position computed[b] + i.
 *               A negative count marks a padding row: its outputs are zeros.
 *   tree_mask   device [num_rows * tokens_per_row] int64 or NULL: bit j of a token's mask lets it
 *               see the key of token j of its row (its ancestors' bits and its own make a
 *               tree; bits from tokens_per_row on are not looked at).  NULL is a chain: token i
 *               sees tokens 0..i.  A token that sees no key at all gets zeros.
 *   q, o        device [num_rows * tokens_per_row, num_q_heads, head_dim] as for the prefill
 *   kv_table    device [num_rows, kv_table_width] int32
 *   max_keys    the most keys (computed + tokens_per_row) of any row, or 0 for all that the table
 *               holds.  It sizes the launch and the workspace, a tight one is the fastest; the
 *               outputs of a row with more keys are NaN.
 *   workspace   at least gdn_attention_decode_workspace_size() bytes (max_keys as given here, or
 *               kv_table_width * kv_block for 0), 256-byte aligned, no initialisation; calls that
 *               may run at the same time need one each.  May be NULL when the size is 0.
 */
gdn_status gdn_attention_decode(const gdn_kv_cache* cache, int32_t num_q_heads, float scale,
                                int32_t num_rows, int32_t tokens_per_row, const int32_t* computed,
                                const int64_t* tree_mask, const void* q, int64_t q_stride,
                                const int32_t* kv_table, int32_t kv_table_width, int32_t kv_block,
                                int64_t max_keys, void* o, void* workspace, size_t workspace_bytes,
                                hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ATTENTION_H */
