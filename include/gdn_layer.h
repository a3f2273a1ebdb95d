/*
 * gdn_layer.h -- the operators around the gated delta rule, in libgdn.so beside gdn.h.
 *
 * A recurrent layer's serving step needs more than the rule itself: the slot maps and
 * packed offsets of the step, the short convolution that makes q, k and v, a scan for
 * the layers whose recurrence has no delta rule, and the norms behind and between the
 * blocks.  These entry points cover them:
 *
 *   gdn_step_plan              cu_seqlens, state slots, export lists and per-token maps
 *                              of one step, on the GPU, from request lengths and block
 *                              tables
 *   gdn_causal_conv_prefill,
 *   gdn_causal_conv_decode     short causal convolution with SiLU and per-head L2 norm
 *   gdn_ssm_chunk_prefill,
 *   gdn_ssm_recurrent_decode   selective state space scan (scalar decay per head)
 *   gdn_gated_norm             grouped RMS norm with a gate, behind the recurrence
 *   gdn_residual_norm          norm after a block, gate, scaled residual add and the
 *                              next block's norm, in one pass
 *
 * The conventions of gdn.h hold here too (caller-owned device memory, nothing
 * allocated, work only enqueued on `stream`, no synchronisation, capturable, slots
 * bounds-checked on the device, host arguments validated before anything is enqueued,
 * gdn_last_error() for the message).  Differences and additions:
 *   Size        A call whose launch would take more than 2^32 - 1 threads (16 million rows of a
 *               wide norm, 2^29 tokens) returns GDN_ERR_UNSUPPORTED.
 *   Parameters  Weights, biases and every per-head parameter are fp32, whatever the
 *               activations' dtype.
 *   Strides     Where an argument has a row stride (in elements), its rows may be columns
 *               of a wider matrix (a projection's output); everything else is dense.
 *   Arithmetic  All sums, softplus / SiLU evaluations, norms and states are fp32 or
 *               wider.  Two operands of the scan's bf16 prefill are rounded to bf16 on their
 *               way into the matrix cores: the decayed scores and the copy of the state that
 *               C is multiplied with, by at most 2^-8 of each product.  The state itself, fp32
 *               prefills and decode round nothing below fp32.  A row's or a sequence's results
 *               are bitwise the same whatever shares its call.
 *   Range       No operand is narrowed below its own dtype's range: the scan's bf16 path
 *               feeds the matrix cores bf16 operands, so bf16's range is the only bound.
 *               Sums of squares are fp32: a head or row whose sum passes fp32's range comes
 *               out as zeros; under the root (with eps) what is below 2^-126 counts as 2^-126.
 *   Non-finite  A non-finite input of the scan reaches no earlier token and no other sequence.
 *               One in x makes its column of y NaN from its token to the chunk's end, and the
 *               column's state, and so y after that, not finite, also where the recurrence
 *               would give an infinity of a sign.
 */
#ifndef GDN_LAYER_H
#define GDN_LAYER_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activation of a gate or of the convolution's output. */
typedef enum { GDN_ACT_NONE = 0, GDN_ACT_SILU = 1, GDN_ACT_SIGMOID = 2 } gdn_activation;

/*
 * One step's plan.  Requests [0, num_decode_rows) are decode rows, the rest prefills.
 *   computed    device [num_requests] int32: tokens already in the caches (negative
 *               counts as 0).
 *   new_tokens  device [num_requests] int32: tokens of this step.  A decode row takes one
 *               token; with 0 or less it is a padding row.  A prefill may be empty.
 *               A decode row continues a cached state, so its computed has to be at least 1:
 *               with 0 its slot_in is -1, which the decode entry points take as padding, and
 *               its token is lost.  A request's first token is a prefill, of one token or more.
 *   state_table device [num_requests, state_table_width] int32: the cache slot of each
 *               request's state after (j + 1) * state_block tokens, j = 0..; state_block
 *               is a positive multiple of 64 (the prefix-cache block).
 *   run_slot    device [num_requests] int32: the slot of the request's state anywhere else.
 * With slot(r, p) = -1 for p <= 0, state_table[r][p / state_block - 1] when p is a
 * multiple of state_block (-1 past the table's width) and run_slot[r] otherwise:
 *   slot_in, slot_out    [num_decode_rows]: slot(r, computed), slot(r, computed + 1); -1 in
 *               a padding row.  As gdn_recurrent_decode takes them: the state moves into the
 *               block's slot when the token completes a block.
 *   cu_seqlens  [N + 1], N = num_requests - num_decode_rows: packed offsets of the prefills,
 *               relative to token num_decode_rows (sums stop at 2^31 - 1).
 *   start_pos, init_slot, final_slot [N]: computed, slot(r, computed) and
 *               slot(r, computed + new).
 *   export_offsets [N + 1], export_slots [export_capacity]: the states on the state_block
 *               grid, as gdn_chunk_prefill takes them with export_grid = state_block.  An
 *               export that is the final state is -1 (final_slot stores it); entries past
 *               export_offsets[N] are -1; exports past the capacity are dropped.
 *   token_request, token_position [token_capacity] int32: the request and absolute position
 *               of each token row, decode rows first; -1 in padding rows and past the end.
 *   token_kv_slot [token_capacity] int64: kv_table[r][p / kv_block] * kv_block + p % kv_block
 *               for the token at position p, the row of a paged key/value cache; -1 in padding
 *               rows, past kv_table's width or where its entry is negative.
 *   kv_table    device [num_requests, kv_table_width] int32, read for token_kv_slot alone.
 *   token_request, token_position and token_kv_slot may be NULL, and export_slots when
 *   export_capacity is 0.
 * num_requests == 0 writes the padding of the outputs.
 */
gdn_status gdn_step_plan(int32_t num_requests, int32_t num_decode_rows, const int32_t* computed,
                         const int32_t* new_tokens, const int32_t* state_table,
                         int32_t state_table_width, int32_t state_block, const int32_t* run_slot,
                         const int32_t* kv_table, int32_t kv_table_width, int32_t kv_block,
                         int64_t token_capacity, int64_t export_capacity, int32_t* slot_in,
                         int32_t* slot_out, int32_t* cu_seqlens, int32_t* start_pos,
                         int32_t* init_slot, int32_t* final_slot, int32_t* export_offsets,
                         int32_t* export_slots, int32_t* token_request, int32_t* token_position,
                         int64_t* token_kv_slot, hipStream_t stream);

/* The convolution's channels, C = channels[0] + channels[1] + channels[2] of them, as up
 * to three runs that go to separate dense outputs (q, k, v of the rule; C, B, x of the scan).
 * channels[i] is a multiple of 8, 0 for an unused run (its output may be NULL), C > 0.
 * l2_dim[i] is 0, or 32, 64, 128 or 256: then each l2_dim[i] channels of run i are a head,
 * divided by sqrt(sum of squares + l2_eps) after the activation; it divides channels[i].
 * width (2, 3 or 4) is the number of taps; dtype is that of x, the outputs and the states. */
typedef struct {
    int32_t channels[3];
    int32_t l2_dim[3];
    int32_t width;
    int32_t dtype;        /* a gdn_dtype value */
    int32_t activation;   /* GDN_ACT_NONE or GDN_ACT_SILU */
    float l2_eps;
} gdn_conv_shape;

/*
 * Short causal convolution of packed sequences, each channel by itself:
 *     a_t = bias + sum_{j < width} weight[j] x_{t - width + 1 + j},   y_t = act(a_t)
 * and the per-head L2 norm.  Inputs before a sequence's first token come from its state,
 * zeros without one; a state is the last width - 1 inputs, oldest first.
 *   x          device [total_tokens, C] with row stride x_stride (elements, a multiple of 8)
 *   weight     device [C, width] fp32, oldest tap first;  bias device [C] fp32 or NULL
 *   y0, y1, y2 device [total_tokens, channels[i]], written
 *   conv_pool  device [num_slots, width - 1, C] (dtype), read at init_slot, written at
 *              final_slot (and at export_slots)
 *   cu_seqlens, init_slot, final_slot, start_pos, export_*  as for gdn_chunk_prefill, with
 *              export_states [num_export_states, width - 1, C] (dtype).
 * A zero-length sequence copies its state (zeros without one).
 */
gdn_status gdn_causal_conv_prefill(const gdn_conv_shape* shape, int32_t num_seqs,
                                   int64_t total_tokens, const int32_t* cu_seqlens, const void* x,
                                   int64_t x_stride, const float* weight, const float* bias, void* y0,
                                   void* y1, void* y2, void* conv_pool, int32_t num_slots,
                                   const int32_t* init_slot, const int32_t* final_slot,
                                   const int32_t* start_pos, int32_t export_grid,
                                   void* export_states, const int32_t* export_offsets,
                                   const int32_t* export_slots, int64_t num_export_states,
                                   hipStream_t stream);

/* The same for one token of each of num_rows cached rows: the state at slot_in[b] gives the
 * earlier inputs, the shifted state goes to slot_out[b].  A row whose slot_in is outside
 * [0, num_slots) is padding: its outputs are zero and no state is written.  Bitwise what
 * gdn_causal_conv_prefill gives for one-token sequences. */
gdn_status gdn_causal_conv_decode(const gdn_conv_shape* shape, int32_t num_rows, const void* x,
                                  int64_t x_stride, const float* weight, const float* bias, void* y0,
                                  void* y1, void* y2, void* conv_pool, int32_t num_slots,
                                  const int32_t* slot_in, const int32_t* slot_out,
                                  hipStream_t stream);

/* Parameters of the scan, device fp32 [num_v_heads] each: the decay rate A (negative), the
 * bias added to dt (or NULL) and the skip factor D (or NULL).  With dt_softplus the step is
 * softplus(dt + bias), without it dt + bias. */
typedef struct {
    const float* A;
    const float* dt_bias;
    const float* D;
    int32_t dt_softplus;
} gdn_ssm_params;

/* Bytes of device workspace gdn_ssm_chunk_prefill needs (0 for an unsupported shape) on the
 * current device, for exactly this many sequences and tokens: a call with fewer may need
 * more, since calls with few sequences take another launch than calls with many. */
size_t gdn_ssm_chunk_prefill_workspace_size(const gdn_shape* shape, int32_t num_seqs,
                                            int64_t total_tokens);

/* The most that any call with at most max_seqs sequences and max_tokens tokens needs: the
 * size of a workspace that is allocated once for steps of all sizes. */
size_t gdn_ssm_chunk_prefill_workspace_bound(const gdn_shape* shape, int32_t max_seqs,
                                             int64_t max_tokens);

/*
 * Selective state space scan of packed sequences.  Per value head, with step d and state
 * S [d_k][d_v]:
 *     S <- exp(d A) S + d b x^T;   y = scale S^T c + D x
 * in 64-token chunks on the absolute grid.  The head layout is gdn_shape's: b and c are the
 * num_k_heads groups of width d_k (the state size), x and y the num_v_heads heads of width
 * d_v, and head h reads group h / (num_v_heads / num_k_heads).
 *   c, b       device [total_tokens, num_k_heads, d_k] (dtype)
 *   x, y       device [total_tokens, num_v_heads, d_v] (dtype; y written)
 *   dt         device [total_tokens, num_v_heads] fp32
 *   state_pool device [num_slots, num_v_heads, d_k, d_v] fp32
 *   the remaining arguments, the zero-length sequences and the split of a prompt across
 *   calls are gdn_chunk_prefill's.  workspace is 256-byte aligned and holds
 *   at least gdn_ssm_chunk_prefill_workspace_size() bytes (may be NULL when that is 0).
 */
gdn_status gdn_ssm_chunk_prefill(const gdn_shape* shape, const gdn_ssm_params* params,
                                 int32_t num_seqs, int64_t total_tokens, const int32_t* cu_seqlens,
                                 const void* c, const void* b, const void* x, const float* dt, void* y,
                                 float* state_pool, int32_t num_slots, const int32_t* init_slot,
                                 const int32_t* final_slot, const int32_t* start_pos,
                                 int32_t export_grid, float* export_states,
                                 const int32_t* export_offsets, const int32_t* export_slots,
                                 int64_t num_export_states, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/* One token of each of num_rows cached rows; slots and padding rows as for
 * gdn_recurrent_decode. */
gdn_status gdn_ssm_recurrent_decode(const gdn_shape* shape, const gdn_ssm_params* params,
                                    int32_t num_rows, const void* c, const void* b, const void* x,
                                    const float* dt, void* y, float* state_pool, int32_t num_slots,
                                    const int32_t* slot_in, const int32_t* slot_out,
                                    hipStream_t stream);

/*
 * Gated RMS norm of each group of dim values, rms(v) = v / sqrt(mean(v^2) + eps):
 *     gate_first == 0:  y = rms(x) weight act(z)        (behind the gated delta rule)
 *     gate_first != 0:  y = rms(x act(z)) weight        (behind a state space scan)
 *   x, z   device [num_rows, num_groups, dim] (dtype), row strides x_stride, z_stride in
 *          elements; z may be NULL (no gate)
 *   weight device fp32 [dim], shared by the groups, or [num_groups, dim] with
 *          weight_per_group
 *   y      device [num_rows, num_groups, dim] (dtype), dense; may be x itself when x is dense
 * Any 1 <= dim <= 16384, any row stride and alignment to an element; aligned rows of whole
 * 16-byte vectors are the fastest.
 */
gdn_status gdn_gated_norm(int64_t num_rows, int32_t num_groups, int32_t dim, int32_t dtype,
                          const void* x, int64_t x_stride, const void* z, int64_t z_stride,
                          const float* weight, int32_t weight_per_group, float eps,
                          int32_t gate_first, int32_t activation, void* y, hipStream_t stream);

/*
 * Between two blocks, for each row of dim values:
 *     n  = rms(x) post_weight          (x itself when post_weight is NULL)
 *     r' = residual + residual_scale act(gate) n      (no gate when it is NULL)
 *     y  = rms(r') pre_weight          (left out when y is NULL)
 *   x, gate      device [num_rows, dim] (dtype), row strides x_stride, gate_stride
 *   residual, residual_out  device [num_rows, dim] of residual_dtype, dense; may be the same
 *                memory.  residual_dtype is GDN_F32, or dtype.
 *   y            device [num_rows, dim] (dtype), dense, not overlapping the others; its norm
 *                is taken of r' as stored.
 * 1 <= dim <= 16384.
 */
gdn_status gdn_residual_norm(int64_t num_rows, int32_t dim, int32_t dtype, int32_t residual_dtype,
                             const void* x, int64_t x_stride, const float* post_weight,
                             const void* gate, int64_t gate_stride, int32_t activation,
                             float residual_scale, const void* residual, void* residual_out,
                             const float* pre_weight, float eps, void* y, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_LAYER_H */
