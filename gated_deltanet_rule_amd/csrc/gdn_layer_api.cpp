// gdn_layer_api.cpp -- the C ABI of the layer operators (include/gdn_layer.h): host-side
// validation and dispatch to the gfx950 launchers, by the same rules as gdn_api.cpp (every
// scalar and pointer the host can see is checked before any work is enqueued; a bad value
// returns an error status and a message naming it; no fallback path).
#include <cmath>
#include <cstddef>

#include "gdn_layer.h"
#include "gdn_check.h"
#include "gdn_layer_internal.h"

namespace {

using gdn::aligned;
using gdn::check_ptrs;
using gdn::fail;
using gdn::hip_status;

constexpr int64_t kMaxTokens = 0x7fffffffLL - 2 * GDN_CHUNK;
constexpr int kMaxDim = 16384;

// A launcher's result: a call too large for one launch is the caller's to split.
gdn_status launched(hipError_t e, const char* what) {
    if (e == hipErrorInvalidConfiguration) return fail(GDN_ERR_UNSUPPORTED, "%s exceeds the launch grid of 2^32 - 1 threads", what);
    return hip_status(e, what);
}

size_t elem(int32_t dtype) { return dtype == GDN_BF16 ? 2 : 4; }

gdn_status check_dtype(int32_t dtype, const char* name) {
    if (dtype != GDN_F32 && dtype != GDN_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "%s %d is neither GDN_F32 (0) nor GDN_BF16 (1)", name, dtype);
    return GDN_OK;
}

// The packed-sequence arguments shared by the prefill entry points (pointers that depend
// on the operator are checked by the caller).
gdn_status check_packed(int32_t num_seqs, int64_t total_tokens, int32_t num_slots, const int32_t* cu_seqlens,
                        const int32_t* init_slot, const int32_t* final_slot, const int32_t* start_pos,
                        const void* pool, int32_t export_grid, const void* export_states,
                        const int32_t* export_offsets, const int32_t* export_slots, int64_t num_export_states) {
    if (num_seqs < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "num_seqs %d is negative", num_seqs);
    if (total_tokens < 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "total_tokens %lld is negative", (long long)total_tokens);
    if (total_tokens > kMaxTokens)
        return fail(GDN_ERR_UNSUPPORTED, "total_tokens %lld exceeds the supported 2^31 - 129", (long long)total_tokens);
    if (num_slots < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "num_slots %d is negative", num_slots);
    if (export_grid < 0 || export_grid % GDN_CHUNK != 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "export_grid %d is not a multiple of chunk size %d (use 0 for no export)",
                    export_grid, GDN_CHUNK);
    if (num_export_states < 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "num_export_states %lld is negative", (long long)num_export_states);
    if (num_seqs == 0) return GDN_OK;
    gdn_status st = check_ptrs({{"cu_seqlens", cu_seqlens, 4}, {"init_slot", init_slot, 4}, {"final_slot", final_slot, 4}});
    if (st != GDN_OK) return st;
    if (start_pos && !aligned(start_pos, 4)) return fail(GDN_ERR_INVALID_ARGUMENT, "start_pos is not 4-byte aligned");
    if (num_slots > 0) {
        st = check_ptrs({{"pool", pool, 16}});
        if (st != GDN_OK) return st;
    }
    if (export_grid > 0) {
        st = check_ptrs({{"export_offsets", export_offsets, 4}});
        if (st != GDN_OK) return st;
        if (num_export_states > 0) {
            st = export_slots ? check_ptrs({{"export_slots", export_slots, 4}})
                              : check_ptrs({{"export_states", export_states, 16}});
            if (st != GDN_OK) return st;
        }
    }
    return GDN_OK;
}

gdn_status check_conv_shape(const gdn_conv_shape* s) {
    if (!s) return fail(GDN_ERR_INVALID_ARGUMENT, "shape is NULL");
    int64_t c = 0;
    for (int i = 0; i < 3; ++i) {
        if (s->channels[i] < 0)
            return fail(GDN_ERR_INVALID_ARGUMENT, "channels[%d] %d is negative", i, s->channels[i]);
        if (s->channels[i] % 8 != 0)
            return fail(GDN_ERR_UNSUPPORTED, "channels[%d] %d is not a multiple of 8", i, s->channels[i]);
        const int d = s->l2_dim[i];
        if (d != 0 && d != 32 && d != 64 && d != 128 && d != 256)
            return fail(GDN_ERR_UNSUPPORTED, "l2_dim[%d] %d: must be 0, 32, 64, 128 or 256", i, d);
        if (d != 0 && s->channels[i] % d != 0)
            return fail(GDN_ERR_INVALID_ARGUMENT, "channels[%d] %d is not a multiple of l2_dim[%d] %d", i, s->channels[i], i, d);
        c += s->channels[i];
    }
    if (c == 0) return fail(GDN_ERR_INVALID_ARGUMENT, "the convolution has no channels");
    if (c > (1 << 20)) return fail(GDN_ERR_UNSUPPORTED, "%lld channels exceed 2^20", (long long)c);
    if (s->width < 2 || s->width > 4) return fail(GDN_ERR_UNSUPPORTED, "width %d: must be 2, 3 or 4", s->width);
    if (s->activation != GDN_ACT_NONE && s->activation != GDN_ACT_SILU)
        return fail(GDN_ERR_UNSUPPORTED, "activation %d: must be GDN_ACT_NONE (0) or GDN_ACT_SILU (1)", s->activation);
    if (!(s->l2_eps >= 0.f) || !std::isfinite(s->l2_eps))
        return fail(GDN_ERR_INVALID_ARGUMENT, "l2_eps is not finite and non-negative");
    return check_dtype(s->dtype, "dtype");
}

gdn_status check_conv_tensors(const gdn_conv_shape* s, const void* x, int64_t x_stride, const float* weight,
                              const float* bias, const void* const y[3]) {
    const int64_t C = (int64_t)s->channels[0] + s->channels[1] + s->channels[2];
    if (x_stride < C || x_stride % 8 != 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "x_stride %lld must be a multiple of 8 of at least the %lld channels",
                    (long long)x_stride, (long long)C);
    gdn_status st = check_ptrs({{"x", x, 16}, {"weight", weight, 16}});
    if (st != GDN_OK) return st;
    if (bias && !aligned(bias, 16)) return fail(GDN_ERR_INVALID_ARGUMENT, "bias is not 16-byte aligned");
    const char* names[3] = {"y0", "y1", "y2"};
    for (int i = 0; i < 3; ++i)
        if (s->channels[i] > 0) {
            st = check_ptrs({{names[i], y[i], 16}});
            if (st != GDN_OK) return st;
        }
    return GDN_OK;
}

gdn::ConvArgs conv_args(const gdn_conv_shape* s, const void* x, int64_t x_stride, const float* weight,
                        const float* bias, void* y0, void* y1, void* y2, void* pool, int32_t num_slots) {
    gdn::ConvArgs a = {};
    for (int i = 0; i < 3; ++i) {
        a.channels[i] = s->channels[i];
        a.l2_dim[i] = s->l2_dim[i];
    }
    a.C = s->channels[0] + s->channels[1] + s->channels[2];
    a.width = s->width;
    a.dtype = s->dtype;
    a.silu = s->activation == GDN_ACT_SILU;
    a.l2_eps = s->l2_eps;
    a.x = x;
    a.x_stride = x_stride;
    a.weight = weight;
    a.bias = bias;
    a.y[0] = y0;
    a.y[1] = y1;
    a.y[2] = y2;
    a.pool = pool;
    a.num_slots = num_slots;
    return a;
}

gdn_status check_ssm(const gdn_shape* shape, const gdn_ssm_params* p) {
    gdn_status st = gdn::check_shape(shape);
    if (st != GDN_OK) return st;
    if (!p) return fail(GDN_ERR_INVALID_ARGUMENT, "params is NULL");
    st = check_ptrs({{"A", p->A, 4}});
    if (st != GDN_OK) return st;
    if (!aligned(p->dt_bias, 4)) return fail(GDN_ERR_INVALID_ARGUMENT, "dt_bias is not 4-byte aligned");
    if (!aligned(p->D, 4)) return fail(GDN_ERR_INVALID_ARGUMENT, "D is not 4-byte aligned");
    return GDN_OK;
}

gdn::SsmArgs ssm_args(const gdn_shape* s, const gdn_ssm_params* p, const void* c, const void* b, const void* x,
                      const float* dt, void* y, float* pool, int32_t num_slots) {
    gdn::SsmArgs a = {};
    a.H_k = s->num_k_heads;
    a.H_v = s->num_v_heads;
    a.d_k = s->d_k;
    a.d_v = s->d_v;
    a.dtype = s->dtype;
    a.scale = s->scale;
    a.A = p->A;
    a.dt_bias = p->dt_bias;
    a.D = p->D;
    a.dt_softplus = p->dt_softplus != 0;
    a.c = c;
    a.b = b;
    a.x = x;
    a.dt = dt;
    a.y = y;
    a.pool = pool;
    a.num_slots = num_slots;
    return a;
}

gdn_status check_norm(int64_t num_rows, int64_t groups, int32_t dim, int32_t dtype, int32_t activation, float eps) {
    if (num_rows < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "num_rows %lld is negative", (long long)num_rows);
    if (groups <= 0) return fail(GDN_ERR_INVALID_ARGUMENT, "num_groups %lld is not positive", (long long)groups);
    if (dim <= 0) return fail(GDN_ERR_INVALID_ARGUMENT, "dim %d is not positive", dim);
    if (dim > kMaxDim) return fail(GDN_ERR_UNSUPPORTED, "dim %d exceeds %d", dim, kMaxDim);
    if (num_rows > 0x7fffffffLL / groups)      // (the launchers know how many threads a norm takes)
        return fail(GDN_ERR_UNSUPPORTED, "num_rows %lld x num_groups %lld exceeds the launch grid", (long long)num_rows, (long long)groups);
    if (activation != GDN_ACT_NONE && activation != GDN_ACT_SILU && activation != GDN_ACT_SIGMOID)
        return fail(GDN_ERR_UNSUPPORTED, "activation %d: must be 0 (none), 1 (SiLU) or 2 (sigmoid)", activation);
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(GDN_ERR_INVALID_ARGUMENT, "eps is not finite and non-negative");
    return check_dtype(dtype, "dtype");
}

}  // namespace

extern "C" {

gdn_status gdn_step_plan(int32_t num_requests, int32_t num_decode_rows, const int32_t* computed,
                         const int32_t* new_tokens, const int32_t* state_table, int32_t state_table_width,
                         int32_t state_block, const int32_t* run_slot, const int32_t* kv_table,
                         int32_t kv_table_width, int32_t kv_block, int64_t token_capacity, int64_t export_capacity,
                         int32_t* slot_in, int32_t* slot_out, int32_t* cu_seqlens, int32_t* start_pos,
                         int32_t* init_slot, int32_t* final_slot, int32_t* export_offsets, int32_t* export_slots,
                         int32_t* token_request, int32_t* token_position, int64_t* token_kv_slot, hipStream_t stream) {
    gdn::clear_error();
    if (num_requests < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "num_requests %d is negative", num_requests);
    if (num_decode_rows < 0 || num_decode_rows > num_requests)
        return fail(GDN_ERR_INVALID_ARGUMENT, "num_decode_rows %d is not in [0, num_requests %d]", num_decode_rows, num_requests);
    if (state_block <= 0 || state_block % GDN_CHUNK != 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "state_block %d is not a positive multiple of chunk size %d", state_block, GDN_CHUNK);
    if (state_table_width < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "state_table_width %d is negative", state_table_width);
    if (token_kv_slot && (kv_block <= 0 || kv_table_width < 0))
        return fail(GDN_ERR_INVALID_ARGUMENT, "kv_block %d must be positive and kv_table_width %d not negative", kv_block, kv_table_width);
    if (token_kv_slot && num_requests > 0 && kv_table_width > 0 && !kv_table)
        return fail(GDN_ERR_INVALID_ARGUMENT, "token_kv_slot is given without a kv_table");
    if (token_capacity < 0 || token_capacity > kMaxTokens)
        return fail(GDN_ERR_INVALID_ARGUMENT, "token_capacity %lld is not in [0, 2^31 - 129]", (long long)token_capacity);
    if (export_capacity < 0 || export_capacity > kMaxTokens)
        return fail(GDN_ERR_INVALID_ARGUMENT, "export_capacity %lld is not in [0, 2^31 - 129]", (long long)export_capacity);
    gdn_status st;
    if (num_requests > 0) {
        st = check_ptrs({{"computed", computed, 4}, {"new_tokens", new_tokens, 4}, {"run_slot", run_slot, 4}});
        if (st != GDN_OK) return st;
        if (state_table_width > 0) {
            st = check_ptrs({{"state_table", state_table, 4}});
            if (st != GDN_OK) return st;
        }
    }
    if (num_decode_rows > 0) {
        st = check_ptrs({{"slot_in", slot_in, 4}, {"slot_out", slot_out, 4}});
        if (st != GDN_OK) return st;
    }
    if (num_requests > num_decode_rows) {
        st = check_ptrs({{"start_pos", start_pos, 4}, {"init_slot", init_slot, 4}, {"final_slot", final_slot, 4}});
        if (st != GDN_OK) return st;
    }
    if (!aligned(kv_table, 4)) return fail(GDN_ERR_INVALID_ARGUMENT, "kv_table is not 4-byte aligned");
    if (!aligned(token_request, 4) || !aligned(token_position, 4))
        return fail(GDN_ERR_INVALID_ARGUMENT, "token_request or token_position is not 4-byte aligned");
    if (!aligned(token_kv_slot, 8)) return fail(GDN_ERR_INVALID_ARGUMENT, "token_kv_slot is not 8-byte aligned");
    if (export_capacity > 0) {
        st = check_ptrs({{"export_slots", export_slots, 4}});
        if (st != GDN_OK) return st;
    }
    st = check_ptrs({{"cu_seqlens", cu_seqlens, 4}, {"export_offsets", export_offsets, 4}});
    if (st != GDN_OK) return st;
    gdn::PlanArgs a = {num_requests, num_decode_rows, computed, new_tokens, state_table, state_table_width, state_block,
                       run_slot, kv_table, kv_table_width, kv_block, token_capacity, export_capacity, slot_in, slot_out,
                       cu_seqlens, start_pos, init_slot, final_slot, export_offsets, export_slots, token_request,
                       token_position, token_kv_slot};
    return launched(gdn::launch_plan(a, stream), "step plan launch");
}

gdn_status gdn_causal_conv_prefill(const gdn_conv_shape* shape, int32_t num_seqs, int64_t total_tokens,
                                   const int32_t* cu_seqlens, const void* x, int64_t x_stride, const float* weight,
                                   const float* bias, void* y0, void* y1, void* y2, void* conv_pool, int32_t num_slots,
                                   const int32_t* init_slot, const int32_t* final_slot, const int32_t* start_pos,
                                   int32_t export_grid, void* export_states, const int32_t* export_offsets,
                                   const int32_t* export_slots, int64_t num_export_states, hipStream_t stream) {
    gdn::clear_error();
    gdn_status st = check_conv_shape(shape);
    if (st != GDN_OK) return st;
    st = check_packed(num_seqs, total_tokens, num_slots, cu_seqlens, init_slot, final_slot, start_pos, conv_pool,
                      export_grid, export_states, export_offsets, export_slots, num_export_states);
    if (st != GDN_OK || num_seqs == 0) return st;
    if (total_tokens > 0) {
        const void* y[3] = {y0, y1, y2};
        st = check_conv_tensors(shape, x, x_stride, weight, bias, y);
        if (st != GDN_OK) return st;
    }
    gdn::ConvArgs a = conv_args(shape, x, x_stride, weight, bias, y0, y1, y2, conv_pool, num_slots);
    a.num_seqs = num_seqs;
    a.total_tokens = total_tokens;
    a.cu_seqlens = cu_seqlens;
    a.init_slot = init_slot;
    a.final_slot = final_slot;
    a.start_pos = start_pos;
    a.export_grid = export_grid;
    a.export_slots = export_grid > 0 ? export_slots : nullptr;
    a.export_states = export_grid > 0 && !export_slots ? export_states : nullptr;
    a.export_offsets = export_grid > 0 ? export_offsets : nullptr;
    a.export_capacity = export_grid > 0 && (a.export_states || a.export_slots) ? num_export_states : 0;
    return launched(gdn::launch_conv(a, stream), "convolution launch");
}

gdn_status gdn_causal_conv_decode(const gdn_conv_shape* shape, int32_t num_rows, const void* x, int64_t x_stride,
                                  const float* weight, const float* bias, void* y0, void* y1, void* y2,
                                  void* conv_pool, int32_t num_slots, const int32_t* slot_in, const int32_t* slot_out,
                                  hipStream_t stream) {
    gdn::clear_error();
    gdn_status st = check_conv_shape(shape);
    if (st != GDN_OK) return st;
    if (num_rows < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "num_rows %d is negative", num_rows);
    if (num_slots < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "num_slots %d is negative", num_slots);
    if (num_rows == 0) return GDN_OK;
    const void* y[3] = {y0, y1, y2};
    st = check_conv_tensors(shape, x, x_stride, weight, bias, y);
    if (st != GDN_OK) return st;
    st = check_ptrs({{"conv_pool", conv_pool, 16}, {"slot_in", slot_in, 4}, {"slot_out", slot_out, 4}});
    if (st != GDN_OK) return st;
    gdn::ConvArgs a = conv_args(shape, x, x_stride, weight, bias, y0, y1, y2, conv_pool, num_slots);
    a.num_seqs = num_rows;
    a.total_tokens = num_rows;
    a.init_slot = slot_in;
    a.final_slot = slot_out;
    return launched(gdn::launch_conv(a, stream), "convolution decode launch");
}

size_t gdn_ssm_chunk_prefill_workspace_size(const gdn_shape* shape, int32_t num_seqs, int64_t total_tokens) {
    if (gdn::check_shape(shape) != GDN_OK || num_seqs < 0 || total_tokens < 0) return 0;
    return gdn::ssm_workspace_bytes(shape->num_v_heads, shape->d_k, shape->d_v, shape->dtype, num_seqs, total_tokens);
}

size_t gdn_ssm_chunk_prefill_workspace_bound(const gdn_shape* shape, int32_t max_seqs, int64_t max_tokens) {
    if (gdn::check_shape(shape) != GDN_OK || max_seqs < 0 || max_tokens < 0) return 0;
    return gdn::ssm_workspace_bound(shape->num_v_heads, shape->d_v, shape->dtype, max_seqs, max_tokens);
}

gdn_status gdn_ssm_chunk_prefill(const gdn_shape* shape, const gdn_ssm_params* params, int32_t num_seqs,
                                 int64_t total_tokens, const int32_t* cu_seqlens, const void* c, const void* b,
                                 const void* x, const float* dt, void* y, float* state_pool, int32_t num_slots,
                                 const int32_t* init_slot, const int32_t* final_slot, const int32_t* start_pos,
                                 int32_t export_grid, float* export_states, const int32_t* export_offsets,
                                 const int32_t* export_slots, int64_t num_export_states, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    gdn::clear_error();
    gdn_status st = check_ssm(shape, params);
    if (st != GDN_OK) return st;
    st = check_packed(num_seqs, total_tokens, num_slots, cu_seqlens, init_slot, final_slot, start_pos, state_pool,
                      export_grid, export_states, export_offsets, export_slots, num_export_states);
    if (st != GDN_OK || num_seqs == 0) return st;
    if ((int64_t)num_seqs * shape->num_v_heads * (shape->d_v / 16) > 0x7fffffffLL)
        return fail(GDN_ERR_UNSUPPORTED, "num_seqs %d x num_v_heads %d exceeds the launch grid", num_seqs, shape->num_v_heads);
    // a chunk's rows are addressed by 31-bit byte offsets
    if ((int64_t)shape->num_v_heads * shape->d_v > (1 << 22))
        return fail(GDN_ERR_UNSUPPORTED, "rows of num_v_heads %d x d_v %d values exceed the supported 2^22", shape->num_v_heads, shape->d_v);
    if ((int64_t)shape->num_k_heads * shape->d_k > (1 << 22))
        return fail(GDN_ERR_UNSUPPORTED, "rows of num_k_heads %d x d_k %d values exceed the supported 2^22", shape->num_k_heads, shape->d_k);
    if (total_tokens > 0) {
        st = check_ptrs({{"c", c, 16}, {"b", b, 16}, {"x", x, 16}, {"dt", dt, 4}, {"y", y, 16}});
        if (st != GDN_OK) return st;
    }
    const size_t need = gdn::ssm_workspace_bytes(shape->num_v_heads, shape->d_k, shape->d_v, shape->dtype, num_seqs, total_tokens);
    if (workspace_bytes < need)
        return fail(GDN_ERR_INVALID_ARGUMENT, "workspace_bytes %zu is smaller than the %zu bytes required", workspace_bytes, need);
    if (need > 0) {
        st = check_ptrs({{"workspace", workspace, 256}});
        if (st != GDN_OK) return st;
    }
    gdn::SsmArgs a = ssm_args(shape, params, c, b, x, dt, y, state_pool, num_slots);
    a.num_seqs = num_seqs;
    a.total_tokens = total_tokens;
    a.cu_seqlens = cu_seqlens;
    a.init_slot = init_slot;
    a.final_slot = final_slot;
    a.start_pos = start_pos;
    a.export_grid = export_grid;
    a.export_slots = export_grid > 0 ? export_slots : nullptr;
    a.export_states = export_grid > 0 && !export_slots ? export_states : nullptr;
    a.export_offsets = export_grid > 0 ? export_offsets : nullptr;
    a.export_capacity = export_grid > 0 && (a.export_states || a.export_slots) ? num_export_states : 0;
    a.workspace = workspace;
    return launched(gdn::launch_ssm_prefill(a, stream), "scan launch");
}

gdn_status gdn_ssm_recurrent_decode(const gdn_shape* shape, const gdn_ssm_params* params, int32_t num_rows,
                                    const void* c, const void* b, const void* x, const float* dt, void* y,
                                    float* state_pool, int32_t num_slots, const int32_t* slot_in,
                                    const int32_t* slot_out, hipStream_t stream) {
    gdn::clear_error();
    gdn_status st = check_ssm(shape, params);
    if (st != GDN_OK) return st;
    if (num_rows < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "num_rows %d is negative", num_rows);
    if (num_slots < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "num_slots %d is negative", num_slots);
    if (num_rows == 0) return GDN_OK;
    if ((int64_t)num_rows * shape->num_v_heads * (shape->d_v / 16) > 0x7fffffffLL)
        return fail(GDN_ERR_UNSUPPORTED, "num_rows %d x num_v_heads %d exceeds the launch grid", num_rows, shape->num_v_heads);
    st = check_ptrs({{"c", c, 16}, {"b", b, 16}, {"x", x, 16}, {"dt", dt, 4}, {"y", y, 16},
                     {"state_pool", state_pool, 16}, {"slot_in", slot_in, 4}, {"slot_out", slot_out, 4}});
    if (st != GDN_OK) return st;
    gdn::SsmArgs a = ssm_args(shape, params, c, b, x, dt, y, state_pool, num_slots);
    a.num_seqs = num_rows;
    a.total_tokens = num_rows;
    a.init_slot = slot_in;
    a.final_slot = slot_out;
    return launched(gdn::launch_ssm_decode(a, stream), "scan decode launch");
}

gdn_status gdn_gated_norm(int64_t num_rows, int32_t num_groups, int32_t dim, int32_t dtype, const void* x,
                          int64_t x_stride, const void* z, int64_t z_stride, const float* weight,
                          int32_t weight_per_group, float eps, int32_t gate_first, int32_t activation, void* y,
                          hipStream_t stream) {
    gdn::clear_error();
    gdn_status st = check_norm(num_rows, num_groups, dim, dtype, activation, eps);
    if (st != GDN_OK || num_rows == 0) return st;
    const int64_t row = (int64_t)num_groups * dim;
    if (x_stride < row) return fail(GDN_ERR_INVALID_ARGUMENT, "x_stride %lld is smaller than a row of %lld", (long long)x_stride, (long long)row);
    if (z && z_stride < row) return fail(GDN_ERR_INVALID_ARGUMENT, "z_stride %lld is smaller than a row of %lld", (long long)z_stride, (long long)row);
    const size_t es = elem(dtype);
    if (!aligned(z, es)) return fail(GDN_ERR_INVALID_ARGUMENT, "z is not %zu-byte aligned", es);
    st = check_ptrs({{"x", x, es}, {"weight", weight, 4}, {"y", y, es}});
    if (st != GDN_OK) return st;
    gdn::GatedNormArgs a = {num_rows, num_groups, dim, dtype, x, x_stride, z, z_stride, weight, weight_per_group != 0,
                            eps, gate_first != 0, activation, y};
    return launched(gdn::launch_gated_norm(a, stream), "gated norm launch");
}

gdn_status gdn_residual_norm(int64_t num_rows, int32_t dim, int32_t dtype, int32_t residual_dtype, const void* x,
                             int64_t x_stride, const float* post_weight, const void* gate, int64_t gate_stride,
                             int32_t activation, float residual_scale, const void* residual, void* residual_out,
                             const float* pre_weight, float eps, void* y, hipStream_t stream) {
    gdn::clear_error();
    gdn_status st = check_norm(num_rows, 1, dim, dtype, activation, eps);
    if (st != GDN_OK) return st;
    if (residual_dtype != GDN_F32 && residual_dtype != dtype)
        return fail(GDN_ERR_UNSUPPORTED, "residual_dtype %d is neither GDN_F32 (0) nor dtype %d", residual_dtype, dtype);
    if (!std::isfinite(residual_scale)) return fail(GDN_ERR_INVALID_ARGUMENT, "residual_scale is not finite");
    if (num_rows == 0) return GDN_OK;
    if (x_stride < dim) return fail(GDN_ERR_INVALID_ARGUMENT, "x_stride %lld is smaller than dim %d", (long long)x_stride, dim);
    if (gate && gate_stride < dim) return fail(GDN_ERR_INVALID_ARGUMENT, "gate_stride %lld is smaller than dim %d", (long long)gate_stride, dim);
    const size_t es = elem(dtype), rs = elem(residual_dtype);
    if (y) {
        st = check_ptrs({{"pre_weight", pre_weight, 4}, {"y", y, es}});
        if (st != GDN_OK) return st;
    }
    if (!aligned(post_weight, 4)) return fail(GDN_ERR_INVALID_ARGUMENT, "post_weight is not 4-byte aligned");
    if (!aligned(gate, es)) return fail(GDN_ERR_INVALID_ARGUMENT, "gate is not %zu-byte aligned", es);
    st = check_ptrs({{"x", x, es}, {"residual", residual, rs}, {"residual_out", residual_out, rs}});
    if (st != GDN_OK) return st;
    gdn::ResidualNormArgs a = {num_rows, dim, dtype, residual_dtype, x, x_stride, post_weight, gate, gate_stride, activation,
                               residual_scale, residual, residual_out, pre_weight, eps, y};
    return launched(gdn::launch_residual_norm(a, stream), "residual norm launch");
}

}  // extern "C"
