// gdn_layer_internal.h -- launcher interface between the layer operators' C ABI
// (gdn_layer_api.cpp) and their kernels (gdn_plan.hip, gdn_conv.hip, gdn_ssm.hip,
// gdn_norm.hip).  Host-side declarations only.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

// Whether a launch may have this many workgroups (of at most 2^32 - 1 threads in all).  The
// launchers return hipErrorInvalidConfiguration for calls that do not fit, before they enqueue
// anything.
inline bool grid_fits(int64_t blocks, int threads) { return blocks <= 0xffffffffLL / threads; }

struct PlanArgs {
    int num_requests, num_decode_rows;
    const int32_t* computed;
    const int32_t* new_tokens;
    const int32_t* state_table;
    int state_table_width, state_block;
    const int32_t* run_slot;
    const int32_t* kv_table;
    int kv_table_width, kv_block;
    int64_t token_capacity, export_capacity;
    int32_t *slot_in, *slot_out, *cu_seqlens, *start_pos, *init_slot, *final_slot, *export_offsets, *export_slots;
    int32_t *token_request, *token_position;
    int64_t* token_kv_slot;
};
hipError_t launch_plan(const PlanArgs& a, hipStream_t stream);

// One convolution call.  Prefill: num_seqs sequences over total_tokens rows.  Decode:
// total_tokens rows of one token each, slots in init_slot / final_slot, cu_seqlens NULL.
struct ConvArgs {
    int channels[3], l2_dim[3];
    int C, width, dtype, silu;
    float l2_eps;
    int num_seqs;
    int64_t total_tokens;
    const int32_t* cu_seqlens;
    const void* x;
    int64_t x_stride;
    const float* weight;
    const float* bias;
    void* y[3];
    void* pool;
    int num_slots;
    const int32_t* init_slot;
    const int32_t* final_slot;
    const int32_t* start_pos;
    int export_grid;
    void* export_states;
    const int32_t* export_offsets;
    const int32_t* export_slots;
    int64_t export_capacity;
};
hipError_t launch_conv(const ConvArgs& a, hipStream_t stream);

// One scan call; decode as for the convolution.
struct SsmArgs {
    int H_k, H_v, d_k, d_v, dtype;
    float scale;
    const float* A;
    const float* dt_bias;
    const float* D;
    int dt_softplus;
    int num_seqs;
    int64_t total_tokens;
    const int32_t* cu_seqlens;
    const void* c;
    const void* b;
    const void* x;
    const float* dt;
    void* y;
    float* pool;
    int num_slots;
    const int32_t* init_slot;
    const int32_t* final_slot;
    const int32_t* start_pos;
    int export_grid;
    float* export_states;
    const int32_t* export_offsets;
    const int32_t* export_slots;
    int64_t export_capacity;
    void* workspace;
};
size_t ssm_workspace_bytes(int H_v, int d_k, int d_v, int dtype, int num_seqs, int64_t total_tokens);
size_t ssm_workspace_bound(int H_v, int d_v, int dtype, int max_seqs, int64_t max_tokens);
hipError_t launch_ssm_prefill(const SsmArgs& a, hipStream_t stream);
hipError_t launch_ssm_decode(const SsmArgs& a, hipStream_t stream);

struct GatedNormArgs {
    int64_t num_rows;
    int groups, dim, dtype;
    const void* x;
    int64_t x_stride;
    const void* z;
    int64_t z_stride;
    const float* weight;
    int weight_per_group;
    float eps;
    int gate_first, activation;
    void* y;
};
hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t stream);

struct ResidualNormArgs {
    int64_t num_rows;
    int dim, dtype, residual_dtype;
    const void* x;
    int64_t x_stride;
    const float* post_weight;
    const void* gate;
    int64_t gate_stride;
    int activation;
    float residual_scale;
    const void* residual;
    void* residual_out;
    const float* pre_weight;
    float eps;
    void* y;
};
hipError_t launch_residual_norm(const ResidualNormArgs& a, hipStream_t stream);

}  // namespace gdn
