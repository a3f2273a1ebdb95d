// gdn_attention_internal.h -- launcher interface between the attention layers' C ABI
// (gdn_attention_api.cpp) and their kernels (gdn_rotary.hip, gdn_kv_cache.hip,
// gdn_attention.hip).  Host-side declarations, and the division both sides share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn_attention.h"

namespace gdn {

// n / d for 0 <= n < 2^31 as a product: with 2^(l-1) < d <= 2^l and m = ceil(2^(31 + l) / d) < 2^32,
// m d exceeds 2^(31 + l) by less than 2^l, so n m / 2^(31 + l) is n / d and less than 1 / d more.
struct Divisor {
    uint32_t d, m, l;
    Divisor() : Divisor(1) {}
    explicit Divisor(uint32_t by) : d(by), m(0), l(0) {
        while ((1ull << l) < d) ++l;
        m = (uint32_t)(((1ull << (31 + l)) + d - 1) / d);
    }
};

struct RotaryArgs {
    gdn_rotary_shape shape;
    int64_t num_tokens;
    const int32_t* positions;
    const float* inv_freq;
    const void* in[2];      // q, k
    int64_t in_stride[2];
    void* out[2];
    int64_t out_stride[2];
};
hipError_t launch_rotary(const RotaryArgs& a, hipStream_t stream);

struct CacheCopyArgs {
    gdn_kv_cache cache;
    int64_t num_tokens;
    const int64_t* slots;
    const void* in[2];      // write: k, v
    int64_t in_stride[2];
    void* out[2];           // read: k, v
};
hipError_t launch_cache_write(const CacheCopyArgs& a, hipStream_t stream);
hipError_t launch_cache_read(const CacheCopyArgs& a, hipStream_t stream);

// One attention call.  Prefill: num_seqs sequences by cu_seqlens (tokens_per_row 0).  Decode:
// num_seqs rows of tokens_per_row tokens, past = computed.
struct AttentionArgs {
    gdn_kv_cache cache;
    int H_q;
    float scale;
    int num_seqs;
    int64_t total_tokens;
    const int32_t* cu_seqlens;
    const int32_t* past;
    int tokens_per_row;
    const int64_t* tree_mask;
    const void* q;
    int64_t q_stride;
    const int32_t* table;
    int table_width, kv_block;
    int capacity;           // keys that the table holds, at most 2^31 - 1025
    int max_keys;           // decode: the launch's bound, at most capacity
    void* o;
    void* workspace;
};
size_t attention_workspace_bytes(int H_q, int H_kv, int head_dim, int num_rows, int tokens_per_row, int64_t max_keys);
hipError_t launch_attention_prefill(const AttentionArgs& a, hipStream_t stream);
hipError_t launch_attention_decode(const AttentionArgs& a, hipStream_t stream);

}  // namespace gdn
