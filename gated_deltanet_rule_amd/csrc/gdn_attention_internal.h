// gdn_attention_internal.h -- launcher interface between the attention layers' C ABI
// (gdn_attention_api.cpp) and their kernels (gdn_rotary.hip, gdn_kv_cache.hip,
// gdn_attention.hip).  Host-side declarations, and what both sides share: division, spans of a
// long context.
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

// Keys of a span of a long context: at least this many for so many rows of a head, doubled until kMaxSpans suffice.  Short
// spans keep more of the chip busy for few requests, long ones start and join less often (16 rows of 128 dims in bf16 at
// 256 / 512 / 1024 keys: one request of 1024 keys 9.5 / 12 / 17 us, 64 requests of up to 8192 keys 266 / 245 / 235 us).  With more
// rows a span's partial sums weigh more: 512 / 1024 / 2048 keys, 16 requests with eight heads and up to 8192 keys, 60 rows 104 / 97 / 93
// us, 68 rows 109 / 99 / 94, 128 rows 136 / 113 / 104, 256 rows 221 / 166 / 166; with two heads and 4096 keys 64 rows 29 / 34 / 54, 68 rows
// 31 / 35 / 55, 128 rows 35 / 37 / 57.  fp32, eight heads, 68 rows 542 / 497 / 506.
constexpr int kMaxSpans = 64;
__host__ __device__ inline int least_span(int rows) { return rows <= 64 ? 512 : 1024; }
__host__ __device__ inline int span_keys(int rows, int keys) {
    int span = least_span(rows);
    while (keys > kMaxSpans * (int64_t)span) span *= 2;
    return span;
}
// Spans of a row of so many keys, at least one of them: up to 2^31 - 1025 keys and spans of 2^25, whose sum takes 32 bits.
__host__ __device__ inline int span_count(int keys, int span) { return (int)(((unsigned)keys + (unsigned)span - 1u) / (unsigned)span); }
// The most spans of any row of at most so many keys.
__host__ __device__ inline int most_spans(int rows, int64_t keys) {
    const int64_t least = least_span(rows);
    if (keys > kMaxSpans * least) return kMaxSpans;
    return keys > 0 ? span_count((int)keys, (int)least) : 1;
}

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
