// gdn_attention.hip -- attention over a paged cache for gfx950.
//
//     o = sum_p w_p v_p / sum_p w_p,   w_p = exp(scale q.k_p - m)
//
// One wave for each query head of a token, one key at a time with a running maximum and sum.
#include <hip/hip_runtime.h>

#include "gdn_attention_internal.h"
#include "gdn_layer_device.h"
#include "gdn_layer_internal.h"
#include "gdn_pages.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

template <typename T, int FORMAT>
__device__ __forceinline__ float cached(const void* p, int64_t i) {
    if constexpr (FORMAT == GDN_CACHE_PLAIN) return (float)static_cast<const T*>(p)[i];
    else if constexpr (FORMAT == GDN_CACHE_INT8) return (float)static_cast<const int8_t*>(p)[i];
    else return __builtin_amdgcn_cvt_f32_fp8((int)static_cast<const uint8_t*>(p)[i], 0);
}

template <typename T, int FORMAT, int D>
__global__ __launch_bounds__(kThreads) void attention_kernel(AttentionArgs a, Divisor block) {
    constexpr int N = D / 64;
    const int lane = threadIdx.x & 63, H = a.cache.num_heads, group = a.H_q / H;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64;
    const int64_t token = unit / a.H_q;
    const int head = (int)(unit - token * a.H_q), h = head / group;
    if (token >= a.total_tokens) return;
    T* o = static_cast<T*>(a.o) + (token * a.H_q + head) * D;
    int seq, past;
    uint64_t mask = 0;
    if (a.tokens_per_row > 0) {
        seq = (int)(token / a.tokens_per_row);
        past = a.past[seq];
        const int i = (int)(token - (int64_t)seq * a.tokens_per_row);
        const uint64_t all = a.tokens_per_row == 64 ? ~0ull : (1ull << a.tokens_per_row) - 1;
        mask = a.tree_mask ? (uint64_t)a.tree_mask[token] & all : (i == 63 ? ~0ull : (2ull << i) - 1);
        if (past < 0) { past = 0; mask = 0; }
    } else {
        int lo = 0, hi = a.num_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (a.cu_seqlens[mid] <= token) lo = mid; else hi = mid;
        }
        seq = lo;
        if (token < a.cu_seqlens[seq] || token >= a.cu_seqlens[seq + 1]) return;
        past = a.past ? max(a.past[seq], 0) : 0;
        const int64_t seen = (int64_t)past + (token - a.cu_seqlens[seq]) + 1;
        past = (int)(seen < a.capacity ? seen : a.capacity);
    }
    const dev::Pages pages = {a.table + (int64_t)seq * a.table_width, a.table_width, block, a.cache.num_rows};
    float q[N], acc[N] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = (float)static_cast<const T*>(a.q)[token * a.q_stride + (int64_t)head * D + lane + 64 * i];
    const int64_t end = (int64_t)past + (mask ? 64 - __builtin_clzll(mask) : 0);
    const int keys = (int)(end < a.capacity ? end : a.capacity);
    if (a.tokens_per_row > 0 && keys > a.max_keys) l = NAN;
    else
        for (int p = 0; p < keys; ++p) {
            if (p >= past && !(mask >> (p - past) & 1)) continue;
            const int64_t row = pages.row(p);
            if (row < 0) continue;
            const int64_t at = (row * H + h) * D + lane;
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) s = fmaf(q[i], cached<T, FORMAT>(a.cache.k, at + 64 * i), s);
            s = dev::group_sum(s, 64) * a.scale;
            float vs = 1.f;
            if constexpr (FORMAT != GDN_CACHE_PLAIN) {
                s *= a.cache.k_scale[row * H + h];
                vs = a.cache.v_scale[row * H + h];
            }
            const float next = fmaxf(m, s), keep = expf(m - next), w = expf(s - next);
            m = next;
            l = l * keep + w;
#pragma unroll
            for (int i = 0; i < N; ++i) acc[i] = acc[i] * keep + w * vs * cached<T, FORMAT>(a.cache.v, at + 64 * i);
        }
#pragma unroll
    for (int i = 0; i < N; ++i) o[lane + 64 * i] = (T)(l == 0.f ? 0.f : acc[i] / l);
}

template <typename T, int FORMAT, int D>
hipError_t launch(const AttentionArgs& a, hipStream_t stream) {
    const int64_t blocks = (a.total_tokens * a.H_q + kThreads / 64 - 1) / (kThreads / 64);
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    attention_kernel<T, FORMAT, D><<<(unsigned)blocks, kThreads, 0, stream>>>(a, Divisor((uint32_t)a.kv_block));
    return hipGetLastError();
}

template <typename T, int FORMAT>
hipError_t launch(const AttentionArgs& a, hipStream_t stream) {
    if (a.cache.head_dim == 64) return launch<T, FORMAT, 64>(a, stream);
    if (a.cache.head_dim == 128) return launch<T, FORMAT, 128>(a, stream);
    return launch<T, FORMAT, 256>(a, stream);
}

template <typename T>
hipError_t launch(const AttentionArgs& a, hipStream_t stream) {
    if (a.cache.format == GDN_CACHE_PLAIN) return launch<T, GDN_CACHE_PLAIN>(a, stream);
    if (a.cache.format == GDN_CACHE_E4M3) return launch<T, GDN_CACHE_E4M3>(a, stream);
    return launch<T, GDN_CACHE_INT8>(a, stream);
}

hipError_t launch(const AttentionArgs& a, hipStream_t stream) {
    return a.cache.dtype == GDN_BF16 ? launch<__bf16>(a, stream) : launch<float>(a, stream);
}

}  // namespace

size_t attention_workspace_bytes(int, int, int, int, int, int64_t) { return 0; }
hipError_t launch_attention_prefill(const AttentionArgs& a, hipStream_t stream) { return launch(a, stream); }
hipError_t launch_attention_decode(const AttentionArgs& a, hipStream_t stream) { return launch(a, stream); }

}  // namespace gdn
