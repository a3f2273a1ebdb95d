// gdn_conv.hip -- short causal convolution with SiLU and per-head L2 norm for gfx950.
//
//     a_t = bias + sum_{j < W} w_j x_{t - W + 1 + j},  u = silu(a),  y = u / sqrt(sum_head u^2 + eps)
//
// Memory-bound: every input is read and every output written once, two flops per tap in
// between.  A thread owns one 16-byte vector of channels of one token; a head's sum of
// squares is a butterfly over the lanes that hold it.  The states (the last W - 1 inputs)
// are written by a second launch, so that a sequence resumed in place reads its old state
// before it is replaced.
#include <hip/hip_runtime.h>

#include "gdn_device.h"
#include "gdn_layer_device.h"
#include "gdn_layer_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// The run and its first channel of channel block cb: runs are cut into blocks of
// kThreads vectors, each run's own, so that heads start at lane multiples.
template <typename T>
__device__ __forceinline__ bool channel_of(const ConvArgs& a, int cb, int& seg, int& ch, int& c) {
    constexpr int W = kThreads * dev::kVec<T>;
    int base = 0;
    for (seg = 0; seg < 3; ++seg) {
        const int n = (a.channels[seg] + W - 1) / W;
        if (cb < n) break;
        cb -= n;
        base += a.channels[seg];
    }
    if (seg == 3) return false;
    ch = cb * W + threadIdx.x * dev::kVec<T>;   // channel within the run
    c = base + ch;                              // channel of x
    return ch < a.channels[seg];
}

template <typename T>
int channel_blocks(const ConvArgs& a) {
    constexpr int W = kThreads * dev::kVec<T>;
    int n = 0;
    for (int i = 0; i < 3; ++i) n += (a.channels[i] + W - 1) / W;
    return n;
}

__device__ __forceinline__ int slot_or_none(const int32_t* slots, int i, int num_slots) {
    const int s = slots[i];
    return s >= 0 && s < num_slots ? s : -1;
}

// Activation and head norm of one vector.  The lanes of a head are consecutive and
// either all active or all not.
template <int V>
__device__ __forceinline__ void finish(const ConvArgs& a, int seg, float (&u)[V]) {
    if (a.silu)
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] = dev::silu(u[i]);
    if (a.l2_dim[seg] > 0) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) s = fmaf(u[i], u[i], s);
        for (int d = a.l2_dim[seg] / V / 2; d > 0; d >>= 1) s += __shfl_xor(s, d);
        const float r = 1.f / sqrtf(s + a.l2_eps);
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] *= r;
    }
}

// Input at local position pos of a sequence (its state below 0), as fp32.
template <typename T, int W, int V>
__device__ __forceinline__ void input_at(const ConvArgs& a, int64_t lo, int64_t pos, int slot, int c, float (&v)[V]) {
    if (pos >= 0) {
        dev::load_vec(static_cast<const T*>(a.x) + (size_t)(lo + pos) * a.x_stride + c, v);
    } else if (slot >= 0) {
        dev::load_vec(static_cast<const T*>(a.pool) + ((size_t)slot * (W - 1) + (W - 1 + pos)) * a.C + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
    }
}

template <typename T, int W>
__global__ __launch_bounds__(kThreads) void conv_kernel(ConvArgs a) {
    constexpr int V = dev::kVec<T>;
    int seg, ch, c;
    const bool live = channel_of<T>(a, blockIdx.y, seg, ch, c);
    if (!live) return;
    const int64_t t = blockIdx.x;
    // the token's sequence: the last one that starts at or before it
    int i, lo, len;
    if (a.cu_seqlens) {
        int l = 0, h = a.num_seqs - 1;
        while (l < h) {
            const int mid = (l + h + 1) >> 1;
            if (a.cu_seqlens[mid] <= t) l = mid;
            else h = mid - 1;
        }
        i = l;
        dev::seq_range(a.cu_seqlens, i, a.total_tokens, lo, len);
        if (t < lo || t >= lo + len) return;
    } else {
        i = lo = (int)t;
        len = 1;
    }
    const int slot = slot_or_none(a.init_slot, i, a.num_slots);
    T* y = static_cast<T*>(a.y[seg]) + (size_t)t * a.channels[seg] + ch;
    float u[V];
    if (!a.cu_seqlens && slot < 0) {            // padding row
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] = 0.f;
        dev::store_vec(y, u);
        return;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) u[e] = a.bias ? a.bias[c + e] : 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float v[V];
        input_at<T, W>(a, lo, t - lo - (W - 1) + j, slot, c, v);
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] = fmaf(a.weight[(size_t)(c + e) * W + j], v[e], u[e]);
    }
    finish(a, seg, u);
    dev::store_vec(y, u);
}

template <typename T, int W>
__global__ __launch_bounds__(kThreads) void conv_state_kernel(ConvArgs a) {
    constexpr int V = dev::kVec<T>;
    int seg, ch, c;
    if (!channel_of<T>(a, blockIdx.y, seg, ch, c)) return;
    const int64_t unit = blockIdx.x;
    float rows[W - 1][V];
    auto put = [&](T* dst) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) dev::store_vec(dst + (size_t)j * a.C + c, rows[j]);
    };
    // where export idx goes, or NULL
    auto export_to = [&](int64_t idx) -> T* {
        if (idx < 0 || idx >= a.export_capacity) return nullptr;
        if (!a.export_slots) return static_cast<T*>(a.export_states) + (size_t)idx * (W - 1) * a.C;
        const int s = a.export_slots[idx];
        return s >= 0 && s < a.num_slots ? static_cast<T*>(a.pool) + (size_t)s * (W - 1) * a.C : nullptr;
    };
    if (unit < a.num_seqs) {
        const int i = (int)unit;
        int lo = i, len = 1;
        if (a.cu_seqlens) dev::seq_range(a.cu_seqlens, i, a.total_tokens, lo, len);
        const int slot = slot_or_none(a.init_slot, i, a.num_slots);
        if (!a.cu_seqlens && slot < 0) return;
        if (a.export_grid > 0) {
            // an export within the first W - 1 tokens holds rows of the old state: it is
            // made here, before the final state may replace them
            const int64_t s = a.start_pos ? a.start_pos[i] : 0;
            const int64_t p = (s / a.export_grid + 1) * a.export_grid - s;
            if (p < W - 1 && p <= len) {
                T* dst = export_to(a.export_offsets[i]);
                if (dst) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) input_at<T, W>(a, lo, p - (W - 1) + j, slot, c, rows[j]);
                    put(dst);
                }
            }
        }
        const int fin = slot_or_none(a.final_slot, i, a.num_slots);
        if (fin < 0) return;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) input_at<T, W>(a, lo, (int64_t)len - (W - 1) + j, slot, c, rows[j]);
        put(static_cast<T*>(a.pool) + (size_t)fin * (W - 1) * a.C);
        return;
    }
    const int64_t idx = unit - a.num_seqs;
    if (idx >= a.export_offsets[a.num_seqs]) return;
    int l = 0, h = a.num_seqs - 1;
    while (l < h) {
        const int mid = (l + h + 1) >> 1;
        if (a.export_offsets[mid] <= idx) l = mid;
        else h = mid - 1;
    }
    int lo, len;
    dev::seq_range(a.cu_seqlens, l, a.total_tokens, lo, len);
    const int64_t s = a.start_pos ? a.start_pos[l] : 0;
    const int64_t p = (s / a.export_grid + 1 + idx - a.export_offsets[l]) * a.export_grid - s;
    if (p < W - 1 || p > len) return;
    T* dst = export_to(idx);
    if (!dst) return;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) input_at<T, W>(a, lo, p - (W - 1) + j, -1, c, rows[j]);
    put(dst);
}

template <typename T, int W>
hipError_t launch_typed(const ConvArgs& a, hipStream_t stream) {
    const unsigned cb = (unsigned)channel_blocks<T>(a);
    if (a.total_tokens > 0) {
        hipLaunchKernelGGL((conv_kernel<T, W>), dim3((unsigned)a.total_tokens, cb), dim3(kThreads), 0, stream, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((conv_state_kernel<T, W>), dim3((unsigned)(a.num_seqs + a.export_capacity), cb), dim3(kThreads), 0,
                       stream, a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_width(const ConvArgs& a, hipStream_t stream) {
    if (a.width == 4) return launch_typed<T, 4>(a, stream);
    if (a.width == 3) return launch_typed<T, 3>(a, stream);
    return launch_typed<T, 2>(a, stream);
}

}  // namespace

hipError_t launch_conv_prefill(const ConvArgs& a, hipStream_t stream) {
    return a.dtype == 1 ? launch_width<__bf16>(a, stream) : launch_width<float>(a, stream);
}

hipError_t launch_conv_decode(const ConvArgs& a, hipStream_t stream) { return launch_conv_prefill(a, stream); }

}  // namespace gdn
