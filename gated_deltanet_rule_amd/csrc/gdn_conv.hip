// gdn_conv.hip -- short causal convolution with SiLU and per-head L2 norm for gfx950.
//
//     a_t = bias + sum_{j < W} w_j x_{t - W + 1 + j},  u = silu(a),  y = u / sqrt(sum_head u^2 + eps)
//
// Memory-bound: every input is read and every output written once.  A lane owns one
// 16-byte vector of channels, a wave 64 of them, and walks a tile of tokens with the last
// W - 1 inputs and the weights in registers, so only the W - 1 rows before a tile are read
// twice.  The inputs of the next kGroup tokens are in flight while kGroup are computed.  A
// head's sum of squares goes over the lanes that hold it.
//
// A sequence's old state is read, and its final state written, by the tile that holds its
// first token: that tile also takes the first W - 1 tokens where they reach beyond it, so
// no other one reads the old state and a resume in place needs no second launch.
//
// 8 prompts of 64 to 4096 tokens, 8192 channels, bf16, states kept every 64 tokens: 149 us,
// 3.75 TB/s (a large copy: 6.6).  The vector ALU is busy 55 % of that, half of it the SiLU's
// two quarter-rate instructions; at the 137 registers of width 4 three waves fit on a SIMD.
// Measured beside it and no faster: four waves with spills (153 us), tiles of 64 tokens (157)
// or as long as one round of resident workgroups takes (152), a tile's pieces side by side in
// the grid (149).
#include <hip/hip_runtime.h>

#include "gdn_device.h"
#include "gdn_internal.h"
#include "gdn_layer_device.h"
#include "gdn_layer_internal.h"

namespace gdn {
namespace {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kGroup = 4;
constexpr int kTile = 32;     // most tokens of a tile

// Runs are cut into pieces of 64 vectors, each run's own, so that heads start at multiples
// of their lanes.
template <typename T>
int pieces(const ConvArgs& a) {
    constexpr int W = 64 * dev::kVec<T>;
    int n = 0;
    for (int i = 0; i < 3; ++i) n += (a.channels[i] + W - 1) / W;
    return n;
}

// Where a lane's channels are: the run, the channel within it, the channel of x.
struct Channels {
    int seg, ch, c;
};

template <typename T>
__device__ __forceinline__ bool channels_of(const ConvArgs& a, int piece, Channels& w) {
    constexpr int W = 64 * dev::kVec<T>;
    int base = 0;
    for (w.seg = 0; w.seg < 3; ++w.seg) {
        const int n = (a.channels[w.seg] + W - 1) / W;
        if (piece < n) break;
        piece -= n;
        base += a.channels[w.seg];
    }
    if (w.seg == 3) return false;
    w.ch = piece * W + (threadIdx.x & 63) * dev::kVec<T>;
    w.c = base + w.ch;
    return w.ch < a.channels[w.seg];
}

__device__ __forceinline__ int slot_or_none(const int32_t* slots, int64_t i, int num_slots) {
    const int s = slots[i];
    return s >= 0 && s < num_slots ? s : -1;
}

// Weights and bias of a lane's channels, and the outputs from W inputs, oldest first.
template <typename T, int W>
struct Taps {
    static constexpr int V = dev::kVec<T>;
    float w[V * W], b[V];

    __device__ __forceinline__ void load(const ConvArgs& a, int c) {
        dev::load_floats(a.weight + (size_t)c * W, w);
        if (a.bias) {
            dev::load_floats(a.bias + c, b);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) b[e] = 0.f;
        }
    }

    // Outputs of N tokens from their W - 1 + N inputs.  The lanes of a head are consecutive and
    // either all active or all not; the tokens' sums go over them side by side.
    template <int N>
    __device__ __forceinline__ void apply(const ConvArgs& a, int l2_dim, const float (*in)[V], float (&u)[N][V]) const {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
                u[k][e] = b[e];
#pragma unroll
                for (int j = 0; j < W; ++j) u[k][e] = fmaf(w[e * W + j], in[k + j][e], u[k][e]);
            }
        if (a.silu)
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int e = 0; e < V; ++e) u[k][e] = dev::silu(u[k][e]);
        if (l2_dim > 0) {
            float s[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                s[k] = 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) s[k] = fmaf(u[k][e], u[k][e], s[k]);
            }
            dev::group_sums(s, l2_dim / V);
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float r = dev::inv_sqrt(s[k] + a.l2_eps);
#pragma unroll
                for (int e = 0; e < V; ++e) u[k][e] *= r;
            }
        }
    }
};

// Input at local position pos of a sequence, the state's rows below 0 (zeros without one).
// At W = 4 a wave reads three of them where it enters a sequence.
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

// The state before local position pos: the W - 1 inputs that end there.
template <typename T, int W>
__device__ __forceinline__ void copy_state(const ConvArgs& a, T* dst, int64_t lo, int64_t pos, int slot, int c) {
    float rows[W - 1][dev::kVec<T>];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) input_at<T, W>(a, lo, pos - (W - 1) + j, slot, c, rows[j]);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) dev::store_vec(dst + (size_t)j * a.C + c, rows[j]);
}

// Where export idx goes, or NULL.
template <typename T, int W>
__device__ __forceinline__ T* export_to(const ConvArgs& a, int64_t idx) {
    if (idx < 0 || idx >= a.export_capacity) return nullptr;
    if (!a.export_slots) return static_cast<T*>(a.export_states) + (size_t)idx * (W - 1) * a.C;
    const int s = slot_or_none(a.export_slots, idx, a.num_slots);
    return s >= 0 ? static_cast<T*>(a.pool) + (size_t)s * (W - 1) * a.C : nullptr;
}

template <typename T, int W>
__global__ __launch_bounds__(kThreads) void conv_prefill_kernel(ConvArgs a, int tile) {
    constexpr int V = dev::kVec<T>;
    Channels w;
    if (!channels_of<T>(a, blockIdx.y * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w)) return;
    const int64_t t0 = (int64_t)blockIdx.x * tile, t1 = t0 + tile < a.total_tokens ? t0 + tile : a.total_tokens;
    const bool last = blockIdx.x + 1 == gridDim.x;
    Taps<T, W> taps;
    if (a.total_tokens > 0) taps.load(a, w.c);
    const int seg = __builtin_amdgcn_readfirstlane(w.seg), l2_dim = a.l2_dim[seg], width = a.channels[seg];
    // the first sequence that starts at t0 or later
    int i = 0;
    {
        int h = a.num_seqs;
        while (i < h) {
            const int mid = (i + h) >> 1;
            if (a.cu_seqlens[mid] >= t0) h = mid;
            else i = mid + 1;
        }
        i = __builtin_amdgcn_readfirstlane(i);
    }
    // the sequence that is under way at t0, then those that start in this tile
    for (i = i > 0 ? i - 1 : 0; i < a.num_seqs; ++i) {
        int lo, len;
        dev::seq_range(a.cu_seqlens, i, a.total_tokens, lo, len);
        lo = __builtin_amdgcn_readfirstlane(lo);
        len = __builtin_amdgcn_readfirstlane(len);
        if (lo >= t1 && !last) break;
        const bool owned = lo >= t0;
        const int64_t hi = (int64_t)lo + len;
        // local positions of this tile: an owned sequence's first W - 1 tokens are all its tile's
        int64_t from = owned ? 0 : t0 - lo, to = (hi < t1 ? hi : t1) - lo;
        if (!owned && from < W - 1) from = W - 1;
        if (owned && to < W - 1) to = len < W - 1 ? len : W - 1;
        const int slot = owned ? slot_or_none(a.init_slot, i, a.num_slots) : -1;
        if (from < to) {
            // Rows as buffers of their own, empty past the tile's last one: loads there give zeros,
            // stores are dropped, and no branch stands between the loads and their use.
            float in[W - 1 + kGroup][V];
            u32x4 next[kGroup];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) input_at<T, W>(a, lo, from - (W - 1) + j, slot, w.c, in[j]);
            const T* x = static_cast<const T*>(a.x);
            T* y = static_cast<T*>(a.y[seg]);
            auto row = [&](const void* base, int64_t p, int64_t stride, int width) {
                return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(static_cast<const T*>(base) + (p < to ? lo + p : 0) * stride), (short)0,
                                                         p < to ? width * (int)sizeof(T) : 0, 0x00020000);
            };
            auto fetch = [&](int64_t p) {
#pragma unroll
                for (int k = 0; k < kGroup; ++k)
                    next[k] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(row(x, p + k, a.x_stride, a.C), w.c * (int)sizeof(T), 0, 0));
            };
            fetch(from);
            for (int64_t p = from; p < to; p += kGroup) {
#pragma unroll
                for (int k = 0; k < kGroup; ++k) dev::widen_vec<T>(next[k], in[W - 1 + k]);
                fetch(p + kGroup);
                float u[kGroup][V];
                taps.apply(a, l2_dim, in, u);
#pragma unroll
                for (int k = 0; k < kGroup; ++k)
                    __builtin_amdgcn_raw_buffer_store_b128(dev::narrow_vec<T>(u[k]), row(y, p + k, width, width), w.ch * (int)sizeof(T), 0, 0);
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
#pragma unroll
                    for (int e = 0; e < V; ++e) in[j][e] = in[kGroup + j][e];
            }
        }
        if (a.export_grid > 0) {
            // the states after this tile's tokens, local positions (from, to]
            const int64_t s = a.start_pos ? a.start_pos[i] : 0, g = a.export_grid;
            for (int64_t p = ((s + from) / g + 1) * g; p <= s + to; p += g) {
                T* dst = export_to<T, W>(a, a.export_offsets[i] + p / g - s / g - 1);
                if (dst) copy_state<T, W>(a, dst, lo, p - s, slot, w.c);
            }
        }
        const int fin = owned ? slot_or_none(a.final_slot, i, a.num_slots) : -1;
        if (fin >= 0) copy_state<T, W>(a, static_cast<T*>(a.pool) + (size_t)fin * (W - 1) * a.C, lo, len, slot, w.c);
    }
}

// One token of each row: the same sums over the row's state and its token.
template <typename T, int W>
__global__ __launch_bounds__(kThreads) void conv_decode_kernel(ConvArgs a) {
    constexpr int V = dev::kVec<T>;
    Channels w;
    if (!channels_of<T>(a, blockIdx.y * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), w)) return;
    const int b = blockIdx.x;
    const int slot = slot_or_none(a.init_slot, b, a.num_slots), fin = slot_or_none(a.final_slot, b, a.num_slots);
    T* y = static_cast<T*>(a.y[w.seg]) + (size_t)b * a.channels[w.seg] + w.ch;
    float in[W][V], u[1][V];
    if (slot < 0) {                              // padding row
#pragma unroll
        for (int e = 0; e < V; ++e) u[0][e] = 0.f;
        dev::store_vec(y, u[0]);
        return;
    }
    Taps<T, W> taps;
    taps.load(a, w.c);
#pragma unroll
    for (int j = 0; j < W; ++j) input_at<T, W>(a, b, j - (W - 1), slot, w.c, in[j]);
    taps.apply(a, a.l2_dim[w.seg], in, u);
    dev::store_vec(y, u[0]);
    if (fin < 0) return;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) dev::store_vec(static_cast<T*>(a.pool) + ((size_t)fin * (W - 1) + j) * a.C + w.c, in[j + 1]);
}

template <typename T, int W>
hipError_t launch_typed(const ConvArgs& a, hipStream_t stream) {
    const unsigned p = (unsigned)pieces<T>(a), py = (p + kWaves - 1) / kWaves;
    if (!a.cu_seqlens) {
        if (!grid_fits(a.total_tokens, kThreads)) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL((conv_decode_kernel<T, W>), dim3((unsigned)a.total_tokens, py), dim3(kThreads), 0, stream, a);
        return hipGetLastError();
    }
    // Shorter tiles while the waves do not fill the card eight to a compute unit.
    int tile = kTile;
    while (tile > kGroup && (a.total_tokens + tile - 1) / tile * p < 8 * (int64_t)device_cus()) tile /= 2;
    const int64_t tiles = (a.total_tokens + tile - 1) / tile;
    if (!grid_fits(tiles, kThreads)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((conv_prefill_kernel<T, W>), dim3((unsigned)(tiles < 1 ? 1 : tiles), py), dim3(kThreads), 0, stream, a, tile);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_width(const ConvArgs& a, hipStream_t stream) {
    if (a.width == 4) return launch_typed<T, 4>(a, stream);
    if (a.width == 3) return launch_typed<T, 3>(a, stream);
    return launch_typed<T, 2>(a, stream);
}

}  // namespace

hipError_t launch_conv(const ConvArgs& a, hipStream_t stream) {
    return a.dtype == 1 ? launch_width<__bf16>(a, stream) : launch_width<float>(a, stream);
}

}  // namespace gdn
