// gdn_kv_cache.hip -- keys and values into and out of a paged cache, for gfx950.
//
//     s = max(|x|, 2^-100) / M,   code = round(x / s)     for each head of a token, M = 448 or 127
//
// Memory-bound: every value crosses HBM once each way.  LPH lanes share a head, 8 values to a
// lane (bf16: one 16-byte vector), so a head's largest value takes log2(LPH) steps across lanes
// and K and V of a head are in flight together.
// 131072 tokens of 8 heads of 128 dims, bf16 to 8 bits, into rows at random / pages of 16 rows / in order: written in 173 / 169 /
// 162 us (4.7 to 5.0 TB/s; an even copy reaches 6.57), read in 159 / 157 / 138 (5.1 to 5.9); plain 215 / 214 / 201 and 208 / 208 / 183.
// Where the rows lie costs little; what else keeps the write from the copy's rate is not isolated.  Four heads to a thread instead of
// one, for more loads in flight: 342 us both ways instead of 328.
#include <hip/hip_runtime.h>

#include "gdn_attention_internal.h"
#include "gdn_layer_device.h"
#include "gdn_layer_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));

// 8 values of T, widened
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    constexpr int V = dev::kVec<T>;
#pragma unroll
    for (int i = 0; i < 8; i += V) {
        float q[V];
        dev::load_vec(p + i, q);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i + j] = q[j];
    }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
    constexpr int V = dev::kVec<T>;
#pragma unroll
    for (int i = 0; i < 8; i += V) {
        float q[V];
#pragma unroll
        for (int j = 0; j < V; ++j) q[j] = v[i + j];
        dev::store_vec(p + i, q);
    }
}

// Largest of each aligned group of `lanes` lanes (a power of two).
__device__ __forceinline__ unsigned group_max(unsigned x, int lanes) {
    const auto with = [&](unsigned y) { x = x > y ? x : y; };
    const auto move = [&](auto f) { with(__builtin_bit_cast(unsigned, f(__builtin_bit_cast(float, x)))); };
    if (lanes > 1) move([](float f) { return dev::dpp_move<0xB1>(f); });
    if (lanes > 2) move([](float f) { return dev::dpp_move<0x4E>(f); });
    if (lanes > 4) move([](float f) { return dev::dpp_move<0x141>(f); });
    if (lanes > 8) move([](float f) { return dev::dpp_move<0x140>(f); });
    if (lanes > 16) with((unsigned)__shfl_xor((int)x, 16));
    if (lanes > 32) with((unsigned)__shfl_xor((int)x, 32));
    return x;
}

// x / by, correctly rounded, for finite x and by > 0, given the correctly rounded 1 / by: two steps on the remainder, of which
// the first gives a neighbour of the quotient and the second the nearest (Markstein's theorem), in five instructions where a division
// of its own takes eleven.  A remainder that underflows belongs to a quotient that is far below every code's half step.
__device__ __forceinline__ float divide(float x, float by, float inverse) {
    float q = x * inverse;
    q = fmaf(fmaf(-q, by, x), inverse, q);
    q = fmaf(fmaf(-q, by, x), inverse, q);
    return copysignf(q, x);                // (a negative zero)
}

template <int FORMAT>
__device__ __forceinline__ u32x2_t codes8(const float (&x)[8], float scale) {
    constexpr float M = FORMAT == GDN_CACHE_E4M3 ? 448.f : 127.f;
    const float inverse = 1.f / scale;
    u32x2_t w = {0u, 0u};
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_amdgcn_fmed3f(divide(x[i], scale, inverse), -M, M);
    if constexpr (FORMAT == GDN_CACHE_E4M3) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            int p = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
            w[i] = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], p, true);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i / 4] |= (unsigned)((int)rintf(v[i]) & 255) << (8 * (i & 3));
    }
    return w;
}

template <int FORMAT>
__device__ __forceinline__ void values8(u32x2_t w, float scale, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (FORMAT == GDN_CACHE_E4M3) {
            const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
            v[4 * i] = lo[0] * scale; v[4 * i + 1] = lo[1] * scale;
            v[4 * i + 2] = hi[0] * scale; v[4 * i + 3] = hi[1] * scale;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = (float)(int8_t)(w[i] >> (8 * j)) * scale;
        }
    }
}

// One head of a token to each group of LPH lanes.
template <typename T, int FORMAT, int LPH>
__global__ __launch_bounds__(kThreads) void write_kernel(CacheCopyArgs a) {
    const int lane = threadIdx.x % LPH, H = a.cache.num_heads, d = a.cache.head_dim;
    const unsigned idx = blockIdx.x * (kThreads / LPH) + threadIdx.x / LPH;
    const int64_t token = idx / (unsigned)H;
    const int h = (int)(idx - (unsigned)token * (unsigned)H), e = lane * 8;
    if (token >= a.num_tokens) return;
    const int64_t slot = a.slots[token];
    if (slot < 0 || slot >= a.cache.num_rows) return;
    void* const cache[2] = {a.cache.k, a.cache.v};
    float* const scales[2] = {a.cache.k_scale, a.cache.v_scale};
    float x[2][8] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (e < d) load8(static_cast<const T*>(a.in[i]) + token * a.in_stride[i] + (int64_t)h * d + e, x[i]);
    const int64_t head = slot * H + h;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (FORMAT == GDN_CACHE_PLAIN) {
            if (e < d) store8(static_cast<T*>(cache[i]) + head * d + e, x[i]);
        } else {
            // as bits, which order like the magnitudes and put infinities and NaN on top
            unsigned top = 0u;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const unsigned v = __builtin_bit_cast(unsigned, x[i][j]) & 0x7fffffffu;
                top = top > v ? top : v;
            }
            const float most = __builtin_bit_cast(float, group_max(top, LPH));
            const bool finite = most < INFINITY;
            const float scale = finite ? fmaxf(most, 0x1p-100f) / (FORMAT == GDN_CACHE_E4M3 ? 448.f : 127.f) : NAN;
            u32x2_t w = {0u, 0u};
            if (finite) w = codes8<FORMAT>(x[i], scale);
            if (e < d) *reinterpret_cast<u32x2_t*>(static_cast<char*>(cache[i]) + head * d + e) = w;
            if (lane == 0) scales[i][head] = scale;
        }
    }
}

template <typename T, int FORMAT, int LPH>
__global__ __launch_bounds__(kThreads) void read_kernel(CacheCopyArgs a) {
    const int lane = threadIdx.x % LPH, H = a.cache.num_heads, d = a.cache.head_dim;
    const unsigned idx = blockIdx.x * (kThreads / LPH) + threadIdx.x / LPH;
    const int64_t token = idx / (unsigned)H;
    const int h = (int)(idx - (unsigned)token * (unsigned)H), e = lane * 8;
    if (token >= a.num_tokens || e >= d) return;
    const int64_t slot = a.slots[token];
    const bool present = slot >= 0 && slot < a.cache.num_rows;
    const int64_t head = (present ? slot : 0) * H + h;
    const void* const cache[2] = {a.cache.k, a.cache.v};
    const float* const scales[2] = {a.cache.k_scale, a.cache.v_scale};
    float x[2][8] = {};
    if (present) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (FORMAT == GDN_CACHE_PLAIN) load8(static_cast<const T*>(cache[i]) + head * d + e, x[i]);
            else
                values8<FORMAT>(*reinterpret_cast<const u32x2_t*>(static_cast<const char*>(cache[i]) + head * d + e), scales[i][head], x[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) store8(static_cast<T*>(a.out[i]) + (token * H + h) * d + e, x[i]);
}

template <typename T, int FORMAT, int LPH>
hipError_t launch(const CacheCopyArgs& a, bool write, hipStream_t stream) {
    constexpr int PER = kThreads / LPH;
    const int64_t heads = a.num_tokens * a.cache.num_heads;
    const int64_t blocks = (heads + PER - 1) / PER;
    if (heads > 0xffffffffLL - PER || !grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    if (write) write_kernel<T, FORMAT, LPH><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
    else read_kernel<T, FORMAT, LPH><<<(unsigned)blocks, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

template <typename T, int FORMAT>
hipError_t launch(const CacheCopyArgs& a, bool write, hipStream_t stream) {
    const int d = a.cache.head_dim;
    if (d <= 64) return launch<T, FORMAT, 8>(a, write, stream);
    if (d <= 128) return launch<T, FORMAT, 16>(a, write, stream);
    if (d <= 256) return launch<T, FORMAT, 32>(a, write, stream);
    return launch<T, FORMAT, 64>(a, write, stream);
}

template <typename T>
hipError_t launch(const CacheCopyArgs& a, bool write, hipStream_t stream) {
    if (a.cache.format == GDN_CACHE_PLAIN) return launch<T, GDN_CACHE_PLAIN>(a, write, stream);
    if (a.cache.format == GDN_CACHE_E4M3) return launch<T, GDN_CACHE_E4M3>(a, write, stream);
    return launch<T, GDN_CACHE_INT8>(a, write, stream);
}

hipError_t launch(const CacheCopyArgs& a, bool write, hipStream_t stream) {
    return a.cache.dtype == GDN_BF16 ? launch<__bf16>(a, write, stream) : launch<float>(a, write, stream);
}

}  // namespace

hipError_t launch_cache_write(const CacheCopyArgs& a, hipStream_t stream) { return launch(a, true, stream); }
hipError_t launch_cache_read(const CacheCopyArgs& a, hipStream_t stream) { return launch(a, false, stream); }

}  // namespace gdn
