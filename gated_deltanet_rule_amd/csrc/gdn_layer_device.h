// gdn_layer_device.h -- device helpers of the layer operators: 16-byte vectors of either
// dtype widened to fp32, activations, the step size of the scan, sums over lane groups.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {
namespace dev {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));

// Elements of T in 16 bytes.
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

// Four or eight fp32 values, 16-byte aligned.
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const f32x4_t x = *reinterpret_cast<const f32x4_t*>(p + i);
        v[i] = x[0]; v[i + 1] = x[1]; v[i + 2] = x[2]; v[i + 3] = x[3];
    }
}

__device__ __forceinline__ void load_vec(const float* p, float (&v)[4]) { load_floats(p, v); }
__device__ __forceinline__ void load_vec(const __bf16* p, float (&v)[8]) {
    const bf16x8_t x = *reinterpret_cast<const bf16x8_t*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)x[i];
}
__device__ __forceinline__ void store_vec(float* p, const float (&v)[4]) {
    f32x4_t x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = v[i];
    *reinterpret_cast<f32x4_t*>(p) = x;
}
__device__ __forceinline__ void store_vec(__bf16* p, const float (&v)[8]) {
    bf16x8_t x;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (__bf16)v[i];
    *reinterpret_cast<bf16x8_t*>(p) = x;
}

// The same from and to 16 bytes in registers.
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
template <typename T>
__device__ __forceinline__ void widen_vec(u32x4_t w, float (&v)[kVec<T>]) {
    if constexpr (sizeof(T) == 4) {
        const f32x4_t x = __builtin_bit_cast(f32x4_t, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = x[i];
    } else {
        const bf16x8_t x = __builtin_bit_cast(bf16x8_t, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)x[i];
    }
}
template <typename T>
__device__ __forceinline__ u32x4_t narrow_vec(const float (&v)[kVec<T>]) {
    if constexpr (sizeof(T) == 4) {
        return __builtin_bit_cast(u32x4_t, f32x4_t{v[0], v[1], v[2], v[3]});
    } else {
        bf16x8_t x;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (__bf16)v[i];
        return __builtin_bit_cast(u32x4_t, x);
    }
}

// e^v as 2^(v log2 e): one rounding of the exponent (|v| 2^-24 relative) and the hardware's
// exp2, good to one unit in the last place; 0 and infinity where the exponent leaves fp32.
__device__ __forceinline__ float exp_fast(float v) { return __builtin_amdgcn_exp2f(v * 1.4426950408889634f); }

// 1 / (1 + e^-v) and v / (1 + e^-v).  The reciprocal is the hardware's (one unit in the
// last place): with the library's exp and division the activation, not memory, bounds the
// kernels that use it.
__device__ __forceinline__ float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.f + exp_fast(-v)); }
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }

// 1 / sqrt(v) of a sum of squares.  Sums below fp32's normal range count as its smallest
// number (the hardware instruction does not take subnormals); NaN stays NaN.
__device__ __forceinline__ float inv_sqrt(float v) { return __builtin_amdgcn_rsqf(v < 1.17549435e-38f ? 1.17549435e-38f : v); }

// log(1 + e^v) without overflow
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

template <int CTRL>
__device__ __forceinline__ float dpp_move(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// Sum over each aligned group of `lanes` (a power of two) lanes, the same bits in all of
// them: every step adds two values that are uniform over the halves it joins.
__device__ __forceinline__ float group_sum(float x, int lanes) {
    if (lanes > 1) x += dpp_move<0xB1>(x);     // quad_perm [1,0,3,2]
    if (lanes > 2) x += dpp_move<0x4E>(x);     // quad_perm [2,3,0,1]
    if (lanes > 4) x += dpp_move<0x141>(x);    // row_half_mirror
    if (lanes > 8) x += dpp_move<0x140>(x);    // row_mirror
    if (lanes > 16) x += __shfl_xor(x, 16);
    if (lanes > 32) x += __shfl_xor(x, 32);
    return x;
}

// group_sum of N values side by side.
template <int N>
__device__ __forceinline__ void group_sums(float (&x)[N], int lanes) {
#define GDN_EACH(term) _Pragma("unroll") for (int k = 0; k < N; ++k) x[k] += term
    if (lanes > 1) GDN_EACH(dpp_move<0xB1>(x[k]));
    if (lanes > 2) GDN_EACH(dpp_move<0x4E>(x[k]));
    if (lanes > 4) GDN_EACH(dpp_move<0x141>(x[k]));
    if (lanes > 8) GDN_EACH(dpp_move<0x140>(x[k]));
    if (lanes > 16) GDN_EACH(__shfl_xor(x[k], 16));
    if (lanes > 32) GDN_EACH(__shfl_xor(x[k], 32));
#undef GDN_EACH
}

}  // namespace dev
}  // namespace gdn
