// gdn_layer_device.h -- device helpers of the layer operators: 16-byte vectors of either
// dtype widened to fp32, activations and the step size of the scan.
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

__device__ __forceinline__ void load_vec(const float* p, float (&v)[4]) {
    const f32x4_t x = *reinterpret_cast<const f32x4_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x[i];
}
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

__device__ __forceinline__ float sigmoid(float v) { return 1.f / (1.f + expf(-v)); }
__device__ __forceinline__ float silu(float v) { return v / (1.f + expf(-v)); }

// log(1 + e^v) without overflow
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

}  // namespace dev
}  // namespace gdn
