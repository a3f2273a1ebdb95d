// gdn_norm.hip -- the norms around a recurrent block for gfx950.
//
//     gated:     y = rms(x) w act(z)  or  rms(x act(z)) w,   rms(v) = v / sqrt(mean(v^2) + eps)
//     residual:  r' = r + s act(gate) (rms(x) w_post),  y = rms(r') w_pre
//
// Memory-bound.  One workgroup per row (or per group of a row); a row's squares are
// summed per thread, then over the wave and the four waves in a fixed order.
#include <hip/hip_runtime.h>

#include "gdn_layer_device.h"
#include "gdn_layer_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float gate_of(float z, int activation) {
    return activation == 1 ? dev::silu(z) : activation == 2 ? dev::sigmoid(z) : z;
}

__device__ __forceinline__ float block_sum(float x, float* sums) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = x;
    __syncthreads();
    return (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void gated_norm_kernel(GatedNormArgs a) {
    __shared__ float sums[kThreads / 64];
    const int64_t row = blockIdx.x / a.groups;
    const int g = (int)(blockIdx.x - row * a.groups);
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride + (size_t)g * a.dim;
    const T* z = a.z ? static_cast<const T*>(a.z) + row * a.z_stride + (size_t)g * a.dim : nullptr;
    const float* w = a.weight + (a.weight_per_group ? (size_t)g * a.dim : 0);
    T* y = static_cast<T*>(a.y) + ((size_t)row * a.groups + g) * a.dim;
    float s = 0.f;
    for (int i = threadIdx.x; i < a.dim; i += kThreads) {
        float v = (float)x[i];
        if (a.gate_first && z) v *= gate_of((float)z[i], a.activation);
        s = fmaf(v, v, s);
    }
    const float r = 1.f / sqrtf(block_sum(s, sums) / a.dim + a.eps);
    for (int i = threadIdx.x; i < a.dim; i += kThreads) {
        const float gate = z ? gate_of((float)z[i], a.activation) : 1.f;
        y[i] = (T)((float)x[i] * gate * r * w[i]);
    }
}

template <typename T, typename R>
__global__ __launch_bounds__(kThreads) void residual_norm_kernel(ResidualNormArgs a) {
    __shared__ float sums[kThreads / 64];
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* z = a.gate ? static_cast<const T*>(a.gate) + row * a.gate_stride : nullptr;
    const R* res = static_cast<const R*>(a.residual) + (size_t)row * a.dim;
    R* out = static_cast<R*>(a.residual_out) + (size_t)row * a.dim;
    float post = 1.f;
    if (a.post_weight) {
        float s = 0.f;
        for (int i = threadIdx.x; i < a.dim; i += kThreads) s = fmaf((float)x[i], (float)x[i], s);
        post = 1.f / sqrtf(block_sum(s, sums) / a.dim + a.eps);
    }
    float s = 0.f;
    for (int i = threadIdx.x; i < a.dim; i += kThreads) {
        float v = (float)x[i] * post;
        if (a.post_weight) v *= a.post_weight[i];
        if (z) v *= gate_of((float)z[i], a.activation);
        const R o = (R)fmaf(a.residual_scale, v, (float)res[i]);
        out[i] = o;
        s = fmaf((float)o, (float)o, s);
    }
    if (!a.y) return;
    const float pre = 1.f / sqrtf(block_sum(s, sums) / a.dim + a.eps);
    T* y = static_cast<T*>(a.y) + (size_t)row * a.dim;
    for (int i = threadIdx.x; i < a.dim; i += kThreads) y[i] = (T)((float)out[i] * pre * a.pre_weight[i]);
}

}  // namespace

hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)(a.num_rows * a.groups));
    if (a.dtype == 1) hipLaunchKernelGGL((gated_norm_kernel<__bf16>), grid, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((gated_norm_kernel<float>), grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_residual_norm(const ResidualNormArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)a.num_rows);
    if (a.dtype == 0) hipLaunchKernelGGL((residual_norm_kernel<float, float>), grid, dim3(kThreads), 0, stream, a);
    else if (a.residual_dtype == 0) hipLaunchKernelGGL((residual_norm_kernel<__bf16, float>), grid, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((residual_norm_kernel<__bf16, __bf16>), grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdn
