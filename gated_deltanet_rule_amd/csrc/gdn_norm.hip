// gdn_norm.hip -- the norms around a recurrent block for gfx950.
//
//     gated:     y = rms(x) w act(z)  or  rms(x act(z)) w,   rms(v) = v / sqrt(mean(v^2) + eps)
//     residual:  r' = r + s act(gate) (rms(x) w_post),  y = rms(r') w_pre
//
// Memory-bound: every operand crosses HBM once.  The values of a norm stay in registers
// between its sum and its output; TPG threads share one norm, R vectors of V elements each,
// as many vectors as its dim needs: one lane, 16 lanes (four norms to a wave), one wave,
// then one workgroup of four or sixteen waves.  A sum is taken per thread in order, then
// over the lanes and the waves in a fixed tree, so a row's bits depend on its dim alone.
// 131072 x 32 gated rows of 128 bf16 values: 554 us, 5.8 TB/s; 16384 residual rows of 4096 with
// an fp32 residual: 174 us, 5.4 TB/s (a large copy: 6.6 TB/s; two arrays added into a third by
// torch: 6.05).  Rows of any other dim or alignment take unaligned vectors: 6709 residual rows
// of 5001 bf16 values 118 us (element by element: 261), 4096 gated rows of 4096 at an odd stride
// 24 us (96).
#include <hip/hip_runtime.h>

#include "gdn_layer_device.h"
#include "gdn_layer_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// Global memory takes vectors at any element's address, so a row that starts or ends anywhere
// costs little more than an aligned one.  Vectors of a row whose last one is not whole: that
// one is moved back to end with the row, and its first `skip` elements, which the vector
// before holds too, are left out of sums (both lanes compute and store the same values).
struct Place {
    int e, skip;
};
template <int V, bool WIDE>
__device__ __forceinline__ Place place(int e, int dim) {
    if (WIDE || dim < V || e + V <= dim) return {e, 0};
    return {dim - V, e + V - dim};
}

template <int V, bool WIDE>
__device__ __forceinline__ float add_squares(const float (&x)[V], int skip, float s) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float v = WIDE || i >= skip ? x[i] : 0.f;
        s = fmaf(v, v, s);
    }
    return s;
}

// V elements at p, of which `left` belong to the row: all of them but for rows shorter than V.
template <typename T, int V, bool WIDE>
__device__ __forceinline__ void load_some(const T* p, int left, float (&v)[V]) {
    constexpr int N = dev::kVec<T>;
    if (WIDE || left >= V) {
#pragma unroll
        for (int i = 0; i < V; i += N) {
            dev::u32x4_t w;
            float q[N];
            if constexpr (WIDE) w = *reinterpret_cast<const dev::u32x4_t*>(p + i);
            else __builtin_memcpy(&w, p + i, 16);
            dev::widen_vec<T>(w, q);
#pragma unroll
            for (int k = 0; k < N; ++k) v[i + k] = q[k];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = i < left ? (float)p[i] : 0.f;
    }
}

template <typename T, int V, bool WIDE>
__device__ __forceinline__ void store_some(T* p, int left, const float (&v)[V]) {
    constexpr int N = dev::kVec<T>;
    if (WIDE || left >= V) {
#pragma unroll
        for (int i = 0; i < V; i += N) {
            float q[N];
#pragma unroll
            for (int k = 0; k < N; ++k) q[k] = v[i + k];
            const dev::u32x4_t w = dev::narrow_vec<T>(q);
            if constexpr (WIDE) *reinterpret_cast<dev::u32x4_t*>(p + i) = w;
            else __builtin_memcpy(p + i, &w, 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < left) p[i] = (T)v[i];
    }
}

// V elements of T as values, v[] = q[] once the loads may be rounded to T in between
template <typename T, int V>
__device__ __forceinline__ void round_to(float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (float)(T)v[i];
}

template <int V>
__device__ __forceinline__ void gate(float (&z)[V], int activation) {
    if (activation == 1)
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = dev::silu(z[i]);
    else if (activation == 2)
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = dev::sigmoid(z[i]);
}

// Sum over the TPG threads of a norm.
template <int TPG>
__device__ __forceinline__ float norm_sum(float x, float* sums) {
    if constexpr (TPG <= 64) {
        return dev::group_sum(x, TPG);
    } else {
        x = dev::group_sum(x, 64);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = x;
        __syncthreads();
        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < TPG / 64; ++w) t[w & 3] += sums[w];
        return (t[0] + t[1]) + (t[2] + t[3]);
    }
}

// U norms per thread, all of their loads issued first.
template <typename T, bool WIDE, int TPG, int R, int U>
__global__ __launch_bounds__(TPG > kThreads ? TPG : kThreads) void gated_norm_kernel(GatedNormArgs a) {
    constexpr int V = dev::kVec<T>, PER = TPG > kThreads ? 1 : kThreads / TPG;
    __shared__ float sums[TPG > 64 ? TPG / 64 : 1];
    const unsigned total = (unsigned)(a.num_rows * a.groups);
    const int lane = threadIdx.x % TPG;
    const float inv_dim = 1.f / (float)a.dim;
    float x[U][R][V], z[U][R][V];
    unsigned idx[U], g[U];
    int64_t row[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        idx[u] = (blockIdx.x * U + u) * PER + threadIdx.x / TPG;
        row[u] = idx[u] / (unsigned)a.groups;
        g[u] = idx[u] - (unsigned)row[u] * (unsigned)a.groups;
        const T* px = static_cast<const T*>(a.x) + row[u] * a.x_stride + (size_t)g[u] * a.dim;
        const T* pz = static_cast<const T*>(a.z) + row[u] * a.z_stride + (size_t)g[u] * a.dim;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int e0 = (lane + r * TPG) * V, e = place<V, WIDE>(e0, a.dim).e;
            if (idx[u] < total && e0 < a.dim) {
                load_some<T, V, WIDE>(px + e, a.dim - e, x[u][r]);
                if (a.z) load_some<T, V, WIDE>(pz + e, a.dim - e, z[u][r]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) x[u][r][i] = z[u][r][i] = 0.f;
            }
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (a.z) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                gate(z[u][r], a.activation);
                if (a.gate_first)
#pragma unroll
                    for (int i = 0; i < V; ++i) x[u][r][i] *= z[u][r][i];
            }
        }
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) s = add_squares<V, WIDE>(x[u][r], place<V, WIDE>((lane + r * TPG) * V, a.dim).skip, s);
        const float n = dev::inv_sqrt(fmaf(norm_sum<TPG>(s, sums), inv_dim, a.eps));
        const float* pw = a.weight + (a.weight_per_group ? (size_t)g[u] * a.dim : 0);
        T* py = static_cast<T*>(a.y) + ((size_t)row[u] * a.groups + g[u]) * a.dim;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int e0 = (lane + r * TPG) * V, e = place<V, WIDE>(e0, a.dim).e;
            if (idx[u] < total && e0 < a.dim) {
                float w[V];
                load_some<float, V, WIDE>(pw + e, a.dim - e, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    w[i] *= x[u][r][i] * n;
                    if (a.z && !a.gate_first) w[i] *= z[u][r][i];
                }
                store_some<T, V, WIDE>(py + e, a.dim - e, w);
            }
        }
    }
}

template <typename T, typename RT, bool WIDE, int TPG, int R>
__global__ __launch_bounds__(TPG > kThreads ? TPG : kThreads) void residual_norm_kernel(ResidualNormArgs a) {
    constexpr int V = dev::kVec<T>, PER = TPG > kThreads ? 1 : kThreads / TPG;
    __shared__ float sums[TPG > 64 ? TPG / 64 : 1];
    const int64_t row = (int64_t)blockIdx.x * PER + threadIdx.x / TPG;
    const int lane = threadIdx.x % TPG;
    const bool live = row < a.num_rows;
    const float inv_dim = 1.f / (float)a.dim;
    const T* px = static_cast<const T*>(a.x) + row * a.x_stride;
    const T* pz = static_cast<const T*>(a.gate) + row * a.gate_stride;
    const RT* pr = static_cast<const RT*>(a.residual) + (size_t)row * a.dim;
    RT* po = static_cast<RT*>(a.residual_out) + (size_t)row * a.dim;
    float x[R][V], q[R][V], z[R][V];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e0 = (lane + r * TPG) * V, e = place<V, WIDE>(e0, a.dim).e;
        if (live && e0 < a.dim) {
            load_some<T, V, WIDE>(px + e, a.dim - e, x[r]);
            load_some<RT, V, WIDE>(pr + e, a.dim - e, q[r]);
            if (a.gate) load_some<T, V, WIDE>(pz + e, a.dim - e, z[r]);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) x[r][i] = q[r][i] = z[r][i] = 0.f;
        }
    }
    if (a.post_weight) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) s = add_squares<V, WIDE>(x[r], place<V, WIDE>((lane + r * TPG) * V, a.dim).skip, s);
        const float n = dev::inv_sqrt(fmaf(norm_sum<TPG>(s, sums), inv_dim, a.eps));
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int e0 = (lane + r * TPG) * V, e = place<V, WIDE>(e0, a.dim).e;
            if (e0 < a.dim) {
                float w[V];
                load_some<float, V, WIDE>(a.post_weight + e, a.dim - e, w);
#pragma unroll
                for (int i = 0; i < V; ++i) x[r][i] *= n * w[i];
            }
        }
    }
    // a residual in place: its shared elements are all read before one of them is written
    if (!WIDE && TPG > 64) __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e0 = (lane + r * TPG) * V;
        const Place at = place<V, WIDE>(e0, a.dim);
        const int e = at.e;
        if (a.gate) {
            gate(z[r], a.activation);
#pragma unroll
            for (int i = 0; i < V; ++i) x[r][i] *= z[r][i];
        }
#pragma unroll
        for (int i = 0; i < V; ++i) q[r][i] = fmaf(a.residual_scale, x[r][i], q[r][i]);
        round_to<RT>(q[r]);
        if (live && e0 < a.dim) {
            store_some<RT, V, WIDE>(po + e, a.dim - e, q[r]);
            s = add_squares<V, WIDE>(q[r], at.skip, s);
        }
    }
    if (!a.y) return;
    const float n = dev::inv_sqrt(fmaf(norm_sum<TPG>(s, sums), inv_dim, a.eps));
    T* py = static_cast<T*>(a.y) + (size_t)row * a.dim;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int e0 = (lane + r * TPG) * V, e = place<V, WIDE>(e0, a.dim).e;
        if (live && e0 < a.dim) {
            float w[V];
            load_some<float, V, WIDE>(a.pre_weight + e, a.dim - e, w);
#pragma unroll
            for (int i = 0; i < V; ++i) w[i] *= q[r][i] * n;
            store_some<T, V, WIDE>(py + e, a.dim - e, w);
        }
    }
}

template <typename T, bool WIDE, int TPG, int R>
hipError_t gated(const GatedNormArgs& a, hipStream_t stream) {
    constexpr int PER = TPG > kThreads ? 1 : kThreads / TPG, THREADS = TPG > kThreads ? TPG : kThreads;
    const int64_t n = (a.num_rows * a.groups + PER - 1) / PER;
    if (!grid_fits(n, THREADS)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((gated_norm_kernel<T, WIDE, TPG, R, 1>), dim3((unsigned)n), dim3(THREADS), 0, stream, a);
    return hipGetLastError();
}

// Threads and vectors by the number of vectors in a norm: the smallest that holds it.
template <typename T, bool WIDE>
hipError_t gated_by_dim(const GatedNormArgs& a, hipStream_t stream) {
    constexpr int V = dev::kVec<T>;
    const int n = (a.dim + V - 1) / V;
    if (n <= 1) return gated<T, WIDE, 1, 1>(a, stream);
    if (n <= 16) return gated<T, WIDE, 16, 1>(a, stream);
    if (n <= 64) return gated<T, WIDE, 64, 1>(a, stream);
    if (n <= 256) return gated<T, WIDE, 64, 4>(a, stream);
    if (n <= 1024) return gated<T, WIDE, 256, 4>(a, stream);
    return gated<T, WIDE, 1024, 4>(a, stream);
}

template <typename T, typename RT, bool WIDE, int TPG, int R>
hipError_t residual(const ResidualNormArgs& a, hipStream_t stream) {
    constexpr int PER = TPG > kThreads ? 1 : kThreads / TPG, THREADS = TPG > kThreads ? TPG : kThreads;
    const int64_t n = (a.num_rows + PER - 1) / PER;
    if (!grid_fits(n, THREADS)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((residual_norm_kernel<T, RT, WIDE, TPG, R>), dim3((unsigned)n), dim3(THREADS), 0, stream, a);
    return hipGetLastError();
}

template <typename T, typename RT, bool WIDE>
hipError_t residual_by_dim(const ResidualNormArgs& a, hipStream_t stream) {
    constexpr int V = dev::kVec<T>;
    const int n = (a.dim + V - 1) / V;
    if (n <= 1) return residual<T, RT, WIDE, 1, 1>(a, stream);
    if (n <= 16) return residual<T, RT, WIDE, 16, 1>(a, stream);
    if (n <= 64) return residual<T, RT, WIDE, 64, 1>(a, stream);
    if (n <= 256) return residual<T, RT, WIDE, 256, 1>(a, stream);
    if (n <= 512) return residual<T, RT, WIDE, 256, 2>(a, stream);
    if (n <= 1024) return residual<T, RT, WIDE, 256, 4>(a, stream);
    return residual<T, RT, WIDE, 1024, 4>(a, stream);
}

// Whether rows of `dim` elements at this address and row stride are whole, aligned 16-byte vectors.
bool wide(const void* p, int64_t stride, int64_t rows, int dim, size_t size) {
    const size_t v = 16 / size;
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && dim % v == 0 && (rows == 1 || stride % v == 0);
}

template <typename T, typename RT>
hipError_t residual_typed(const ResidualNormArgs& a, hipStream_t stream) {
    const bool ok = wide(a.x, a.x_stride, a.num_rows, a.dim, sizeof(T)) && wide(a.residual, a.dim, 1, a.dim, sizeof(T)) &&
                    wide(a.residual_out, a.dim, 1, a.dim, sizeof(T)) && (!a.y || wide(a.y, a.dim, 1, a.dim, sizeof(T))) &&
                    (!a.gate || wide(a.gate, a.gate_stride, a.num_rows, a.dim, sizeof(T))) &&
                    reinterpret_cast<uintptr_t>(a.post_weight) % 16 == 0 && reinterpret_cast<uintptr_t>(a.pre_weight) % 16 == 0;
    return ok ? residual_by_dim<T, RT, true>(a, stream) : residual_by_dim<T, RT, false>(a, stream);
}

template <typename T>
hipError_t gated_typed(const GatedNormArgs& a, hipStream_t stream) {
    const bool ok = wide(a.x, a.x_stride, a.num_rows, a.dim, sizeof(T)) && wide(a.y, a.dim, 1, a.dim, sizeof(T)) &&
                    (!a.z || wide(a.z, a.z_stride, a.num_rows, a.dim, sizeof(T))) && reinterpret_cast<uintptr_t>(a.weight) % 16 == 0;
    return ok ? gated_by_dim<T, true>(a, stream) : gated_by_dim<T, false>(a, stream);
}

}  // namespace

hipError_t launch_gated_norm(const GatedNormArgs& a, hipStream_t stream) {
    return a.dtype == 1 ? gated_typed<__bf16>(a, stream) : gated_typed<float>(a, stream);
}

hipError_t launch_residual_norm(const ResidualNormArgs& a, hipStream_t stream) {
    if (a.dtype == 0) return residual_typed<float, float>(a, stream);
    return a.residual_dtype == 0 ? residual_typed<__bf16, float>(a, stream) : residual_typed<__bf16, __bf16>(a, stream);
}

}  // namespace gdn
