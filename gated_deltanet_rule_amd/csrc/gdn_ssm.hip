// gdn_ssm.hip -- selective state space scan for gfx950, token by token.
//
//     d = softplus(dt + bias),  S <- e^(d A) S + d b x^T,  y = scale S^T c + D x
//
// A workgroup of 256 threads holds 64 columns of one head's state (d_k x 64 fp32) in
// registers: 16 threads of one float4 cover a row's columns, the 16 row groups hold
// every sixteenth row.  Each token decays the state, adds the outer product and sums
// S^T c over the row groups through LDS in a fixed order.  A decode row is one token; a
// packed sequence is walked from its first token to its last.
#include <hip/hip_runtime.h>

#include "gdn_device.h"
#include "gdn_layer_device.h"
#include "gdn_layer_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 64;

template <typename T, int DK, int DV>
__global__ __launch_bounds__(kThreads) void ssm_token_kernel(SsmArgs a) {
    constexpr int TPR = kCols / 4, RG = kThreads / TPR, R = DK / RG, NCW = DV / kCols;
    const int unit = blockIdx.x / NCW;
    const int col0 = kCols * (blockIdx.x - unit * NCW);
    const int i = unit / a.H_v, h = unit - i * a.H_v;
    const int kh = h / (a.H_v / a.H_k);
    const int tid = threadIdx.x, c4 = tid % TPR, rg = tid / TPR;
    const size_t SE = (size_t)DK * DV;

    const int sin = a.init_slot[i];
    const bool have = sin >= 0 && sin < a.num_slots;
    int lo = i, len = 1;
    if (a.cu_seqlens) dev::seq_range(a.cu_seqlens, i, a.total_tokens, lo, len);
    else if (!have) {                            // padding row
        T* y = static_cast<T*>(a.y) + ((size_t)i * a.H_v + h) * DV;
        if (tid < kCols) y[col0 + tid] = (T)0.f;
        return;
    }
    float4 s[R];
#pragma unroll
    for (int m = 0; m < R; ++m)
        s[m] = have ? *reinterpret_cast<const float4*>(a.pool + ((size_t)sin * a.H_v + h) * SE + (size_t)(rg + RG * m) * DV + col0 + 4 * c4)
                    : make_float4(0.f, 0.f, 0.f, 0.f);
    auto put = [&](float* state) {
#pragma unroll
        for (int m = 0; m < R; ++m) *reinterpret_cast<float4*>(state + (size_t)(rg + RG * m) * DV + col0 + 4 * c4) = s[m];
    };
    const int64_t pos0 = a.start_pos ? a.start_pos[i] : 0;
    int64_t next_export = a.export_grid > 0 ? (pos0 / a.export_grid + 1) * a.export_grid : 0, exported = 0;
    const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f, D = a.D ? a.D[h] : 0.f;

    __shared__ float bc[2][DK];
    __shared__ float4 red[RG][TPR];
    for (int t = 0; t < len; ++t) {
        const size_t row = (size_t)(lo + t);
        if (tid < DK) bc[0][tid] = (float)static_cast<const T*>(a.b)[(row * a.H_k + kh) * DK + tid];
        else if (tid < 2 * DK) bc[1][tid - DK] = (float)static_cast<const T*>(a.c)[(row * a.H_k + kh) * DK + tid - DK];
        const T* xp = static_cast<const T*>(a.x) + (row * a.H_v + h) * DV + col0 + 4 * c4;
        const float4 x = make_float4((float)xp[0], (float)xp[1], (float)xp[2], (float)xp[3]);
        const float raw = a.dt[row * a.H_v + h] + bias;
        const float d = a.dt_softplus ? dev::softplus(raw) : raw;
        const float decay = expf(d * A);
        __syncthreads();
        float4 p = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int m = 0; m < R; ++m) {
            const float db = d * bc[0][rg + RG * m], cr = bc[1][rg + RG * m];
            s[m].x = fmaf(db, x.x, decay * s[m].x); s[m].y = fmaf(db, x.y, decay * s[m].y);
            s[m].z = fmaf(db, x.z, decay * s[m].z); s[m].w = fmaf(db, x.w, decay * s[m].w);
            p.x = fmaf(s[m].x, cr, p.x); p.y = fmaf(s[m].y, cr, p.y);
            p.z = fmaf(s[m].z, cr, p.z); p.w = fmaf(s[m].w, cr, p.w);
        }
        red[rg][c4] = p;
        __syncthreads();
        if (rg == 0) {
            float4 o = red[0][c4];
#pragma unroll
            for (int r = 1; r < RG; ++r) {
                const float4 q = red[r][c4];
                o.x += q.x; o.y += q.y; o.z += q.z; o.w += q.w;
            }
            T* y = static_cast<T*>(a.y) + (row * a.H_v + h) * DV + col0 + 4 * c4;
            y[0] = (T)fmaf(D, x.x, a.scale * o.x); y[1] = (T)fmaf(D, x.y, a.scale * o.y);
            y[2] = (T)fmaf(D, x.z, a.scale * o.z); y[3] = (T)fmaf(D, x.w, a.scale * o.w);
        }
        if (a.export_grid > 0 && pos0 + t + 1 == next_export) {
            const int64_t idx = (int64_t)a.export_offsets[i] + exported;
            next_export += a.export_grid;
            ++exported;
            if (idx >= 0 && idx < a.export_capacity) {
                if (!a.export_slots) {
                    put(a.export_states + ((size_t)idx * a.H_v + h) * SE);
                } else {
                    const int sl = a.export_slots[idx];
                    if (sl >= 0 && sl < a.num_slots) put(a.pool + ((size_t)sl * a.H_v + h) * SE);
                }
            }
        }
    }
    const int fin = a.final_slot[i];
    if (fin >= 0 && fin < a.num_slots) put(a.pool + ((size_t)fin * a.H_v + h) * SE);
}

template <typename T, int DK, int DV>
hipError_t launch_typed(const SsmArgs& a, hipStream_t stream) {
    const unsigned blocks = (unsigned)a.num_seqs * (unsigned)a.H_v * (unsigned)(DV / kCols);
    hipLaunchKernelGGL((ssm_token_kernel<T, DK, DV>), dim3(blocks), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_dims(const SsmArgs& a, hipStream_t stream) {
    if (a.d_k == 128 && a.d_v == 128) return launch_typed<T, 128, 128>(a, stream);
    if (a.d_k == 128 && a.d_v == 64) return launch_typed<T, 128, 64>(a, stream);
    if (a.d_k == 64 && a.d_v == 128) return launch_typed<T, 64, 128>(a, stream);
    return launch_typed<T, 64, 64>(a, stream);
}

}  // namespace

size_t ssm_workspace_bytes(int, int, int, int, int, int64_t) { return 0; }

hipError_t launch_ssm_decode(const SsmArgs& a, hipStream_t stream) {
    return a.dtype == 1 ? launch_dims<__bf16>(a, stream) : launch_dims<float>(a, stream);
}

hipError_t launch_ssm_prefill(const SsmArgs& a, hipStream_t stream) { return launch_ssm_decode(a, stream); }

}  // namespace gdn
