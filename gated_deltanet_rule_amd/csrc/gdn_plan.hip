// gdn_plan.hip -- the plan of one step on the GPU (gfx950): packed offsets, state slots,
// export lists and per-token maps from request lengths and block tables.
//
// Everything is a prefix sum over the requests (of prefill lengths and of grid points
// crossed) followed by table lookups.  One workgroup scans the requests in pieces of its
// size, writes the per-request outputs, and then resolves exports and tokens by binary
// search in the offsets it has just written.
#include <hip/hip_runtime.h>

#include "gdn_layer_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 1024;

__device__ __forceinline__ int state_slot(const PlanArgs& a, int r, int64_t p) {
    if (p <= 0) return -1;
    const int64_t blk = p / a.state_block;
    if (p != blk * a.state_block) return a.run_slot[r];
    return blk <= a.state_table_width ? a.state_table[(size_t)r * a.state_table_width + (blk - 1)] : -1;
}

__device__ __forceinline__ int64_t kv_slot(const PlanArgs& a, int r, int64_t p) {
    const int64_t blk = p / a.kv_block;
    if (blk >= a.kv_table_width) return -1;
    const int64_t e = a.kv_table[(size_t)r * a.kv_table_width + blk];
    return e < 0 ? -1 : e * a.kv_block + (p - blk * a.kv_block);
}

__device__ __forceinline__ int saturate(int64_t x) { return x > 0x7fffffff ? 0x7fffffff : (int)x; }

// Inclusive sum over the workgroup of one 64-bit value per thread.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* sums) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t y = __shfl_up((long long)x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 63) sums[wv] = x;
    __syncthreads();
    for (int w = 0; w < wv; ++w) x += sums[w];
    return x;
}

// Largest i in [0, n] with off[i] <= t, off[0] = 0.
__device__ __forceinline__ int owner_of(const int32_t* off, int n, int64_t t) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__global__ __launch_bounds__(kThreads) void plan_kernel(PlanArgs a) {
    __shared__ int64_t sums[kThreads / 64];
    __shared__ int64_t total[2];
    const int tid = threadIdx.x;
    const int B = a.num_decode_rows, N = a.num_requests - B;

    for (int b = tid; b < B; b += kThreads) {
        const int64_t s = a.computed[b] < 0 ? 0 : a.computed[b];
        const bool live = a.new_tokens[b] > 0;
        a.slot_in[b] = live ? state_slot(a, b, s) : -1;
        a.slot_out[b] = live ? state_slot(a, b, s + 1) : -1;
    }
    if (tid == 0) total[0] = total[1] = a.cu_seqlens[0] = a.export_offsets[0] = 0;
    __syncthreads();
    for (int i0 = 0; i0 < N; i0 += kThreads) {
        const int i = i0 + tid, r = B + i;
        int64_t s = 0, n = 0, e = 0;
        if (i < N) {
            s = a.computed[r] < 0 ? 0 : a.computed[r];
            n = a.new_tokens[r] < 0 ? 0 : a.new_tokens[r];
            e = (s + n) / a.state_block - s / a.state_block;
        }
        const int64_t base_n = total[0], base_e = total[1];
        const int64_t sum_n = base_n + block_scan(n, sums);
        const int64_t sum_e = base_e + block_scan(e, sums);
        if (i < N) {
            a.cu_seqlens[i + 1] = saturate(sum_n);
            a.export_offsets[i + 1] = saturate(sum_e);
            a.start_pos[i] = (int)s;
            a.init_slot[i] = state_slot(a, r, s);
            a.final_slot[i] = state_slot(a, r, s + n);
        }
        __syncthreads();
        if (tid == kThreads - 1) {
            total[0] = sum_n;
            total[1] = sum_e;
        }
        __syncthreads();
    }
    const int64_t tokens = N > 0 ? a.cu_seqlens[N] : 0, exports = N > 0 ? a.export_offsets[N] : 0;
    for (int64_t x = tid; x < a.export_capacity; x += kThreads) {
        int slot = -1;
        if (x < exports) {
            const int i = owner_of(a.export_offsets, N, x);
            const int64_t s = a.start_pos[i];
            const int64_t end = s + (a.new_tokens[B + i] < 0 ? 0 : a.new_tokens[B + i]);
            const int64_t p = (s / a.state_block + 1 + x - a.export_offsets[i]) * a.state_block;
            if (p != end) slot = state_slot(a, B + i, p);
        }
        a.export_slots[x] = slot;
    }
    for (int64_t t = tid; t < a.token_capacity; t += kThreads) {
        int r = -1;
        int64_t p = -1;
        if (t < B) {
            if (a.new_tokens[t] > 0) {
                r = (int)t;
                p = a.computed[t] < 0 ? 0 : a.computed[t];
            }
        } else if (t - B < tokens) {
            const int i = owner_of(a.cu_seqlens, N, t - B);
            r = B + i;
            p = a.start_pos[i] + (t - B - a.cu_seqlens[i]);
        }
        if (a.token_request) a.token_request[t] = r;
        if (a.token_position) a.token_position[t] = saturate(p);
        if (a.token_kv_slot) a.token_kv_slot[t] = r < 0 ? -1 : kv_slot(a, r, p);
    }
}

}  // namespace

hipError_t launch_plan(const PlanArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdn
