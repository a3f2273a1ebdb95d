// gdn_plan.hip -- the plan of one step on the GPU (gfx950): packed offsets, state slots,
// export lists and per-token maps from request lengths and block tables.
//
// Everything is a prefix sum over the prefill requests (of lengths and of grid points
// crossed) followed by table lookups; what bounds it is latency, then 16 bytes written per
// token.  Every workgroup sums the requests by itself into LDS, which costs less than a
// second launch would, and resolves its share of rows, exports and tokens by binary search
// there; the first one also writes the per-request outputs.  Beyond kShared requests the
// offsets no longer fit beside each other in LDS: one workgroup writes them, and a second
// launch searches them in memory.  512 requests with 64 prompts of up to 4096 tokens: 7.0 us;
// 64 decode rows: 2.2 us (10.7 us a call from Python, which is the host's marshalling).
#include <hip/hip_runtime.h>

#include "gdn_internal.h"
#include "gdn_layer_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kItems = 4;         // requests of one thread in one piece of the sum
constexpr int kShared = 4096;     // prefill requests whose offsets and starts fit in 48 KiB
constexpr unsigned kCap = 0x7fffffffu;

// min(a + b, 2^31 - 1) for a, b below 2^31: associative, so sums may be taken in any order.
__device__ __forceinline__ unsigned add_sat(unsigned a, unsigned b) { return min(a + b, kCap); }

// Positions are sums of two int32 values: they fit in 32 unsigned bits.
__device__ __forceinline__ int state_slot(const PlanArgs& a, int r, unsigned p) {
    const unsigned blk = p / (unsigned)a.state_block;
    if (p == 0) return -1;
    if (p != blk * (unsigned)a.state_block) return a.run_slot[r];
    return blk <= (unsigned)a.state_table_width ? a.state_table[(size_t)r * a.state_table_width + (blk - 1)] : -1;
}

__device__ __forceinline__ int64_t kv_slot(const PlanArgs& a, int r, unsigned p) {
    const unsigned blk = p / (unsigned)a.kv_block;
    if (blk >= (unsigned)a.kv_table_width) return -1;
    const int64_t e = a.kv_table[(size_t)r * a.kv_table_width + blk];
    return e < 0 ? -1 : e * a.kv_block + (int64_t)(p - blk * (unsigned)a.kv_block);
}

__device__ __forceinline__ unsigned positive(int32_t x) { return x < 0 ? 0u : (unsigned)x; }

// Exclusive saturating sum over the workgroup; total: the sum of all.
__device__ __forceinline__ unsigned block_scan(unsigned x, unsigned* sums, unsigned& total) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    unsigned s = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const unsigned y = (unsigned)__shfl_up((int)s, d);
        if (lane >= d) s = add_sat(s, y);
    }
    __syncthreads();
    if (lane == 63) sums[wv] = s;
    __syncthreads();
    unsigned before = (unsigned)__shfl_up((int)s, 1);
    if (lane == 0) before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        if (w < wv) before = add_sat(before, sums[w]);
        total = add_sat(total, sums[w]);
    }
    return before;
}

// The prefills' offsets and starts, into LDS (cu not NULL) and, where `write` is set, into
// the outputs.
__device__ __forceinline__ void sum_requests(const PlanArgs& a, bool write, int32_t* cu, int32_t* eo, int32_t* st) {
    __shared__ unsigned sums[2][kThreads / 64];
    const int B = a.num_decode_rows, N = a.num_requests - B;
    unsigned base_n = 0, base_e = 0;
    if (threadIdx.x == 0) {
        if (cu) cu[0] = eo[0] = 0;
        if (write) a.cu_seqlens[0] = a.export_offsets[0] = 0;
    }
    for (int i0 = 0; i0 < N; i0 += kThreads * kItems) {
        const int first = i0 + (int)threadIdx.x * kItems;
        unsigned s[kItems], n[kItems], e[kItems], sn = 0, se = 0;
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int i = first + k;
            s[k] = i < N ? positive(a.computed[B + i]) : 0u;
            n[k] = i < N ? positive(a.new_tokens[B + i]) : 0u;
            e[k] = (s[k] + n[k]) / (unsigned)a.state_block - s[k] / (unsigned)a.state_block;
            sn = add_sat(sn, n[k]);
            se = add_sat(se, e[k]);
        }
        unsigned tn, te;
        unsigned an = add_sat(base_n, block_scan(sn, sums[0], tn)), ae = add_sat(base_e, block_scan(se, sums[1], te));
        base_n = add_sat(base_n, tn);
        base_e = add_sat(base_e, te);
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int i = first + k;
            an = add_sat(an, n[k]);
            ae = add_sat(ae, e[k]);
            if (i >= N) continue;
            if (cu) {
                cu[i + 1] = (int32_t)an;
                eo[i + 1] = (int32_t)ae;
                st[i] = (int32_t)s[k];
            }
            if (write) {
                a.cu_seqlens[i + 1] = (int32_t)an;
                a.export_offsets[i + 1] = (int32_t)ae;
                a.start_pos[i] = (int32_t)s[k];
                a.init_slot[i] = state_slot(a, B + i, s[k]);
                a.final_slot[i] = state_slot(a, B + i, s[k] + n[k]);
            }
        }
    }
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

// Decode rows, exports and tokens, from the prefills' offsets and starts.
__device__ __forceinline__ void fill_rows(const PlanArgs& a, const int32_t* cu, const int32_t* eo, const int32_t* st) {
    const int B = a.num_decode_rows, N = a.num_requests - B;
    const int64_t first = (int64_t)blockIdx.x * kThreads + threadIdx.x, step = (int64_t)gridDim.x * kThreads;
    for (int64_t t = first; t < B; t += step) {
        const unsigned s = positive(a.computed[t]);
        const bool live = a.new_tokens[t] > 0;
        const int in = state_slot(a, (int)t, s), out = state_slot(a, (int)t, s + 1);
        a.slot_in[t] = live ? in : -1;
        a.slot_out[t] = live ? out : -1;
    }
    const int64_t tokens = cu[N], exports = eo[N];
    for (int64_t t = first; t < a.token_capacity; t += step) {
        int r = -1;
        unsigned p = 0;
        if (t < B) {
            if (a.new_tokens[t] > 0) {
                r = (int)t;
                p = positive(a.computed[t]);
            }
        } else if (t - B < tokens) {
            const int i = owner_of(cu, N, t - B);
            r = B + i;
            p = (unsigned)st[i] + (unsigned)(t - B - cu[i]);
        }
        if (a.token_request) a.token_request[t] = r;
        if (a.token_position) a.token_position[t] = r < 0 ? -1 : (int32_t)min(p, kCap);
        if (a.token_kv_slot) a.token_kv_slot[t] = r < 0 ? -1 : kv_slot(a, r, p);
    }
    for (int64_t x = first; x < a.export_capacity; x += step) {
        int slot = -1;
        if (x < exports) {
            const int i = owner_of(eo, N, x);
            const unsigned s = (unsigned)st[i], end = s + positive(a.new_tokens[B + i]);
            const unsigned p = (s / (unsigned)a.state_block + 1u + (unsigned)(x - eo[i])) * (unsigned)a.state_block;
            if (p != end) slot = state_slot(a, B + i, p);
        }
        a.export_slots[x] = slot;
    }
}

__global__ __launch_bounds__(kThreads) void plan_kernel(PlanArgs a) {
    extern __shared__ int32_t lds[];
    const int N = a.num_requests - a.num_decode_rows;
    int32_t *cu = lds, *eo = lds + N + 1, *st = lds + 2 * (N + 1);
    sum_requests(a, blockIdx.x == 0, cu, eo, st);
    __syncthreads();
    fill_rows(a, cu, eo, st);
}

__global__ __launch_bounds__(kThreads) void plan_requests_kernel(PlanArgs a) { sum_requests(a, true, nullptr, nullptr, nullptr); }

__global__ __launch_bounds__(kThreads) void plan_rows_kernel(PlanArgs a) { fill_rows(a, a.cu_seqlens, a.export_offsets, a.start_pos); }

}  // namespace

hipError_t launch_plan(const PlanArgs& a, hipStream_t stream) {
    const int N = a.num_requests - a.num_decode_rows;
    int64_t work = a.token_capacity > a.export_capacity ? a.token_capacity : a.export_capacity;
    if (work < a.num_decode_rows) work = a.num_decode_rows;
    int64_t blocks = (work + kThreads - 1) / kThreads;
    // as many workgroups as the card holds at once: more would only repeat the sum
    if (blocks > 4 * device_cus()) blocks = 4 * device_cus();
    if (blocks < 1) blocks = 1;
    if (N <= kShared) {
        hipLaunchKernelGGL(plan_kernel, dim3((unsigned)blocks), dim3(kThreads), (size_t)(3 * N + 2) * 4, stream, a);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(plan_requests_kernel, dim3(1), dim3(kThreads), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(plan_rows_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace gdn
