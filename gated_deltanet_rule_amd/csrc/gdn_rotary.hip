// gdn_rotary.hip -- rotary positions for gfx950.
//
//     (a, b) <- factor (a cos t - b sin t, b cos t + a sin t),   t = p f_i
//
// Memory-bound: every value crosses HBM once each way.  A workgroup takes a token: its threads
// first form the cosines and sines, one frequency each, into LDS, where all heads
// share them; then they turn the heads' pairs, V pairs to a thread as two 16-byte vectors.
// 131072 tokens of 32 + 8 heads of 128 dims in bf16: 467 us, 5.7 TB/s of 6.6 for a large copy; 64 tokens: 3.4 us, of
// which the copy's share is 0.2 and the rest a launch.  4099 tokens of 16 + 2 heads of 256 dims in fp32: 35 us, where an even copy of as
// much takes 25; 65536 tokens 462 us, 5.2 TB/s.
// Where rows or parts are not whole vectors V is 1, and a token of few heads leaves most of its workgroup idle: 65536 tokens of 8 + 2 heads
// of 80 dims, all of the head 65 us (3.2 TB/s), a quarter of it 125 (1.7); of 1 + 1 heads of 64 dims 44 us (0.8).
#include <hip/hip_runtime.h>

#include "gdn_attention_internal.h"
#include "gdn_layer_device.h"
#include "gdn_layer_internal.h"
#include "gdn_pages.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;

struct RotaryKernelArgs {
    RotaryArgs a;
    Divisor units_of_head;
    int turned;      // of a head's units, those that turn; the rest copy (none in place)
};

// V elements of T as floats, one 16-byte vector or a single element
template <typename T, int V>
__device__ __forceinline__ void load(const T* p, float (&v)[V]) {
    if constexpr (V == 1) v[0] = (float)p[0];
    else dev::load_vec(p, v);
}
template <typename T, int V>
__device__ __forceinline__ void store(T* p, const float (&v)[V]) {
    if constexpr (V == 1) p[0] = (T)v[0];
    else dev::store_vec(p, v);
}

// cos and sin of p f, times factor.  p f has up to 55 bits and 1 / (2 pi) more: products are taken as a double and the rest that
// it leaves off, so that the part of a turn is exact to 2^-52 however many turns there are.  fp32 values take cosine and sine of it in
// 64 bits, rounded once; for bf16 ones fp32 does, 2^-15 of a half step off.
template <typename T>
__device__ __forceinline__ float2 turn(int p, float f, float factor) {
#pragma clang fp contract(off)             // (a product taken into a sum would be another number than the one whose rest is taken)
    constexpr double kTurn = 0x1.45f306dc9c883p-3, kRest = -0x1.6b01ec5417056p-57;        // 1 / (2 pi) and what is left of it
    const double x = (double)p * (double)f, rest = fma((double)p, (double)f, -x), turns = x * kTurn;
    const double part = (turns - rint(turns)) + (fma(x, kTurn, -turns) + fma(rest, kTurn, x * kRest));
    if constexpr (sizeof(T) == 4) {
        double s, c;
        sincospi(2. * part, &s, &c);
        return {(float)(c * factor), (float)(s * factor)};
    } else {
        float s, c;
        sincospif(2.f * (float)part, &s, &c);
        return {c * factor, s * factor};
    }
}

// A head's units: pairs V j .. V j + V - 1 for j < turned, then 2 V elements each that only copy.
template <typename T, int V, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryKernelArgs k) {
    extern __shared__ float2 turns[];
    const gdn_rotary_shape& s = k.a.shape;
    const int half = s.rotary_dim / 2, heads = s.num_q_heads + s.num_k_heads;
    const int64_t token = blockIdx.x;
    const int position = k.a.positions[token];
    for (int i = threadIdx.x; i < half; i += kThreads) turns[i] = turn<T>(position, k.a.inv_freq[i], s.factor);
    __syncthreads();
    if (position < 0) return;
    const int units = heads * (int)k.units_of_head.d;
    for (int i = threadIdx.x; i < units; i += kThreads) {
        const int head = (int)dev::divide(i, k.units_of_head), unit = i - head * (int)k.units_of_head.d;
        const int which = head >= s.num_q_heads, h = which ? head - s.num_q_heads : head;
        const T* in = static_cast<const T*>(k.a.in[which]) + token * k.a.in_stride[which] + (int64_t)h * s.head_dim;
        T* out = static_cast<T*>(k.a.out[which]) + token * k.a.out_stride[which] + (int64_t)h * s.head_dim;
        float a[V], b[V];
        if (unit >= k.turned) {
            const int e = s.rotary_dim + (unit - k.turned) * 2 * V;
            load<T, V>(in + e, a);
            const bool both = e + 2 * V <= s.head_dim;
            if (both) load<T, V>(in + e + V, b);
            store<T, V>(out + e, a);
            if (both) store<T, V>(out + e + V, b);
            continue;
        }
        const int ea = INTERLEAVED ? 2 * V * unit : V * unit, eb = INTERLEAVED ? ea + V : ea + half;
        const float2* cs = turns + V * unit;
        load<T, V>(in + ea, a);
        load<T, V>(in + eb, b);
        float x[V], y[V];
        if constexpr (INTERLEAVED) {
            // the 2 V elements as pairs in order
            float v[2 * V], w[2 * V];
#pragma unroll
            for (int j = 0; j < V; ++j) { v[j] = a[j]; v[V + j] = b[j]; }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 c = cs[j];
                w[2 * j] = v[2 * j] * c.x - v[2 * j + 1] * c.y;
                w[2 * j + 1] = v[2 * j + 1] * c.x + v[2 * j] * c.y;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) { x[j] = w[j]; y[j] = w[V + j]; }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 c = cs[j];
                x[j] = a[j] * c.x - b[j] * c.y;
                y[j] = b[j] * c.x + a[j] * c.y;
            }
        }
        store<T, V>(out + ea, x);
        store<T, V>(out + eb, y);
    }
}

template <typename T, int V>
hipError_t launch(const RotaryArgs& a, hipStream_t stream) {
    const gdn_rotary_shape& s = a.shape;
    const bool in_place = (s.num_q_heads == 0 || a.in[0] == a.out[0]) && (s.num_k_heads == 0 || a.in[1] == a.out[1]);
    RotaryKernelArgs k = {a, Divisor(), s.rotary_dim / (2 * V)};
    const int copied = in_place ? 0 : (s.head_dim - s.rotary_dim + 2 * V - 1) / (2 * V);
    k.units_of_head = Divisor(k.turned + copied);
    if (!grid_fits(a.num_tokens, kThreads)) return hipErrorInvalidConfiguration;
    const size_t lds = (size_t)(s.rotary_dim / 2) * sizeof(float2);
    if (s.interleaved) rotary_kernel<T, V, true><<<(unsigned)a.num_tokens, kThreads, lds, stream>>>(k);
    else rotary_kernel<T, V, false><<<(unsigned)a.num_tokens, kThreads, lds, stream>>>(k);
    return hipGetLastError();
}

template <typename T>
hipError_t launch(const RotaryArgs& a, hipStream_t stream) {
    constexpr int V = dev::kVec<T>;
    const gdn_rotary_shape& s = a.shape;
    bool wide = s.rotary_dim % (2 * V) == 0 && s.head_dim % V == 0;
    for (int i = 0; i < 2; ++i) {
        if ((i ? s.num_k_heads : s.num_q_heads) == 0) continue;
        wide = wide && a.in_stride[i] % V == 0 && a.out_stride[i] % V == 0 && (uintptr_t)a.in[i] % 16 == 0 && (uintptr_t)a.out[i] % 16 == 0;
    }
    if (!wide) return launch<T, 1>(a, stream);
    return launch<T, V>(a, stream);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, hipStream_t stream) {
    return a.shape.dtype == GDN_BF16 ? launch<__bf16>(a, stream) : launch<float>(a, stream);
}

}  // namespace gdn
