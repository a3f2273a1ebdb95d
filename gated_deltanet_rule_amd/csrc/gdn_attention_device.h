// gdn_attention_device.h -- device helpers of the attention kernels: matrix operands of either
// dtype, cache formats widened into them, a token's visible keys, exchanges between lane groups.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gdn_attention_internal.h"
#include "gdn_layer_device.h"
#include "gdn_pages.h"

namespace gdn {
namespace dev {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

// Eight values along the contraction, one lane's share of a matrix operand.  With bf16 one
// instruction contracts all lanes' eight; with fp32 eight instructions take one value of each
// lane in turn.  Both sum over the same products, so operands are laid out alike.
template <typename T>
struct Frag;
template <>
struct Frag<__bf16> {
    using type = bf16x8_t;
};
template <>
struct Frag<float> {
    using type = f32x8_t;
};
template <typename T>
using frag_t = typename Frag<T>::type;

// acc[i] += sum_k a[row 4 (lane / 16) + i][k] b[k][lane % 16]
__device__ __forceinline__ f32x4_t mma16(bf16x8_t a, bf16x8_t b, f32x4_t acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mma16(f32x8_t a, f32x8_t b, f32x4_t acc) {
#pragma unroll
    for (int j = 0; j < 8; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], acc, 0, 0, 0);
    return acc;
}

// Four 8-bit codes as values of T (exact in bf16: at most 8 significant bits).
template <typename T, int FORMAT>
__device__ __forceinline__ void codes4(unsigned w, T (&v)[4]) {
    if constexpr (FORMAT == GDN_CACHE_INT8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (T)(float)(int8_t)(w >> (8 * i));
    } else if constexpr (sizeof(T) == 2) {
        const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false), hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true);
        v[0] = lo[0]; v[1] = lo[1]; v[2] = hi[0]; v[3] = hi[1];
    } else {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
        v[0] = lo[0]; v[1] = lo[1]; v[2] = hi[0]; v[3] = hi[1];
    }
}

// Eight codes (the two words from w0) as an operand.
template <typename T, int FORMAT>
__device__ __forceinline__ frag_t<T> codes8(unsigned w0, unsigned w1) {
    T a[4], b[4];
    codes4<T, FORMAT>(w0, a);
    codes4<T, FORMAT>(w1, b);
    frag_t<T> f;
#pragma unroll
    for (int i = 0; i < 4; ++i) { f[i] = a[i]; f[4 + i] = b[i]; }
    return f;
}

// A value and that of the lane 32 (16) further, as two values that both lanes hold alike: the
// exchange swaps the halves (the odd and even rows) of two copies.  Its results are read as whole
// words first: a bit_cast of a vector's element takes the first one here, whichever is named.
__device__ __forceinline__ void pair32(float x, float& a, float& b) {
    const unsigned u = __builtin_bit_cast(unsigned, x);
    const auto h = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const unsigned lo = h[0], hi = h[1];
    a = __builtin_bit_cast(float, lo);
    b = __builtin_bit_cast(float, hi);
}
__device__ __forceinline__ void pair16(float x, float& a, float& b) {
    const unsigned u = __builtin_bit_cast(unsigned, x);
    const auto h = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const unsigned lo = h[0], hi = h[1];
    a = __builtin_bit_cast(float, lo);
    b = __builtin_bit_cast(float, hi);
}

// The larger (the sum) of a value over the four lanes l, l ^ 16, l ^ 32, l ^ 48, the same bits
// in all of them.  fmaxf leaves a NaN out; it comes back through the weights.
__device__ __forceinline__ float across_max(float x) {
    float a, b;
    pair32(x, a, b);
    pair16(fmaxf(a, b), a, b);
    return fmaxf(a, b);
}
__device__ __forceinline__ float across_sum(float x) {
    float a, b;
    pair32(x, a, b);
    pair16(a + b, a, b);
    return a + b;
}

// The keys that a token sees: positions below `all`, and `first` + j for the bits j of `mask`.
struct Sees {
    int all, first;
    uint64_t mask;
    // positions p .. p + 63 as bits
    __device__ __forceinline__ uint64_t from(int p) const {
        const int n = all - p, b = first - p;
        uint64_t m = n >= 64 ? ~0ull : (n <= 0 ? 0ull : (1ull << n) - 1);
        if (b > -64 && b < 64) m |= b >= 0 ? mask << b : mask >> -b;
        return m;
    }
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

}  // namespace dev
}  // namespace gdn
