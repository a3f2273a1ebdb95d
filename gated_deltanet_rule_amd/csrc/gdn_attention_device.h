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

// The sum of eight weights that were rounded to bf16.  The instruction rounds to nearest but cuts its smallest terms off (0.1 of
// a half step too little in the mean, beside terms 2^20 apart), so sums over many keys add such sums in fp32.
__device__ __forceinline__ float sum8(bf16x8_t w, float sum) {
    const bf16x2_t one = {(__bf16)1.f, (__bf16)1.f};
#pragma unroll
    for (int i = 0; i < 8; i += 2) sum = __builtin_amdgcn_fdot2_f32_bf16(bf16x2_t{w[i], w[i + 1]}, one, sum, false);
    return sum;
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

constexpr float kLog2e = 1.4426950408889634f;

struct AttentionKernelArgs {
    AttentionArgs a;
    Divisor block, group, rows;    // kv_block, query heads of a head, tokens_per_row
    int spans;                     // decode: of the workspace, the most that a row may have
    int row_tiles;                 // decode: workgroups for the rows of a head
    float* part;                   // [tokens][H_q][spans][D]
    float2* stats;                 // [tokens][H_q][spans]: running maximum, sum
};

// Where a workgroup's rows come from.
struct Unit {
    int seq, h;             // sequence (row of the call), cache head
    int64_t first;          // its first token in q and o
    int tokens, past;       // new tokens, cached tokens (clipped to what the table holds)
    int row0, rows;         // first row of the tile, rows of the sequence's head
    int lo, hi;             // keys [lo, hi)
    int span, spans;        // which of the row's spans; spans of the row
};

// gdn_attention_wide.hip: bf16 prompts, and decode rows (without the join of their spans).
hipError_t launch_attention_wide(const AttentionKernelArgs& k, hipStream_t stream);

// A unit is its workgroup's: its fields go into scalar registers, which the compiler does not see where they come out of memory,
// so that the branches and addresses made of them are scalar too.
__device__ __forceinline__ void make_uniform(Unit& u) {
    const auto one = [](int& x) { x = __builtin_amdgcn_readfirstlane(x); };
    one(u.seq); one(u.h); one(u.tokens); one(u.past); one(u.row0); one(u.rows); one(u.lo); one(u.hi); one(u.span); one(u.spans);
    const unsigned lo = __builtin_amdgcn_readfirstlane((unsigned)u.first), hi = __builtin_amdgcn_readfirstlane((unsigned)((uint64_t)u.first >> 32));
    u.first = (int64_t)((uint64_t)hi << 32 | lo);
}

// Keys of a decode row, all of its tokens' among them, as far as its table goes; < 0 for a padding row.
__device__ __forceinline__ int row_keys(const AttentionArgs& a, int past) {
    if (past < 0) return -1;
    const int64_t keys = (int64_t)past + a.tokens_per_row;
    return (int)(keys < a.capacity ? keys : a.capacity);
}

// Outputs of `count` rows of a tile set to one value, by `threads` threads.
template <typename T, int D>
__device__ __forceinline__ void fill_rows(const AttentionKernelArgs& k, const Unit& u, int count, int threads, float value) {
    const int G = (int)k.group.d;
    for (int i = threadIdx.x; i < count * (D / 4); i += threads) {
        const int r = u.row0 + i / (D / 4), e = i % (D / 4) * 4;
        if (r >= u.rows) break;
        const int t = (int)dev::divide(r, k.group);
        T* o = static_cast<T*>(k.a.o) + ((u.first + t) * k.a.H_q + u.h * G + (r - t * G)) * D + e;
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = (T)value;
    }
}

// Decode: the span of keys and the tile of `per` rows of workgroup blockIdx.x.  False where there is nothing to
// attend to: a padding row's outputs are zeros then, those of a row with more keys than max_keys NaN.
template <typename T, int D>
__device__ __forceinline__ bool decode_unit(const AttentionKernelArgs& k, int per, int threads, Unit& u) {
    // The row tiles of one span of keys stand 8 apart: on the same XCD, whose L2 then holds its keys.  Its heads stand on
    // different ones, which keeps them evenly loaded: all on one was 1-3 % faster without row tiles, but 124 us for 107 with trees
    // of 16 rows, whose longest spans then meet on one XCD.
    const unsigned id = blockIdx.x, tile = id / 8 % (unsigned)k.row_tiles, at = id / (8 * (unsigned)k.row_tiles) * 8 + id % 8;
    const unsigned H = (unsigned)k.a.cache.num_heads, by_head = at / H, spans = (unsigned)k.spans;
    u.h = (int)(at - by_head * H);
    u.seq = (int)(by_head / spans);
    u.span = (int)(by_head - (unsigned)u.seq * spans);
    if (u.seq >= k.a.num_seqs) return false;
    u.past = k.a.past[u.seq];
    u.tokens = k.a.tokens_per_row;
    u.first = (int64_t)u.seq * u.tokens;
    u.rows = u.tokens * (int)k.group.d;
    u.row0 = (int)tile * per;
    const int keys = row_keys(k.a, u.past);
    if (keys <= 0 || keys > k.a.max_keys) {
        if (u.span == 0) fill_rows<T, D>(k, u, per, threads, keys > 0 ? NAN : 0.f);
        return false;
    }
    const int span = span_keys(u.rows, keys);
    u.spans = span_count(keys, span);
    if (u.span >= u.spans) return false;
    u.past = u.past < k.a.capacity ? u.past : k.a.capacity;
    u.lo = u.span * span;
    u.hi = keys - u.lo < span ? keys : u.lo + span;
    make_uniform(u);
    return true;
}

// Packed prompts: tile number `tile` of `per` rows.  The first tile of sequence i is number cu[i] G / per + i, so
// that a tile's sequence is found by bisection and no two share a tile; false for the tiles in between.
__device__ __forceinline__ bool prompt_unit(const AttentionKernelArgs& k, int per, int tile, int h, Unit& u) {
    const int G = (int)k.group.d;
    const int64_t total = k.a.total_tokens;
    const auto token = [&](int i) {
        const int64_t c = k.a.cu_seqlens[i];
        return c < 0 ? 0 : (c > total ? total : c);
    };
    // 64 sequences at a time, a lane each: the last whose first tile is not behind this one
    const int lane = threadIdx.x & 63;
    int lo = 0, step = 1;
    while ((int64_t)step * 64 < k.a.num_seqs) step *= 64;
    for (; step > 0; step /= 64) {
        const int64_t i = lo + (int64_t)lane * step;
        const bool reached = i < k.a.num_seqs && token((int)i) * G / per + i <= tile;
        lo += step * (63 - __builtin_clzll(__ballot(reached) | 1));
    }
    u.seq = lo;
    u.h = h;
    const int64_t b = token(lo), e = token(lo + 1), row0 = (tile - b * G / per - lo) * per;
    if (row0 < 0 || row0 >= (e - b) * G) return false;
    u.first = b;
    u.tokens = (int)(e - b);
    u.rows = u.tokens * G;
    u.row0 = (int)row0;
    const int past = k.a.past ? k.a.past[lo] : 0;
    u.past = past < 0 ? 0 : (past < k.a.capacity ? past : k.a.capacity);
    const int last = (u.row0 + per < u.rows ? u.row0 + per : u.rows) - 1;
    const int64_t keys = (int64_t)u.past + (int)dev::divide(last, k.group) + 1;
    u.lo = 0;
    u.hi = (int)(keys < k.a.capacity ? keys : k.a.capacity);
    u.span = 0;
    u.spans = 1;
    make_uniform(u);
    return true;
}

// Keys that row r of a unit (a query head of a token) sees without a tree: a prompt may end past the last position.
__device__ __forceinline__ int causal_keys(const AttentionKernelArgs& k, const Unit& u, int r) {
    const int64_t n = (int64_t)u.past + (int)dev::divide(r, k.group) + 1;
    return n < 0x7fffffff ? (int)n : 0x7fffffff;
}

// The keys that row r sees.
__device__ __forceinline__ dev::Sees row_sees(const AttentionKernelArgs& k, const Unit& u, int r) {
    if (!k.a.tree_mask) return {causal_keys(k, u, r), 0, 0};
    const int t = (int)dev::divide(r, k.group);
    const uint64_t all = u.tokens >= 64 ? ~0ull : (1ull << u.tokens) - 1;
    return {u.past, u.past, (uint64_t)k.a.tree_mask[u.first + t] & all};
}

}  // namespace gdn
