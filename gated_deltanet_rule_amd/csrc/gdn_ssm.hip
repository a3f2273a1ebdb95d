// gdn_ssm.hip -- selective state space scan for gfx950: chunked prefill on the matrix
// cores, and one token of each of many cached rows.
//
//     d = softplus(dt + bias),  S <- e^(d A) S + d b x^T,  y = scale S^T c + D x
//
// Prefill.  Within a chunk of up to 64 tokens (rows i, j) with start state S (d_k x d_v)
//     G    = inclusive cumsum of d A inside the chunk
//     W_ij = (c_i . b_j) e^(G_i - G_j) d_j  for j <= i, else 0
//     Y    = scale (diag(e^G) C S + W X) + D X
//     S   <- e^(G_last) S + B^T diag(e^(G_last - G) d) X
// Only S goes from chunk to chunk.  Two workgroup shapes run the same arithmetic per
// element, so a sequence's bits do not depend on which one its call takes:
//   whole heads   one workgroup per (sequence, head), each of its waves 16 or 32 of the
//                 columns with its part of S in accumulators; W is formed once and
//                 shared in LDS, the last wave making the gates a chunk ahead.  For calls with
//                 enough chains to fill the card.  16 x 8192 tokens of 32 heads (128 x 128,
//                 bf16): 981 us, 3.6 TB/s (a large copy: 6.6 TB/s, 534 us for these bytes).
//                 No unit is full (vector ALU 48 % of the time, matrix cores 33 %, LDS 31 %):
//                 with two waves on a SIMD their phases' waits show, a quarter of a wave's
//                 time for memory and barriers, 41 % for the next instruction to issue.  Four
//                 waves on a SIMD (16 columns each) cost twice the operand reads and took
//                 1537 us.
//   strips        one workgroup per (sequence, head, 16 columns), for calls with few chains,
//                 bound by the length of the longest one.  W and the decays do not depend on
//                 S: a launch of their own forms them for all chunks side by side, once for
//                 all strips of a head, and leaves them in the workspace.  Then four waves
//                 form Y, each a quarter of the chunk's tokens, four advance S, each a quarter
//                 of its rows, and four stage; S passes between them in LDS, by chunk parity,
//                 so one barrier per chunk is enough.  One prompt of 8192 tokens: 146 us, of
//                 them 19 for W; a chunk takes 1.0 us against 3.6 us in whole heads.
//                 Bound by the 40 KB that each strip takes in per chunk, of which B and C are
//                 32: with 16 compute units reading the same lines at once about 20 B a cycle
//                 arrive at each.  Forming W in the strips took 188 us, B and C copied into
//                 operand order beside W 151 to 161, B through the LDS's direct loads 146,
//                 strips of 32 columns (half as many workgroups) 184.
// Operands.  16x16 tiles; lane l holds column l % 16 and rows 4 (l / 16) .. + 3 of a result
// (that is the "tile half" below), and the same elements are what an operand needs along k,
// so W and S turn from results into operands in place: products are formed as
// W^T = B C^T, Y^T = S^T C^T + X^T W^T, and a lane ends up with four neighbouring columns of
// Y.  B^T and X come out of LDS by transposing reads.
// Precision.  bf16: the decayed d x is split into three bf16 parts (8 bits each, exact), so
// the state keeps fp32 accuracy; W and the S that multiplies C are rounded once to bf16 (each
// by at most 2^-8 relative to its own product, on a y that is rounded to bf16 itself).  fp32: fp32
// matrix products, nothing rounded below fp32.  G is summed in 64 bits and kept as a pair, as
// its differences are what counts: behind one large step a single fp32 G is off by more than
// the small steps that follow it.
// A non-finite x must not reach earlier tokens through the zeros of W: a chunk that holds one
// takes it out of the product and sets its column to NaN from its token on.
//
// Decode.  A workgroup of 256 threads holds 64 columns of one head's state in registers;
// bound by the states' traffic: 64 rows of 32 heads move 270 MB in 45 us (6.0 TB/s) back to back
// on one set of states, 55 us (4.9 TB/s) on others each time.
#include <hip/hip_runtime.h>

#include <cstddef>

#include "gdn_device.h"
#include "gdn_internal.h"
#include "gdn_layer_device.h"
#include "gdn_layer_internal.h"

namespace gdn {
namespace {

using dev::kC;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
typedef __attribute__((address_space(3))) volatile u32x2 lds_vu32x2;
typedef __amdgpu_buffer_rsrc_t rsrc_t;

// ---------------------------------------------------------------- operands

// A value that is the same in every lane, in a scalar register for certain: loaded values are
// otherwise kept in vector registers, and buffers made from them are taken apart lane by lane.
__device__ __forceinline__ int uniform(int x) {
    x = __builtin_amdgcn_readfirstlane(x);
    asm("" : "+s"(x));
    return x;
}

// A chunk's rows of a token-major tensor as a raw buffer of `bytes`: loads past it give
// zeros and stores past it are dropped, which is how rows beyond a chunk's end enter.
__device__ __forceinline__ rsrc_t rows_rsrc(const void* base, int bytes) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(base);
    const uint64_t at = (uint64_t)(unsigned)uniform((int)(p >> 32)) << 32 | (unsigned)uniform((int)p);
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(at), (short)0, uniform(bytes), 0x00020000);
}
__device__ __forceinline__ u32x4 load16(rsrc_t r, int off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// What a lane holds of one 16-wide k tile (Half: four elements), and products over a pair
// of tiles.
template <typename T>
struct Ops;

template <>
struct Ops<__bf16> {
    typedef bf16x4 Half;
    static constexpr int kTerms = 3;
    static constexpr int kPad = 16;      // LDS rows: an odd multiple of 8 dwords, with the swizzle below conflict free

    static __device__ __forceinline__ f32x4 mma(Half a0, Half a1, Half b0, Half b1, f32x4 c) {
        const bf16x8 a = __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7);
        const bf16x8 b = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ Half round(f32x4 v) { return __builtin_convertvector(v, bf16x4); }
    static __device__ __forceinline__ f32x4 widen(Half h) {
        const u32x2 w = __builtin_bit_cast(u32x2, h);
        return f32x4{__builtin_bit_cast(float, w[0] << 16), __builtin_bit_cast(float, w[0] & 0xffff0000u),
                     __builtin_bit_cast(float, w[1] << 16), __builtin_bit_cast(float, w[1] & 0xffff0000u)};
    }
    static __device__ __forceinline__ Half load_half(rsrc_t r, int off) {
        return __builtin_bit_cast(Half, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
    }
    static __device__ __forceinline__ void store_half(Half h, rsrc_t r, int off) {
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, h), r, off, 0, 0);
    }
    // v = t[2] + t[1] + t[0] exactly: the leading 8 bits of what is left, three times
    static __device__ __forceinline__ void split(f32x4 v, Half (&t)[kTerms]) {
#pragma clang fp contract(off)
#pragma unroll
        for (int k = kTerms - 1; k >= 0; --k) {
            u32x4 w = __builtin_bit_cast(u32x4, v);
            t[k] = __builtin_bit_cast(Half, u32x2{__builtin_amdgcn_perm(w[1], w[0], 0x07060302u), __builtin_amdgcn_perm(w[3], w[2], 0x07060302u)});
            if (k > 0) {
                w = w & 0xffff0000u;
                v = v - __builtin_bit_cast(f32x4, w);
            }
        }
    }
    // Column swizzle of an LDS row: its 16-byte groups in pairs, swapped in every other eight rows.
    static __device__ __forceinline__ int column(int row, int c) { return c ^ (row & 8); }
    // Four elements of a row, as one 8-byte read: two of them paired into one instruction
    // cost four times as much on this card, and a volatile read is never paired.
    // t: a multiple of 16, g4: the lane's place in it (the swizzle moves only that).
    static __device__ __forceinline__ Half row_half(const __bf16* m, int pitch, int row, int t, int g4) {
        const u32x2 w = *(lds_vu32x2*)(m + (row * pitch + (g4 ^ (row & 8))) + t);
        return __builtin_bit_cast(Half, w);
    }
    // Rows r0 + 4 (l / 16) + e of column c0 + l % 16 (a transposing read: lane l points at
    // row r0 + l / 4, columns c0 + 4 (l % 4)).
    static __device__ __forceinline__ Half col_half(const __bf16* m, int pitch, int r0, int c0, int lane) {
        const int row = lane >> 2, at = row * pitch + ((4 * (lane & 3)) ^ (row & 8));
        return __builtin_bit_cast(Half, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(m + at + (r0 * pitch + c0))));
    }
    // larger of m's and w's exponents, two bf16 to a word; whether one says infinity or NaN
    static __device__ __forceinline__ unsigned exponents(u32x4 w, unsigned m) {
#pragma unroll
        for (int i = 0; i < 4; ++i) m = __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m), __builtin_bit_cast(u16x2, w[i] & 0x7f807f80u)));
        return m;
    }
    static __device__ __forceinline__ bool not_finite(unsigned m) { return (m >> 16) == 0x7f80u || (m & 0xffffu) == 0x7f80u; }
};

template <>
struct Ops<float> {
    typedef f32x4 Half;
    static constexpr int kTerms = 1;
    static constexpr int kPad = 4;

    static __device__ __forceinline__ f32x4 mma(Half a0, Half a1, Half b0, Half b1, f32x4 c) {
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a0[e], b0[e], c, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a1[e], b1[e], c, 0, 0, 0);
        return c;
    }
    static __device__ __forceinline__ Half round(f32x4 v) { return v; }
    static __device__ __forceinline__ f32x4 widen(Half h) { return h; }
    static __device__ __forceinline__ Half load_half(rsrc_t r, int off) { return __builtin_bit_cast(Half, load16(r, off)); }
    static __device__ __forceinline__ void store_half(Half h, rsrc_t r, int off) {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, h), r, off, 0, 0);
    }
    static __device__ __forceinline__ void split(f32x4 v, Half (&t)[kTerms]) { t[0] = v; }
    static __device__ __forceinline__ int column(int, int c) { return c; }
    static __device__ __forceinline__ Half row_half(const float* m, int pitch, int row, int t, int g4) {
        return *reinterpret_cast<const f32x4*>(m + (row * pitch + g4) + t);
    }
    static __device__ __forceinline__ Half col_half(const float* m, int pitch, int r0, int c0, int lane) {
        const float* p = m + (4 * (lane >> 4) * pitch + (lane & 15)) + (r0 * pitch + c0);
        return f32x4{p[0], p[pitch], p[2 * pitch], p[3 * pitch]};
    }
    static __device__ __forceinline__ unsigned exponents(u32x4 w, unsigned m) {
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, w[i] & 0x7f800000u);
        return m;
    }
    static __device__ __forceinline__ bool not_finite(unsigned m) { return m == 0x7f800000u; }
};

// ---------------------------------------------------------------- steps and decays of a chunk

struct Gates {
    float hi[kC], lo[kC];   // G log2 e = hi + lo
    float d[kC];            // step
    float w[kC];            // e^(G_last - G) d
    float eg[kC];           // e^G; rows past the chunk's end repeat the last one
};

// Inclusive sum over a wave in 64 bits, as dev::wave_inclusive_sum.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double dpp_term64(double x) {
    const u32x2 w = __builtin_bit_cast(u32x2, x);
    return __builtin_bit_cast(double, u32x2{(unsigned)__builtin_amdgcn_update_dpp(0, (int)w[0], CTRL, ROW_MASK, 0xf, true),
                                            (unsigned)__builtin_amdgcn_update_dpp(0, (int)w[1], CTRL, ROW_MASK, 0xf, true)});
}
__device__ __forceinline__ double wave_sum64(double x) {
    x += dpp_term64<0x111, 0xf>(x);
    x += dpp_term64<0x112, 0xf>(x);
    x += dpp_term64<0x114, 0xf>(x);
    x += dpp_term64<0x118, 0xf>(x);
    x += dpp_term64<0x142, 0xa>(x);
    x += dpp_term64<0x143, 0xc>(x);
    return x;
}

// Smallest exponent (to base 2) that a token's decay is taken to have: 2^-2^20 is 0 in any sum,
// and 64 of them leave G known to 2^-24 (six additions of 64 bits below 2^26), its pair to 2^-22.
constexpr double kLeast = -1048576.0;

// One wave, lane l for the chunk's token l of n.
__device__ __forceinline__ void make_gates(Gates& g, float dt, float bias, float A, int softplus, int n, int lane) {
    const float raw = dt + bias;
    float d = softplus ? dev::softplus(raw) : raw;
    if (lane >= n) d = 0.f;
    const double own = (double)d * (double)A * 1.4426950408889634074;
    const double G = wave_sum64(own < kLeast ? kLeast : own);      // (NaN stays)
    const u32x2 w = __builtin_bit_cast(u32x2, G);
    const double last = __builtin_bit_cast(double, u32x2{(unsigned)__builtin_amdgcn_readlane((int)w[0], kC - 1),
                                                         (unsigned)__builtin_amdgcn_readlane((int)w[1], kC - 1)});
    const float hi = (float)G;
    g.hi[lane] = hi;
    g.lo[lane] = (float)(G - (double)hi);
    g.d[lane] = d;
    g.w[lane] = d * __builtin_amdgcn_exp2f((float)(last - G));
    g.eg[lane] = __builtin_amdgcn_exp2f(hi);
}

// A tile of W^T from the scores c_i . b_j: lane l holds i = 16 it + l % 16, j = 16 jt + 4 (l / 16) + e.
template <typename T>
__device__ __forceinline__ typename Ops<T>::Half decayed(const Gates& g, f32x4 sc, int it, int jt, int lane) {
    const int i = 16 * it + (lane & 15), j0 = 16 * jt + 4 * (lane >> 4);
    const f32x4 hi = *reinterpret_cast<const f32x4*>(g.hi + j0), lo = *reinterpret_cast<const f32x4*>(g.lo + j0), d = *reinterpret_cast<const f32x4*>(g.d + j0);
    const float gi = g.hi[i], gl = g.lo[i];
    f32x4 diff;
#pragma unroll
    for (int e = 0; e < 4; ++e) diff[e] = (gi - hi[e]) + (gl - lo[e]);
    f32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = j0 + e <= i ? sc[e] * (__builtin_amdgcn_exp2f(diff[e]) * d[e]) : 0.f;
    return Ops<T>::round(w);
}

// The decayed steps times x of one tile half, in parts.  (Without contraction: it would split
// the unrounded product instead, where the compiler finds it.)
template <typename T>
__device__ __forceinline__ void weighted(f32x4 x, f32x4 w, typename Ops<T>::Half (&out)[Ops<T>::kTerms]) {
#pragma clang fp contract(off)
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = x[e] * w[e];
    Ops<T>::split(v, out);
}

// Takes non-finite values out of a column's tile halves (lane: rows 4 (l / 16) + e of tile t,
// one column); returns the first row that held one, kC without.
template <typename T>
__device__ __forceinline__ int take_out(typename Ops<T>::Half (&x)[kC / 16], int lane) {
    int first = kC;
#pragma unroll
    for (int t = kC / 16 - 1; t >= 0; --t) {
        f32x4 v = Ops<T>::widen(x[t]);
#pragma unroll
        for (int e = 3; e >= 0; --e)
            if (!(fabsf(v[e]) < __builtin_inff())) {
                v[e] = 0.f;
                first = 16 * t + 4 * (lane >> 4) + e;
            }
        x[t] = Ops<T>::round(v);
    }
    first = min(first, __shfl_xor(first, 16));
    return min(first, __shfl_xor(first, 32));
}

// Sequence and position bookkeeping of a workgroup.
struct Walk {
    int lo, len, skew, chunks;
    int64_t start;
    __device__ __forceinline__ Walk(const SsmArgs& a, int i) {
        dev::seq_range(a.cu_seqlens, i, a.total_tokens, lo, len);
        lo = uniform(lo);
        len = uniform(len);
        start = uniform(a.start_pos ? a.start_pos[i] : 0);
        skew = (int)(start & (kC - 1));
        chunks = dev::seq_chunks(len, skew);
    }
    // first row of chunk c and its tokens, 0 past the last chunk
    __device__ __forceinline__ void span(int c, int64_t& row, int& n) const {
        int b, e;
        dev::chunk_span(c, skew, len, b, e);
        n = c < chunks ? e - b : 0;
        row = lo + (n > 0 ? b : 0);
    }
    // local position after chunk c
    __device__ __forceinline__ int end_of(int c) const {
        int b, e;
        dev::chunk_span(c, skew, len, b, e);
        return e;
    }
};

// The states on the export grid, in order: chunks end at every one of its positions.
struct Exports {
    int64_t next, idx;      // local position of the next one (past any sequence without a grid), its place in the list
    __device__ __forceinline__ Exports(const SsmArgs& a, const Walk& walk, int i) {
        const bool any = a.export_grid > 0 && walk.chunks > 0;
        next = any ? (walk.start / a.export_grid + 1) * a.export_grid - walk.start : INT64_MAX;
        idx = any ? a.export_offsets[i] : 0;
    }
    // called after every chunk with its end: where the state goes, or NULL
    __device__ __forceinline__ float* take(const SsmArgs& a, int end, size_t state) {
        if (end != next) return nullptr;
        const int64_t at = idx++;
        next += a.export_grid;
        if (at < 0 || at >= a.export_capacity) return nullptr;
        if (!a.export_slots) return a.export_states + (size_t)at * state;
        const int sl = a.export_slots[at];
        return sl >= 0 && sl < a.num_slots ? a.pool + (size_t)sl * state : nullptr;
    }
};

// Workgroups go to the 8 XCDs round robin by index: renumber them so that each XCD gets a
// contiguous run, and the heads of a group, which read the same b and c, share one L2.
__device__ __forceinline__ unsigned xcd_run(unsigned wg) {
    return (gridDim.x & 7u) == 0 ? (wg & 7u) * (gridDim.x >> 3) + (wg >> 3) : wg;
}

// Rows [row, row + n) of a [tokens, heads, width] tensor at one head, from column c0 on.
template <typename T>
__device__ __forceinline__ rsrc_t head_rows(const void* base, int64_t row, int n, int heads, int h, int width, int c0, int columns) {
    const T* p = static_cast<const T*>(base) + ((size_t)row * heads + h) * width + c0;
    return rows_rsrc(p, n > 0 ? (int)(((size_t)(n - 1) * heads * width + columns) * sizeof(T)) : 0);
}

// dt of row + lane, 0 from n on.
__device__ __forceinline__ float load_step(const SsmArgs& a, int64_t row, int n, int h, int lane) {
    const rsrc_t r = rows_rsrc(a.dt + (size_t)row * a.H_v + h, n > 0 ? ((n - 1) * a.H_v + 1) * 4 : 0);
    return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, lane * a.H_v * 4, 0, 0));
}

// Where lane l's part of block s lies in operand order (a block: 32 columns of bf16, 16 of fp32).
// A wave stages a few rows of every block at once, and the blocks are a multiple of the LDS's
// width apart: moving each block's rows along spreads them over the banks.
template <typename T, int N>
__device__ __forceinline__ int swizzled(int s, int l) {
    constexpr int BLOCKS = N * (int)sizeof(T) / 64;
    return l ^ (16 / BLOCKS * s);
}

// A 64 x N block on its way from memory to LDS through the registers of TH threads.
template <typename T, int N, int TH>
struct Staged {
    static constexpr int V = 16 / sizeof(T), PER_ROW = N / V, VECS = kC * PER_ROW;
    static constexpr int K = (VECS + TH - 1) / TH;
    u32x4 v[K];

    __device__ __forceinline__ void load(rsrc_t r, int row_bytes, int tid) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int u = tid + k * TH;
            v[k] = load16(r, (u / PER_ROW) * row_bytes + (u % PER_ROW) * 16);      // past the block: past the buffer's end too
        }
    }
    // row-major, rows swizzled as Ops<T>::column says
    __device__ __forceinline__ void store(T* m, int pitch, int tid) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int u = tid + k * TH, row = u / PER_ROW;
            if (VECS % TH == 0 || u < VECS) *reinterpret_cast<u32x4*>(m + row * pitch + Ops<T>::column(row, (u % PER_ROW) * V)) = v[k];
        }
    }
    // as operands of rows: the two (bf16) or one (fp32) halves of a lane side by side, the lanes
    // of block s where swizzled() says
    __device__ __forceinline__ void store_operands(T* m, int tid) const {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int u = tid + k * TH, row = u / PER_ROW, c = (u % PER_ROW) * V;
            if constexpr (sizeof(T) == 2) {
                // pair block (row tile, c / 32), lane (row % 16, group), half (c / 16) % 2
                T* p = m + ((row >> 4) * (N / 32) + (c >> 5)) * 512 + swizzled<T, N>(c >> 5, (row & 15) + 16 * ((c & 15) >> 2)) * 8 + ((c >> 4) & 1) * 4;
                *reinterpret_cast<u32x2*>(p) = u32x2{v[k][0], v[k][1]};
                *reinterpret_cast<u32x2*>(p + 128) = u32x2{v[k][2], v[k][3]};
            } else {
                T* p = m + ((row >> 4) * (N / 16) + (c >> 4)) * 256 + swizzled<T, N>(c >> 4, (row & 15) + 16 * ((c & 15) >> 2)) * 4;
                *reinterpret_cast<u32x4*>(p) = v[k];
            }
        }
    }
    __device__ __forceinline__ bool any_not_finite(int tid) const {
        unsigned m = 0;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (VECS % TH == 0 || tid + k * TH < VECS) m = Ops<T>::exponents(v[k], m);
        return Ops<T>::not_finite(m);
    }
};

// A lane's two halves of pair s of an operand block stored by Staged::store_operands.
template <typename T, int N>
__device__ __forceinline__ void pair_of(const T* block, int s, int lane, typename Ops<T>::Half& h0, typename Ops<T>::Half& h1) {
    typedef typename Ops<T>::Half Half;
    if constexpr (sizeof(T) == 2) {
        const bf16x8 v = *reinterpret_cast<const bf16x8*>(block + s * 512 + swizzled<T, N>(s, lane) * 8);
        h0 = __builtin_shufflevector(v, v, 0, 1, 2, 3);
        h1 = __builtin_shufflevector(v, v, 4, 5, 6, 7);
    } else {
        h0 = *reinterpret_cast<const Half*>(block + 2 * s * 256 + swizzled<T, N>(2 * s, lane) * 4);
        h1 = *reinterpret_cast<const Half*>(block + (2 * s + 1) * 256 + swizzled<T, N>(2 * s + 1, lane) * 4);
    }
}

// The scores of one tile: sum over d_k of b_j (rows of LDS) and c_i (the lane's halves).
template <typename T, int DK, typename C>
__device__ __forceinline__ f32x4 score_tile(const T* b, int pitch, int jt, int lane, C c_pair) {
    typedef typename Ops<T>::Half Half;
    f32x4 sc = {0.f, 0.f, 0.f, 0.f};
    const int row = 16 * jt + (lane & 15), g4 = 4 * (lane >> 4);
#pragma unroll
    for (int s = 0; s < DK / 32; ++s) {
        Half c0, c1;
        c_pair(s, c0, c1);
        sc = Ops<T>::mma(Ops<T>::row_half(b, pitch, row, 32 * s, g4), Ops<T>::row_half(b, pitch, row, 32 * s + 16, g4), c0, c1, sc);
    }
    return sc;
}

// ---------------------------------------------------------------- whole heads

template <typename T, int DK, int DV>
struct HeadSmem {
    static constexpr int BP = DK + Ops<T>::kPad, XP = DV + Ops<T>::kPad;
    alignas(16) T b[kC * BP];
    T x[kC * XP];
    T c[kC * DK];            // operand order
    T w[10 * 256];           // lower tiles of W, a lane's half each
    Gates gate[2];           // by chunk parity
    int bad[2];              // chunk + 1 where its x holds a non-finite value
};

template <typename T, int DK, int DV, int CT>
__global__ __launch_bounds__(4 * DV / CT, sizeof(T) == 2 ? 2 : 1) void ssm_head_kernel(SsmArgs a) {
    typedef typename Ops<T>::Half Half;
    typedef HeadSmem<T, DK, DV> SM;
    constexpr int NW = DV / (16 * CT), TH = 64 * NW, NT = DK / 16, TT = kC / 16, TERMS = Ops<T>::kTerms;
    __shared__ SM sm;
    const int unit = (int)xcd_run(blockIdx.x), i = unit / a.H_v, h = unit - i * a.H_v;
    const int kh = h / (a.H_v / a.H_k);
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int li = lane & 15, g4 = 4 * (lane >> 4), col0 = 16 * CT * wv;
    const size_t state = (size_t)a.H_v * DK * DV;
    const int sin = a.init_slot[i], fin = a.final_slot[i];      // on their way beside the walk's loads
    const Walk walk(a, i);
    const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f, D = a.D ? a.D[h] : 0.f;
    const int krow = a.H_k * DK * (int)sizeof(T), vrow = a.H_v * DV * (int)sizeof(T);

    // S[nt][ct]: rows 16 nt + g4 + e, column col0 + 16 ct + li
    f32x4 S[NT][CT];
    // (a uniform address for each element beside one offset per lane: the alternative keeps
    // an address per element in registers)
    const unsigned mine = (unsigned)(g4 * DV + col0 + li);
    auto at = [](int nt, int ct, int e) { return (16 * nt + e) * DV + 16 * ct; };
    const bool have = sin >= 0 && sin < a.num_slots;
    {
        const float* src = have ? a.pool + (size_t)sin * state + (size_t)h * DK * DV : nullptr;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[nt][ct][e] = have ? (src + at(nt, ct, e))[mine] : 0.f;
        // waited for here, once: inside the loop the wait would also take in the prefetches
        __builtin_amdgcn_s_waitcnt(0x0F70);
    }
    auto put = [&](float* dst) {
        dst += (size_t)h * DK * DV;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int e = 0; e < 4; ++e) (dst + at(nt, ct, e))[mine] = S[nt][ct][e];
    };

    Staged<T, DK, TH> sb, sc;
    Staged<T, DV, TH> sx;
    float dt_next = 0.f;
    auto fetch = [&](int c) {
        int64_t row;
        int n;
        walk.span(c, row, n);
        sb.load(head_rows<T>(a.b, row, n, a.H_k, kh, DK, 0, DK), krow, tid);
        sc.load(head_rows<T>(a.c, row, n, a.H_k, kh, DK, 0, DK), krow, tid);
        sx.load(head_rows<T>(a.x, row, n, a.H_v, h, DV, 0, DV), vrow, tid);
    };
    auto fetch_dt = [&](int c) {
        int64_t row;
        int n;
        walk.span(c, row, n);
        dt_next = load_step(a, row, n, h, lane);
    };
    auto gates = [&](int c) {
        int64_t row;
        int n;
        walk.span(c, row, n);
        make_gates(sm.gate[c & 1], dt_next, bias, A, a.dt_softplus, n, lane);
    };
    if (tid < 2) sm.bad[tid] = 0;
    fetch(0);
    if (wv == NW - 1) {                       // the last wave makes the gates, a chunk ahead
        fetch_dt(0);
        gates(0);
        fetch_dt(1);
    }
    __syncthreads();

    Exports exports(a, walk, i);
    for (int c = 0; c < walk.chunks; ++c) {
        const Gates& g = sm.gate[c & 1];
        sb.store(sm.b, SM::BP, tid);
        sc.store_operands(sm.c, tid);
        sx.store(sm.x, SM::XP, tid);
        if (sx.any_not_finite(tid)) sm.bad[c & 1] = c + 1;
        dev::lds_barrier();
        fetch(c + 1);
        // lower tiles of W, in turn
        auto form = [&](int blk) {
            const int it = blk >= 6 ? 3 : blk >= 3 ? 2 : blk >= 1 ? 1 : 0, jt = blk - it * (it + 1) / 2;
            const T* cb = sm.c + it * 16 * DK;
            const f32x4 s = score_tile<T, DK>(sm.b, SM::BP, jt, lane, [&](int p, Half& h0, Half& h1) { pair_of<T, DK>(cb, p, lane, h0, h1); });
            *reinterpret_cast<Half*>(sm.w + blk * 256 + lane * 4) = decayed<T>(g, s, it, jt, lane);
        };
        // ten tiles: the last wave, which makes the gates, forms one of them or none
        static_assert(NW == 4 || NW == 8, "");
        if constexpr (NW == 4) {
            form(wv < 3 ? wv : 9);
            if (wv < 3) {
                form(wv + 3);
                form(wv + 6);
            }
        } else {
            if (wv < 7) form(wv);
            if (wv < 3) form(wv + 7);
        }
        __builtin_amdgcn_sched_barrier(0);
        // Y^T = S^T C^T, then the rows' e^G
        f32x4 y[TT][CT];
#pragma unroll
        for (int it = 0; it < TT; ++it)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) y[it][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < NT / 2; ++s) {
            Half s0[CT], s1[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                s0[ct] = Ops<T>::round(S[2 * s][ct]);
                s1[ct] = Ops<T>::round(S[2 * s + 1][ct]);
            }
#pragma unroll
            for (int it = 0; it < TT; ++it) {
                Half c0, c1;
                pair_of<T, DK>(sm.c + it * 16 * DK, s, lane, c0, c1);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) y[it][ct] = Ops<T>::mma(s0[ct], s1[ct], c0, c1, y[it][ct]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int it = 0; it < TT; ++it) {
            const float eg = g.eg[16 * it + li];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[it][ct][e] *= eg;
        }
        if (wv == NW - 1) {
            gates(c + 1);
            fetch_dt(c + 2);
        }
        dev::lds_barrier();
        // Y^T += X^T W^T
        Half x[CT][TT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int t = 0; t < TT; ++t) x[ct][t] = Ops<T>::col_half(sm.x, SM::XP, 16 * t, col0 + 16 * ct, lane);
        const bool poisoned = sm.bad[c & 1] == c + 1;
        if (poisoned)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const int bad = take_out<T>(x[ct], lane);
#pragma unroll
                for (int it = 0; it < TT; ++it)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (__shfl(bad, g4 + e) <= 16 * it + li) y[it][ct][e] = __builtin_nanf("");
            }
#pragma unroll
        for (int it = 0; it < TT; ++it)
#pragma unroll
            for (int s = 0; s <= it / 2; ++s) {
                const Half w0 = *reinterpret_cast<const Half*>(sm.w + (it * (it + 1) / 2 + 2 * s) * 256 + lane * 4);
                Half w1 = {};
                if (2 * s + 1 <= it) w1 = *reinterpret_cast<const Half*>(sm.w + (it * (it + 1) / 2 + 2 * s + 1) * 256 + lane * 4);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) y[it][ct] = Ops<T>::mma(x[ct][2 * s], x[ct][2 * s + 1], w0, w1, y[it][ct]);
            }
        int64_t row;
        int n;
        walk.span(c, row, n);
        const rsrc_t ry = head_rows<T>(a.y, row, n, a.H_v, h, DV, 0, DV);
#pragma unroll
        for (int it = 0; it < TT; ++it)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const int t = 16 * it + li, p = col0 + 16 * ct + g4;
                const f32x4 xt = Ops<T>::widen(Ops<T>::row_half(sm.x, SM::XP, t, col0 + 16 * ct, g4));
                f32x4 o;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = fmaf(a.scale, y[it][ct][e], D * xt[e]);
                Ops<T>::store_half(Ops<T>::round(o), ry, t * vrow + p * (int)sizeof(T));
            }
        __builtin_amdgcn_sched_barrier(0);
        // S <- e^(G_last) S + B^T (w X), x as it came
        if (poisoned)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int t = 0; t < TT; ++t) x[ct][t] = Ops<T>::col_half(sm.x, SM::XP, 16 * t, col0 + 16 * ct, lane);
        const float decay = g.eg[kC - 1];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[nt][ct][e] *= decay;
#pragma unroll
        for (int s = 0; s < TT / 2; ++s) {
            Half v0[CT][TERMS], v1[CT][TERMS];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const float* w = g.w + 32 * s + g4;
                weighted<T>(Ops<T>::widen(x[ct][2 * s]), *reinterpret_cast<const f32x4*>(w), v0[ct]);
                weighted<T>(Ops<T>::widen(x[ct][2 * s + 1]), *reinterpret_cast<const f32x4*>(w + 16), v1[ct]);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const Half b0 = Ops<T>::col_half(sm.b, SM::BP, 32 * s, 16 * nt, lane), b1 = Ops<T>::col_half(sm.b, SM::BP, 32 * s + 16, 16 * nt, lane);
#pragma unroll
                for (int k = 0; k < TERMS; ++k)
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) S[nt][ct] = Ops<T>::mma(b0, b1, v0[ct][k], v1[ct][k], S[nt][ct]);
                if (nt % 2 == 1) __builtin_amdgcn_sched_barrier(0);
            }
        }
        float* dst = exports.take(a, walk.end_of(c), state);
        if (dst) put(dst);
        dev::lds_barrier();
    }
    if (fin >= 0 && fin < a.num_slots) put(a.pool + (size_t)fin * state);
}

// ---------------------------------------------------------------- strips

// The strips of a head, and the heads of a group, need the same scores: a first launch forms W
// and the decays of every chunk, all chunks side by side, and leaves them in the workspace.
// Record of a chunk and head:
template <typename T>
struct Weights {
    T w[10 * 256];           // lower tiles of W, a lane's half each
    float d[kC];             // e^(G_last - G) d
    float eg[kC];            // e^G
};

// Records of a sequence start here: far enough from those of the one before, whatever its skew.
__device__ __forceinline__ int64_t first_record(int lo, int i) { return (lo >> 6) + 2 * (int64_t)i; }
int64_t record_count(int num_seqs, int64_t total_tokens) { return (total_tokens >> 6) + 2 * (int64_t)num_seqs; }

constexpr int kHeadBatch = 4;     // heads of one workgroup

template <typename T, int DK>
__global__ __launch_bounds__(256) void ssm_weights_kernel(SsmArgs a) {
    constexpr int BP = DK + Ops<T>::kPad;
    typedef typename Ops<T>::Half Half;
    __shared__ __attribute__((aligned(16))) T smb[kC * BP], smc[kC * DK];
    __shared__ Gates gate[kHeadBatch];
    const int R = a.H_v / a.H_k, batches = (R + kHeadBatch - 1) / kHeadBatch;
    const unsigned unit = xcd_run(blockIdx.x);      // a row's heads on one XCD: they lie on different L2 channels
    const int64_t record = unit / (unsigned)(a.H_k * batches);
    const int part = (int)(unit - record * (a.H_k * batches)), kh = part / batches, r0 = kHeadBatch * (part - kh * batches);
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    int i = 0;
    for (int hi = a.num_seqs - 1; i < hi;) {      // the last sequence whose records start at this one or before
        const int mid = (i + hi + 1) >> 1;
        int lo, len;
        dev::seq_range(a.cu_seqlens, mid, a.total_tokens, lo, len);
        if (first_record(lo, mid) <= record) i = mid;
        else hi = mid - 1;
    }
    i = __builtin_amdgcn_readfirstlane(i);
    const Walk walk(a, i);
    const int64_t c = record - first_record(walk.lo, i);
    if (c < 0 || c >= walk.chunks) return;
    int64_t row;
    int n;
    walk.span((int)c, row, n);
    Staged<T, DK, 256> sb, sc;
    const int krow = a.H_k * DK * (int)sizeof(T);
    sb.load(head_rows<T>(a.b, row, n, a.H_k, kh, DK, 0, DK), krow, tid);
    sc.load(head_rows<T>(a.c, row, n, a.H_k, kh, DK, 0, DK), krow, tid);
    Weights<T>* out = static_cast<Weights<T>*>(a.workspace) + record * a.H_v + kh * R + r0;
    if (r0 + wv < R) {
        const int h = kh * R + r0 + wv;
        const float dt = load_step(a, row, n, h, lane);
        make_gates(gate[wv], dt, a.dt_bias ? a.dt_bias[h] : 0.f, a.A[h], a.dt_softplus, n, lane);
        out[wv].d[lane] = gate[wv].w[lane];
        out[wv].eg[lane] = gate[wv].eg[lane];
    }
    sb.store(smb, BP, tid);
    sc.store_operands(smc, tid);
    __syncthreads();
    const int heads = R - r0 < kHeadBatch ? R - r0 : kHeadBatch;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        const int blk = wv + 4 * k;
        if (blk >= 10) break;
        const int it = blk >= 6 ? 3 : blk >= 3 ? 2 : blk >= 1 ? 1 : 0, jt = blk - it * (it + 1) / 2;
        const T* cb = smc + it * 16 * DK;
        const f32x4 s = score_tile<T, DK>(smb, BP, jt, lane, [&](int p, Half& h0, Half& h1) { pair_of<T, DK>(cb, p, lane, h0, h1); });
        for (int r = 0; r < heads; ++r) *reinterpret_cast<Half*>(out[r].w + blk * 256 + lane * 4) = decayed<T>(gate[r], s, it, jt, lane);
    }
}

constexpr int kStrip = 16;
constexpr int kStripThreads = 768;

template <typename T, int DK>
struct StripSmem {
    static constexpr int BP = DK + Ops<T>::kPad, XP = kStrip + (sizeof(T) == 4 ? 4 : 0);
    // C comes from LDS (operand order) where it fits beside the rest, else each wave loads its own
    static constexpr bool kStageC = sizeof(T) == 2;
    alignas(16) T b[2][kC * BP];                    // by chunk parity, as all of it
    T c[2][kStageC ? kC * DK : 8];
    T x[2][kC * XP];
    T v[2][Ops<T>::kTerms][kC * XP];      // e^(G_last - G) d x, in parts
    T s[2][DK * kStrip];                  // the state as operand, rounded to T
    int bad[2];
};

template <typename T, int DK, int DV>
__global__ __launch_bounds__(kStripThreads, 3) void ssm_strip_kernel(SsmArgs a) {
    typedef typename Ops<T>::Half Half;
    typedef StripSmem<T, DK> SM;
    constexpr int NT = DK / 64, TT = kC / 16, TERMS = Ops<T>::kTerms, NS = DV / kStrip, PAIRS = DK / 32;
    __shared__ SM sm;
    const unsigned wg = xcd_run(blockIdx.x);
    const int col0 = kStrip * (int)(wg % NS), unit = (int)(wg / NS), i = unit / a.H_v, h = unit - i * a.H_v;
    const int kh = h / (a.H_v / a.H_k);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wv = wave & 3;             // its quarter of the tokens, of the state's rows, of the staging
    const int li = lane & 15, g4 = 4 * (lane >> 4);
    const size_t state = (size_t)a.H_v * DK * DV;
    const int sin = a.init_slot[i], fin = a.final_slot[i];      // on their way beside the walk's loads
    const Walk walk(a, i);
    const int krow = a.H_k * DK * (int)sizeof(T), vrow = a.H_v * DV * (int)sizeof(T);

    // Three groups of four waves run loops of their own between the same barriers (so that the
    // waits of each count its own loads and stores alone): one forms Y of chunk c, one advances
    // S over it, one stages chunk c + 1.  Loads run two chunks ahead of their use, in two
    // register sets by chunk parity; an odd count of chunks is made even by one without tokens,
    // which changes nothing.
    const Weights<T>* rec = static_cast<const Weights<T>*>(a.workspace) + first_record(walk.lo, i) * a.H_v + h;
    // a record's buffer, empty past the last chunk
    auto record = [&](int c) { return rows_rsrc(rec + (size_t)(c < walk.chunks ? c : 0) * a.H_v, c < walk.chunks ? (int)sizeof(Weights<T>) : 0); };
    auto load_float = [](rsrc_t r, int off) { return __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0)); };
    constexpr int kDOff = offsetof(Weights<T>, d), kEgOff = offsetof(Weights<T>, eg), kHalf = 4 * (int)sizeof(T);
    if (tid < 2) sm.bad[tid] = 0;
    if (wave < 4) {
        const float D = a.D ? a.D[h] : 0.f;
        Half cf[2][2 * PAIRS], w[2][TT];
        float egs[2];
        auto fetch = [&](int c, int p) {
            int64_t row;
            int n;
            walk.span(c, row, n);
            const rsrc_t r = record(c);
#pragma unroll
            for (int jt = 0; jt < TT; ++jt)      // tiles past the diagonal: past the buffer, zeros
                w[p][jt] = Ops<T>::load_half(r, jt <= wv ? ((wv * (wv + 1) / 2 + jt) * 64 + lane) * kHalf : (int)sizeof(Weights<T>));
            egs[p] = load_float(r, kEgOff + 4 * (16 * wv + li));
            if constexpr (!SM::kStageC) {
                const rsrc_t rc = head_rows<T>(a.c, row, n, a.H_k, kh, DK, 0, DK);
#pragma unroll
                for (int t = 0; t < 2 * PAIRS; ++t) cf[p][t] = Ops<T>::load_half(rc, (16 * wv + li) * krow + (16 * t + g4) * (int)sizeof(T));
            }
        };
        auto body = [&](int c, int p) {
            Half x[TT];
            if constexpr (SM::kStageC)
#pragma unroll
                for (int s = 0; s < PAIRS; ++s) pair_of<T, DK>(sm.c[p] + wv * 16 * DK, s, lane, cf[p][2 * s], cf[p][2 * s + 1]);
#pragma unroll
            for (int t = 0; t < TT; ++t) x[t] = Ops<T>::col_half(sm.x[p], SM::XP, 16 * t, 0, lane);
            f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < PAIRS; ++s) {
                Half s0, s1;
                pair_of<T, DK>(sm.s[p], s, lane, s0, s1);
                y = Ops<T>::mma(s0, s1, cf[p][2 * s], cf[p][2 * s + 1], y);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] *= egs[p];
            const bool poisoned = sm.bad[p] == c + 1;
            const int bad = poisoned ? take_out<T>(x, lane) : kC;
#pragma unroll
            for (int s = 0; s < TT / 2; ++s)
                if (2 * s <= wv) y = Ops<T>::mma(x[2 * s], x[2 * s + 1], w[p][2 * s], w[p][2 * s + 1], y);
            fetch(c + 2, p);
            int64_t row;
            int n;
            walk.span(c, row, n);
            const rsrc_t ry = head_rows<T>(a.y, row, n, a.H_v, h, DV, col0, kStrip);
            const int t = 16 * wv + li;
            const f32x4 xt = Ops<T>::widen(Ops<T>::row_half(sm.x[p], SM::XP, t, 0, g4));
            f32x4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = fmaf(a.scale, y[e], D * xt[e]);
            if (poisoned)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (__shfl(bad, g4 + e) <= t) o[e] = __builtin_nanf("");
            Ops<T>::store_half(Ops<T>::round(o), ry, t * vrow + g4 * (int)sizeof(T));
            dev::lds_barrier();
        };
        fetch(0, 0);
        fetch(1, 1);
        __syncthreads();
        dev::lds_barrier();
        for (int c = 0; c < walk.chunks; c += 2) {
            body(c, 0);
            body(c + 1, 1);
        }
        return;
    }

    if (wave < 8) {
        f32x4 S[NT];                         // rows 16 (NT wv + nt) + g4 + e, column col0 + li
        const unsigned mine = (unsigned)((16 * NT * wv + g4) * DV + col0 + li);
        auto at = [](int nt, int e) { return (16 * nt + e) * DV; };
        auto put = [&](float* dst) {
            dst += (size_t)h * DK * DV;
    #pragma unroll
            for (int nt = 0; nt < NT; ++nt)
    #pragma unroll
                for (int e = 0; e < 4; ++e) (dst + at(nt, e))[mine] = S[nt][e];
        };
        auto share = [&](int parity) {       // a lane's half of tile t in operand order
    #pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int t = NT * wv + nt;
                T* p = sizeof(T) == 2 ? sm.s[parity] + (t >> 1) * 512 + swizzled<T, DK>(t >> 1, lane) * 8 + (t & 1) * 4
                                   : sm.s[parity] + t * 256 + swizzled<T, DK>(t, lane) * 4;
                *reinterpret_cast<Half*>(p) = Ops<T>::round(S[nt]);
            }
        };
        float decays[2];
        auto fetch = [&](int c, int p) { decays[p] = load_float(record(c), kEgOff + 4 * (kC - 1)); };
        Exports exports(a, walk, i);
        auto body = [&](int c, int p) {
            const float decay = c < walk.chunks ? decays[p] : 1.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[nt][e] *= decay;
#pragma unroll
            for (int s = 0; s < TT / 2; ++s) {
                Half v0[TERMS], v1[TERMS];
#pragma unroll
                for (int k = 0; k < TERMS; ++k) {
                    v0[k] = Ops<T>::col_half(sm.v[p][k], SM::XP, 32 * s, 0, lane);
                    v1[k] = Ops<T>::col_half(sm.v[p][k], SM::XP, 32 * s + 16, 0, lane);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int n0 = 16 * (NT * wv + nt);
                    const Half b0 = Ops<T>::col_half(sm.b[p], SM::BP, 32 * s, n0, lane), b1 = Ops<T>::col_half(sm.b[p], SM::BP, 32 * s + 16, n0, lane);
#pragma unroll
                    for (int k = 0; k < TERMS; ++k) S[nt] = Ops<T>::mma(b0, b1, v0[k], v1[k], S[nt]);
                }
            }
            share(p ^ 1);
            fetch(c + 2, p);
            float* dst = exports.take(a, walk.end_of(c), state);
            if (dst) put(dst);
            dev::lds_barrier();
        };
        const bool have = sin >= 0 && sin < a.num_slots;
        const float* src = have ? a.pool + (size_t)sin * state + (size_t)h * DK * DV : nullptr;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[nt][e] = have ? (src + at(nt, e))[mine] : 0.f;
        share(0);
        fetch(0, 0);
        fetch(1, 1);
        __syncthreads();
        dev::lds_barrier();
        for (int c = 0; c < walk.chunks; c += 2) {
            body(c, 0);
            body(c + 1, 1);
        }
        if (fin >= 0 && fin < a.num_slots) put(a.pool + (size_t)fin * state);
        return;
    }

    const int ltid = tid - 512, xr = ltid >> 2, xc = 4 * (ltid & 3);      // staging: a row and four columns of x
    Staged<T, DK, 256> sb[2], sc[2];
    Half sx[2];
    float ds[2];
    auto fetch = [&](int c, int p) {
        int64_t row;
        int n;
        walk.span(c, row, n);
        sb[p].load(head_rows<T>(a.b, row, n, a.H_k, kh, DK, 0, DK), krow, ltid);
        if constexpr (SM::kStageC) sc[p].load(head_rows<T>(a.c, row, n, a.H_k, kh, DK, 0, DK), krow, ltid);
        sx[p] = Ops<T>::load_half(head_rows<T>(a.x, row, n, a.H_v, h, DV, col0, kStrip), xr * vrow + xc * (int)sizeof(T));
        ds[p] = load_float(record(c), kDOff + 4 * xr);
    };
    auto stage = [&](int c, int p) {
        const int at = xr * SM::XP + Ops<T>::column(xr, xc);
        sb[p].store(sm.b[p], SM::BP, ltid);
        if constexpr (SM::kStageC) sc[p].store_operands(sm.c[p], ltid);
        *reinterpret_cast<Half*>(sm.x[p] + at) = sx[p];
        const f32x4 v = Ops<T>::widen(sx[p]);
        if (!(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))) < __builtin_inff()) ||
            !(v[0] == v[0] && v[1] == v[1] && v[2] == v[2] && v[3] == v[3])) sm.bad[p] = c + 1;
        Half part[TERMS];
        weighted<T>(v, f32x4{ds[p], ds[p], ds[p], ds[p]}, part);
#pragma unroll
        for (int k = 0; k < TERMS; ++k) *reinterpret_cast<Half*>(sm.v[p][k] + at) = part[k];
    };
    auto body = [&](int c, int p) {
        stage(c + 1, p ^ 1);
        fetch(c + 3, p ^ 1);
        dev::lds_barrier();
    };
    fetch(0, 0);
    fetch(1, 1);
    __syncthreads();
    stage(0, 0);
    fetch(2, 0);
    dev::lds_barrier();
    for (int c = 0; c < walk.chunks; c += 2) {
        body(c, 0);
        body(c + 1, 1);
    }
}

// ---------------------------------------------------------------- decode

constexpr int kThreads = 256;
constexpr int kCols = 64;

// 16 threads of one float4 cover a row's columns, the 16 row groups hold every sixteenth
// row; S^T c is summed over the row groups through LDS in a fixed order.
template <typename T, int DK, int DV>
__global__ __launch_bounds__(kThreads) void ssm_decode_kernel(SsmArgs a) {
    constexpr int TPR = kCols / 4, RG = kThreads / TPR, R = DK / RG, NCW = DV / kCols;
    const int unit = blockIdx.x / NCW;
    const int col0 = kCols * (blockIdx.x - unit * NCW);
    const int i = unit / a.H_v, h = unit - i * a.H_v;
    const int kh = h / (a.H_v / a.H_k);
    const int tid = threadIdx.x, c4 = tid % TPR, rg = tid / TPR;
    const size_t SE = (size_t)DK * DV;

    const int sin = a.init_slot[i], fin = a.final_slot[i];
    T* y = static_cast<T*>(a.y) + ((size_t)i * a.H_v + h) * DV + col0 + 4 * c4;
    if (sin < 0 || sin >= a.num_slots) {         // padding row
        if (rg == 0) y[0] = y[1] = y[2] = y[3] = (T)0.f;
        return;
    }
    const float* src = a.pool + ((size_t)sin * a.H_v + h) * SE + col0 + 4 * c4;
    f32x4 s[R];
#pragma unroll
    for (int m = 0; m < R; ++m) s[m] = *reinterpret_cast<const f32x4*>(src + (size_t)(rg + RG * m) * DV);
    __shared__ float bc[2][DK];
    __shared__ f32x4 red[RG][TPR];
    if (tid < DK) bc[0][tid] = (float)static_cast<const T*>(a.b)[((size_t)i * a.H_k + kh) * DK + tid];
    else if (tid < 2 * DK) bc[1][tid - DK] = (float)static_cast<const T*>(a.c)[((size_t)i * a.H_k + kh) * DK + tid - DK];
    const T* xp = static_cast<const T*>(a.x) + ((size_t)i * a.H_v + h) * DV + col0 + 4 * c4;
    const f32x4 x = {(float)xp[0], (float)xp[1], (float)xp[2], (float)xp[3]};
    const float raw = a.dt[(size_t)i * a.H_v + h] + (a.dt_bias ? a.dt_bias[h] : 0.f), D = a.D ? a.D[h] : 0.f;
    const float d = a.dt_softplus ? dev::softplus(raw) : raw;
    const float decay = expf(d * a.A[h]);
    __syncthreads();
    f32x4 p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int m = 0; m < R; ++m) {
        const float db = d * bc[0][rg + RG * m], cr = bc[1][rg + RG * m];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[m][e] = fmaf(db, x[e], decay * s[m][e]);
            p[e] = fmaf(s[m][e], cr, p[e]);
        }
    }
    red[rg][c4] = p;
    if (fin >= 0 && fin < a.num_slots) {
        float* dst = a.pool + ((size_t)fin * a.H_v + h) * SE + col0 + 4 * c4;
#pragma unroll
        for (int m = 0; m < R; ++m) *reinterpret_cast<f32x4*>(dst + (size_t)(rg + RG * m) * DV) = s[m];
    }
    dev::lds_barrier();
    if (rg == 0) {
        f32x4 o = red[0][c4];
#pragma unroll
        for (int r = 1; r < RG; ++r)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] += red[r][c4][e];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = (T)fmaf(D, x[e], a.scale * o[e]);
    }
}

// ---------------------------------------------------------------- launches

template <typename T, int DK, int DV>
hipError_t decode_typed(const SsmArgs& a, hipStream_t stream) {
    const int64_t blocks = (int64_t)a.num_seqs * a.H_v * (DV / kCols);
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((ssm_decode_kernel<T, DK, DV>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

// Strips for calls with few chains.  A compute unit takes one strip at a time, in about 1.1 us a
// chunk (bf16, 128 x 128) behind two launches; a whole head takes 3.6 us a chunk, however many
// compute units have one.  So strips pay for few rounds of them over the card, the more rounds
// the longer the sequences have to be.  Measured (us, heads / strips, equal sequences), bf16 of
// 128 x 128: one round of 128 tokens 13 / 16, of 320 24 / 17, of 4096 237 / 76; two of 320 25 / 26,
// of 512 36 / 30; three of 832 54 / 57, of 4096 246 / 222, and of 64 x 64 156 / 197.  fp32: one round
// of 128 30 / 17; two of 128 32 / 25, of 64 x 64 17 / 19; three of 512 106 / 72 and 52 / 50; four of
// 1600 323 / 263 and 154 / 185.  What counts is the longest sequence, which the host
// does not know: lengths spread evenly from nothing up make it 2 n / (n + 1) times the mean of n.
// Where they are not, the rule is off: every sequence counts for a full set of strips, so a prompt
// of 8192 tokens (bf16, 32 heads of 128 x 128) that takes 150 us alone takes 265 beside one single
// token, as its strips share half of the XCDs, and 465 in whole heads beside two.  Nor does it look
// at d_k and d_v: where 128 x 128 and 64 x 64 above point to different launches, both take heads.
constexpr int kMaxRounds = 3;
bool in_strips(int H_v, int d_v, int dtype, int num_seqs, int64_t total_tokens) {
    const int64_t strips = (int64_t)num_seqs * H_v * (d_v / kStrip), cus = device_cus(), rounds = (strips + cus - 1) / cus;
    if (strips == 0 || rounds > (dtype == 1 ? 2 : kMaxRounds)) return false;
    const int64_t chunks = dtype == 1 ? 3 * rounds + 1 : (int64_t)1 << rounds;
    return 2 * total_tokens >= chunks * kC * (num_seqs + 1);
}

template <typename T, int DK, int DV>
hipError_t prefill_typed(const SsmArgs& a, hipStream_t stream) {
    const int64_t chains = (int64_t)a.num_seqs * a.H_v;
    if (!in_strips(a.H_v, DV, a.dtype, a.num_seqs, a.total_tokens)) {
        if (!grid_fits(chains, 4 * DV)) return hipErrorInvalidConfiguration;
        // Eight waves of 16 columns where a compute unit has one head at a time anyway (bf16 with no
        // more heads than compute units; fp32, by its LDS), four of 32 where two heads share one
        // (us, eight / four, 1024 tokens of 32 heads of 128 x 128: bf16 8 sequences 80 / 87, 12
        // sequences 138 / 118; fp32 217 / 252 and 419 / 485).
        if constexpr (DV == 128 && sizeof(T) == 2)
            if (chains > device_cus()) {
                hipLaunchKernelGGL((ssm_head_kernel<T, DK, DV, 2>), dim3((unsigned)chains), dim3(256), 0, stream, a);
                return hipGetLastError();
            }
        hipLaunchKernelGGL((ssm_head_kernel<T, DK, DV, 1>), dim3((unsigned)chains), dim3(4 * DV), 0, stream, a);
        return hipGetLastError();
    }
    const int R = a.H_v / a.H_k;
    const int64_t blocks = record_count(a.num_seqs, a.total_tokens) * a.H_k * ((R + kHeadBatch - 1) / kHeadBatch);
    if (!grid_fits(blocks, 256)) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((ssm_weights_kernel<T, DK>), dim3((unsigned)blocks), dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((ssm_strip_kernel<T, DK, DV>), dim3((unsigned)(chains * (DV / kStrip))), dim3(kStripThreads), 0, stream, a);
    return hipGetLastError();
}

template <typename T>
hipError_t prefill_dims(const SsmArgs& a, hipStream_t stream) {
    if (a.d_k == 128 && a.d_v == 128) return prefill_typed<T, 128, 128>(a, stream);
    if (a.d_k == 128 && a.d_v == 64) return prefill_typed<T, 128, 64>(a, stream);
    if (a.d_k == 64 && a.d_v == 128) return prefill_typed<T, 64, 128>(a, stream);
    return prefill_typed<T, 64, 64>(a, stream);
}

template <typename T>
hipError_t decode_dims(const SsmArgs& a, hipStream_t stream) {
    if (a.d_k == 128 && a.d_v == 128) return decode_typed<T, 128, 128>(a, stream);
    if (a.d_k == 128 && a.d_v == 64) return decode_typed<T, 128, 64>(a, stream);
    if (a.d_k == 64 && a.d_v == 128) return decode_typed<T, 64, 128>(a, stream);
    return decode_typed<T, 64, 64>(a, stream);
}

}  // namespace

size_t ssm_workspace_bytes(int H_v, int, int d_v, int dtype, int num_seqs, int64_t total_tokens) {
    if (!in_strips(H_v, d_v, dtype, num_seqs, total_tokens)) return 0;
    return (size_t)record_count(num_seqs, total_tokens) * (size_t)H_v * (dtype == 1 ? sizeof(Weights<__bf16>) : sizeof(Weights<float>));
}

// Strips that pay for some tokens pay for more, and records grow with both counts: the most is
// at all the tokens and the largest count of sequences that still takes strips.
size_t ssm_workspace_bound(int H_v, int d_v, int dtype, int max_seqs, int64_t max_tokens) {
    const int64_t cus = device_cus(), per_seq = (int64_t)H_v * (d_v / kStrip);
    int64_t n = kMaxRounds * cus / per_seq;
    for (n = n < max_seqs ? n : max_seqs; n > 0; --n)
        if (in_strips(H_v, d_v, dtype, (int)n, max_tokens)) return ssm_workspace_bytes(H_v, 0, d_v, dtype, (int)n, max_tokens);
    return 0;
}

hipError_t launch_ssm_decode(const SsmArgs& a, hipStream_t stream) {
    return a.dtype == 1 ? decode_dims<__bf16>(a, stream) : decode_dims<float>(a, stream);
}

hipError_t launch_ssm_prefill(const SsmArgs& a, hipStream_t stream) {
    return a.dtype == 1 ? prefill_dims<__bf16>(a, stream) : prefill_dims<float>(a, stream);
}

}  // namespace gdn
