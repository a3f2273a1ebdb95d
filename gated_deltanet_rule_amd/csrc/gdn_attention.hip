// gdn_attention.hip -- attention over a paged cache for gfx950: decode rows of one or more
// tokens, and fp32 prompts.
//
//     o = sum_p w_p v_p / sum_p w_p,   w_p = 2^(c q.k_p - m),   c = scale log2 e
//
// The query heads of a cache head, and the tokens of a row, are the rows of one product, 16 NT
// of them to a workgroup.  Its four waves take every fourth tile of 32 keys, each with a
// running maximum and sum of its own, and meet in LDS at the end.  The products are formed
// transposed, S^T = K Q^T and O^T = V^T P^T, 16 x 16 tiles with a query row to each lane of a
// group of 16: a lane then holds four keys' weights of its row for each tile of 16 keys, which is
// the operand that the second product takes if V's rows are taken in that order, so weights
// never move between lanes and a row's factors are the lane's own.  K goes from memory into
// operands directly (a lane's 16 bytes of a key are eight steps of the contraction; queries are
// laid out alike); V goes through the wave's own LDS, which hands it out transposed.
//
// A long context is cut into spans that workgroups take side by side, joined by a second
// launch.  The spans follow from the row's own number of keys and the shape, so a row's bits do
// not depend on what shares its call.
#include <hip/hip_runtime.h>

#include "gdn_attention_device.h"
#include "gdn_layer_internal.h"

namespace gdn {
namespace {

using dev::f32x4_t;
using dev::u32x4_t;

constexpr int kThreads = 256, kWaves = 4, kTile = 32;

// V's rows in LDS: bf16 rows are D values, their 16-byte chunks exchanged by key so that neither the
// stores (16 keys, one chunk) nor the transposing loads (4 keys, two chunks to a group of 16 lanes)
// meet in a bank; fp32 rows are padded by four.
template <typename T, int D>
struct VTile {
    static constexpr int kRow = sizeof(T) == 2 ? D * 2 : (D + 4) * 4;      // bytes
    static constexpr int kBytes = kTile * kRow;
    __device__ static __forceinline__ int chunk(int key, int c) {
        if constexpr (sizeof(T) == 4) return key * kRow + c * 16;
        else if constexpr (D >= 128) return key * kRow + ((c ^ ((2 * key) & 15)) * 16);
        else return key * kRow + ((c ^ (key & 6)) * 16);
    }
    // V^T for dims 16 t .. 16 t + 15: lane % 16 is the dim, the eight keys 4 (lane / 16) + 0..3 of both halves of the tile
    __device__ static __forceinline__ dev::frag_t<T> load(const char* lds, int t, int lane) {
        if constexpr (sizeof(T) == 2) {
            const int key = 4 * (lane / 16) + lane % 16 / 4, c = 2 * t + (lane & 3) / 2;
            typedef __attribute__((address_space(3))) dev::s16x4_t* lds_ptr;
            const auto a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(lds + chunk(key, c) + (lane & 1) * 8));
            const auto b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(lds + chunk(key + 16, c) + (lane & 1) * 8));
            const dev::bf16x4_t x = __builtin_bit_cast(dev::bf16x4_t, a), y = __builtin_bit_cast(dev::bf16x4_t, b);
            return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            dev::f32x8_t f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int key = 16 * (j / 4) + 4 * (lane / 16) + j % 4;
                f[j] = *reinterpret_cast<const float*>(lds + key * kRow + (16 * t + lane % 16) * 4);
            }
            return f;
        }
    }
    __device__ static __forceinline__ float at(const char* lds, int key, int dim) {
        return (float)*reinterpret_cast<const T*>(lds + chunk(key, dim * (int)sizeof(T) / 16) + dim * (int)sizeof(T) % 16);
    }
};

// What a lane holds of one key for one tile: its 16-byte pieces of the stored row and the operands they make.
// Piece i of lane l is bytes 64 i + 16 (l / 16) of the head's row.
template <typename T, int FORMAT, int D>
struct Stored {
    static constexpr bool kCodes = FORMAT != GDN_CACHE_PLAIN;
    static constexpr int kElem = kCodes ? 1 : (int)sizeof(T);
    static constexpr int kPieces = D * kElem / 64;
    static constexpr int kFrags = D / 32;
    // operand f of the contraction over dims: eight dims for each lane
    __device__ static __forceinline__ int dim(int f, int lane) {
        if constexpr (kCodes) return f / 2 * 64 + lane / 16 * 16 + f % 2 * 8;
        else if constexpr (sizeof(T) == 2) return f * 32 + lane / 16 * 8;
        else return f * 32 + lane / 16 * 4;         // two pieces, 16 dims apart
    }
    __device__ static __forceinline__ dev::frag_t<T> frag(const u32x4_t (&p)[kPieces], int f) {
        if constexpr (kCodes) return dev::codes8<T, FORMAT>(p[f / 2][f % 2 * 2], p[f / 2][f % 2 * 2 + 1]);
        else if constexpr (sizeof(T) == 2) return __builtin_bit_cast(dev::bf16x8_t, p[f]);
        else {
            const f32x4_t x = __builtin_bit_cast(f32x4_t, p[2 * f]), y = __builtin_bit_cast(f32x4_t, p[2 * f + 1]);
            return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
    // the query's operand f: the same dims
    __device__ static __forceinline__ dev::frag_t<T> query(const T* q, int f, int lane) {
        if constexpr (sizeof(T) == 2) return *reinterpret_cast<const dev::bf16x8_t*>(q + dim(f, lane));
        else {
            const int second = kCodes ? 4 : 16;
            const f32x4_t x = *reinterpret_cast<const f32x4_t*>(q + dim(f, lane)), y = *reinterpret_cast<const f32x4_t*>(q + dim(f, lane) + second);
            return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    }
};

template <typename T, int FORMAT, int D>
__device__ __forceinline__ void load_pieces(const void* cache, int64_t head, int lane, u32x4_t (&p)[Stored<T, FORMAT, D>::kPieces]) {
    using S = Stored<T, FORMAT, D>;
    const char* at = static_cast<const char*>(cache) + head * (D * S::kElem) + lane / 16 * 16;
#pragma unroll
    for (int i = 0; i < S::kPieces; ++i) p[i] = *reinterpret_cast<const u32x4_t*>(at + 64 * i);
}

// A piece's values into V's tile in LDS; with `clean`, what is not finite as zero.  Returns whether all were finite.
template <typename T, int FORMAT, int D>
__device__ __forceinline__ bool stage(char* lds, int key, int lane, const u32x4_t (&p)[Stored<T, FORMAT, D>::kPieces], bool present, bool clean) {
    using S = Stored<T, FORMAT, D>;
    bool fine = true;
#pragma unroll
    for (int i = 0; i < S::kPieces; ++i) {
        if constexpr (S::kCodes) {
            T v[16];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                T c[4];
                dev::codes4<T, FORMAT>(p[i][w], c);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * w + j] = c[j];
            }
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const bool ok = dev::finite((float)v[j]);
                fine &= ok || !present;
                if (!present || (clean && !ok)) v[j] = (T)0.f;
            }
            constexpr int N = 16 / (int)sizeof(T);
            const int first = (64 * i + lane / 16 * 16) * (int)sizeof(T) / 16;
#pragma unroll
            for (int c = 0; c < (int)sizeof(T); ++c) {
                u32x4_t w;
                __builtin_memcpy(&w, v + c * N, 16);
                *reinterpret_cast<u32x4_t*>(lds + VTile<T, D>::chunk(key, first + c)) = w;
            }
        } else {
            constexpr int N = 16 / (int)sizeof(T);
            T v[N];
            __builtin_memcpy(v, &p[i], 16);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const bool ok = dev::finite((float)v[j]);
                fine &= ok || !present;
                if (!present || (clean && !ok)) v[j] = (T)0.f;
            }
            u32x4_t w;
            __builtin_memcpy(&w, v, 16);
            *reinterpret_cast<u32x4_t*>(lds + VTile<T, D>::chunk(key, 4 * i + lane / 16)) = w;
        }
    }
    return fine;
}

// LDS of a workgroup: V's tiles of the four waves, which the waves' sums share at the end; then the
// waves' scales and statistics.
template <typename T, int D>
struct Lds {
    static constexpr int kSum = 16 * (D + 4) * 4;              // 16 rows of a wave's sums
    static constexpr int kWave = VTile<T, D>::kBytes > kSum ? VTile<T, D>::kBytes : kSum;
    static constexpr int kScales = kWaves * 2 * kTile * 4;
    static constexpr int kTotal = kWaves * kWave + kScales + kWaves * 16 * 8;
};

template <typename T, int FORMAT, int D, int NT>
__device__ __forceinline__ void attend(const AttentionKernelArgs& k, const Unit& u, char* lds) {
    using S = Stored<T, FORMAT, D>;
    constexpr int kDims = D / 16;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane % 16, quad = lane / 16, G = (int)k.group.d;
    char* const vt = lds + wave * Lds<T, D>::kWave;
    float* const scales = reinterpret_cast<float*>(lds + kWaves * Lds<T, D>::kWave) + wave * 2 * kTile;
    float2* const stats = reinterpret_cast<float2*>(lds + kWaves * Lds<T, D>::kWave + Lds<T, D>::kScales);
    const dev::Pages pages = {k.a.table + (int64_t)u.seq * k.a.table_width, k.a.table_width, k.block, k.a.cache.num_rows};
    const int H = k.a.cache.num_heads;
    const float c = k.a.scale * kLog2e;

    dev::frag_t<T> q[NT][S::kFrags];
    dev::Sees sees[NT];
    int some = 0x7fffffff;                     // every row sees the keys below this
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = u.row0 + 16 * n + col, t = (int)dev::divide(r, k.group);
        const bool live = r < u.rows;
        sees[n] = {0, 0, 0};
        if (live) {
            const T* p = static_cast<const T*>(k.a.q) + (u.first + t) * k.a.q_stride + (int64_t)(u.h * G + (r - t * G)) * D;
#pragma unroll
            for (int f = 0; f < S::kFrags; ++f) q[n][f] = S::query(p, f, lane);
            sees[n] = row_sees(k, u, r);
        } else {
#pragma unroll
            for (int f = 0; f < S::kFrags; ++f) q[n][f] = dev::frag_t<T>{};
        }
    }
    some = k.a.tree_mask ? u.past : u.past + (int)dev::divide(u.row0, k.group) + 1;

    f32x4_t o[NT][kDims] = {};
    float m[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) { m[n] = -INFINITY; l[n] = 0.f; }

    for (int p0 = u.lo + wave * kTile; p0 < u.hi; p0 += kWaves * kTile) {
        // the lane's two keys
        int64_t row[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int p = p0 + 16 * b + col;
            row[b] = p < u.hi ? pages.row(p) : -1;
        }
        const bool there[2] = {row[0] >= 0, row[1] >= 0};
        u32x4_t kp[2][S::kPieces], vp[2][S::kPieces];
#pragma unroll
        for (int b = 0; b < 2; ++b) load_pieces<T, FORMAT, D>(k.a.cache.k, (there[b] ? row[b] : 0) * H + u.h, lane, kp[b]);
#pragma unroll
        for (int b = 0; b < 2; ++b) load_pieces<T, FORMAT, D>(k.a.cache.v, (there[b] ? row[b] : 0) * H + u.h, lane, vp[b]);
        float vscale[2] = {1.f, 1.f};
        if constexpr (S::kCodes) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const float ks = there[b] ? k.a.cache.k_scale[row[b] * H + u.h] : 0.f;
                vscale[b] = there[b] ? k.a.cache.v_scale[row[b] * H + u.h] : 0.f;
                if (quad == 0) {
                    scales[16 * b + col] = ks * c;
                    scales[kTile + 16 * b + col] = vscale[b];
                }
            }
        }
        // keys that are there, as bits
        const uint32_t present = (uint32_t)(__ballot(there[0]) & 0xffff) | (uint32_t)(__ballot(there[1]) & 0xffff) << 16;
        const bool partial = present != 0xffffffffu || p0 + kTile > some;

        f32x4_t s[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int b = 0; b < 2; ++b) s[n][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int f = 0; f < S::kFrags; ++f)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const dev::frag_t<T> kf = S::frag(kp[b], f);
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n][b] = dev::mma16(kf, q[n][f], s[n][b]);
            }
        uint32_t seen[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) seen[n] = partial ? (uint32_t)sees[n].from(p0) & present : 0xffffffffu;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float top = -INFINITY;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                f32x4_t by = {c, c, c, c};
                if constexpr (S::kCodes) by = *reinterpret_cast<const f32x4_t*>(scales + 16 * b + 4 * quad);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[n][b][i] *= by[i];
                    if (partial && !(seen[n] >> (16 * b + 4 * quad + i) & 1)) s[n][b][i] = -INFINITY;
                    top = fmaxf(top, s[n][b][i]);
                }
            }
            top = dev::across_max(top);
            const float next = fmaxf(m[n], top);
            if (__any(next > m[n])) {
                const float keep = m[n] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m[n] - next);
                l[n] *= keep;
#pragma unroll
                for (int t = 0; t < kDims; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][t][i] *= keep;
                m[n] = next;
            }
        }
        // V: through the wave's LDS.  Where some rows do not see some keys, what is not finite must not meet a weight of zero:
        // it is added to the rows that see it, and stands as zero in the product.
        bool fine = true;
#pragma unroll
        for (int b = 0; b < 2; ++b) fine &= stage<T, FORMAT, D>(vt, 16 * b + col, lane, vp[b], there[b], false);
        if (partial) {
            fine &= dev::finite(vscale[0]) && dev::finite(vscale[1]);
            uint64_t bad = __ballot(!fine);
            if (bad) {
                bad |= bad >> 32;
                bad |= bad >> 16;
                for (int key = 0; key < kTile; ++key) {
                    if (!(bad >> (key % 16) & 1)) continue;
                    float vs = 1.f;
                    if constexpr (S::kCodes) vs = scales[kTile + key];
#pragma unroll
                    for (int t = 0; t < kDims; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float v = VTile<T, D>::at(vt, key, 16 * t + 4 * quad + i);
                            if (!dev::finite(vs)) v = NAN;
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                if (!dev::finite(v) && (seen[n] >> key & 1)) o[n][t][i] += v;
                        }
                }
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    stage<T, FORMAT, D>(vt, 16 * b + col, lane, vp[b], there[b], true);
                    if (S::kCodes && quad == 0 && !dev::finite(vscale[b])) scales[kTile + 16 * b + col] = 0.f;
                }
            }
        }
        dev::frag_t<T> w[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float base = m[n] == -INFINITY ? 0.f : m[n];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                f32x4_t by = {1.f, 1.f, 1.f, 1.f};
                if constexpr (S::kCodes) by = *reinterpret_cast<const f32x4_t*>(scales + kTile + 16 * b + 4 * quad);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = __builtin_amdgcn_exp2f(s[n][b][i] - base);
                    l[n] += x;
                    w[n][4 * b + i] = (T)(x * by[i]);
                }
            }
        }
#pragma unroll
        for (int t = 0; t < kDims; ++t) {
            const dev::frag_t<T> vf = VTile<T, D>::load(vt, t, lane);
#pragma unroll
            for (int n = 0; n < NT; ++n) o[n][t] = dev::mma16(vf, w[n], o[n][t]);
        }
    }

    // the four waves' sums, 16 rows at a time
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        l[n] = dev::across_sum(l[n]);
        __syncthreads();
        float* const mine = reinterpret_cast<float*>(vt);
#pragma unroll
        for (int t = 0; t < kDims; ++t) *reinterpret_cast<f32x4_t*>(mine + col * (D + 4) + 16 * t + 4 * quad) = o[n][t];
        if (quad == 0) stats[wave * 16 + col] = {m[n], l[n]};
        __syncthreads();
        const int r = threadIdx.x / 16, row = u.row0 + 16 * n + r;
        float top = -INFINITY, sum = 0.f, by[kWaves];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stats[w * 16 + r].x);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            by[w] = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(stats[w * 16 + r].x - top);
            sum += by[w] * stats[w * 16 + r].y;
        }
        if (row < u.rows) {
            const int t = (int)dev::divide(row, k.group);
            const int64_t at = (u.first + t) * k.a.H_q + u.h * G + (row - t * G);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int e = 0; e < D / 64; ++e) {
                const int dim = 64 * e + threadIdx.x % 16 * 4;
                f32x4_t x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < kWaves; ++w) {
                    // a wave without keys holds zeros: nothing of it is taken
                    const f32x4_t v = *reinterpret_cast<const f32x4_t*>(reinterpret_cast<const float*>(lds + w * Lds<T, D>::kWave) + r * (D + 4) + dim);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] += by[w] * v[i];
                }
                if (u.spans > 1) {
                    *reinterpret_cast<f32x4_t*>(k.part + (at * k.spans + u.span) * D + dim) = x;
                } else {
                    T* out = static_cast<T*>(k.a.o) + at * D + dim;
#pragma unroll
                    for (int i = 0; i < 4; ++i) out[i] = (T)(x[i] * inv);
                }
            }
            if (u.spans > 1 && threadIdx.x % 16 == 0) k.stats[at * k.spans + u.span] = {top, sum};
        }
    }
}

template <typename T, int FORMAT, int D, int NT>
__global__ __launch_bounds__(kThreads) void decode_kernel(AttentionKernelArgs k) {
    extern __shared__ __align__(16) char lds[];
    Unit u;
    if (decode_unit<T, D>(k, 16 * NT, kThreads, u)) attend<T, FORMAT, D, NT>(k, u, lds);
}

template <typename T, int FORMAT, int D, int NT>
__global__ __launch_bounds__(kThreads) void prompt_kernel(AttentionKernelArgs k) {
    extern __shared__ __align__(16) char lds[];
    const unsigned H = (unsigned)k.a.cache.num_heads, tile = blockIdx.x / H;
    Unit u;
    if (prompt_unit(k, 16 * NT, (int)tile, (int)(blockIdx.x - tile * H), u)) attend<T, FORMAT, D, NT>(k, u, lds);
}

// A row's spans joined: one wave for each query head of a token.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void join_kernel(AttentionKernelArgs k) {
    const int64_t at = (int64_t)blockIdx.x * (kThreads / 64) + threadIdx.x / 64;
    const int lane = threadIdx.x & 63;
    if (at >= k.a.total_tokens * k.a.H_q) return;
    const int64_t token = at / k.a.H_q;
    const int keys = row_keys(k.a, k.a.past[dev::divide((unsigned)token, k.rows)]);
    if (keys <= 0 || keys > k.a.max_keys) return;
    const int span = span_keys(k.a.tokens_per_row * (int)k.group.d, keys), spans = (keys + span - 1) / span;
    if (spans == 1) return;
    const float2 mine = lane < spans ? k.stats[at * k.spans + lane] : float2{-INFINITY, 0.f};
    float top = mine.x;
#pragma unroll
    for (int i = 1; i < 64; i *= 2) top = fmaxf(top, __shfl_xor(top, i));
    const float by = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mine.x - top);
    const float sum = dev::group_sum(by * mine.y, 64);
    constexpr int N = D / 64;
    float x[N] = {};
    const float* p = k.part + at * k.spans * D + lane * N;
    for (int s = 0; s < spans; ++s) {
        const float f = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, by), s));
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] += f * p[s * D + i];
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    T* o = static_cast<T*>(k.a.o) + at * D + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = (T)(x[i] * inv);
}

// ---------------------------------------------------------------- launches

AttentionKernelArgs kernel_args(const AttentionArgs& a) {
    AttentionKernelArgs k = {};
    k.a = a;
    if (a.cache.num_rows == 0) {        // no key is there
        k.a.capacity = 0;
        k.a.max_keys = 0;
    }
    k.block = Divisor((uint32_t)a.kv_block);
    k.group = Divisor((uint32_t)(a.H_q / a.cache.num_heads));
    return k;
}

int most_spans(int rows, int64_t keys) {
    const int64_t n = (keys + least_span(rows) - 1) / least_span(rows);
    return (int)(n < kMaxSpans ? (n > 0 ? n : 1) : kMaxSpans);
}

template <typename T, int FORMAT, int D, int NT>
hipError_t launch_rows(AttentionKernelArgs k, hipStream_t stream) {
    const int rows = k.a.tokens_per_row * (int)k.group.d;
    k.row_tiles = (rows + 16 * NT - 1) / (16 * NT);
    const int64_t blocks = ((int64_t)k.a.num_seqs * k.spans * k.a.cache.num_heads + 7) / 8 * 8 * k.row_tiles;
    if (!grid_fits(blocks, kThreads)) return hipErrorInvalidConfiguration;
    decode_kernel<T, FORMAT, D, NT><<<(unsigned)blocks, kThreads, Lds<T, D>::kTotal, stream>>>(k);
    return hipGetLastError();
}

template <typename T, int FORMAT, int D>
hipError_t launch_decode(const AttentionArgs& a, hipStream_t stream) {
    AttentionKernelArgs k = kernel_args(a);
    const int rows = a.tokens_per_row * (int)k.group.d;
    k.rows = Divisor((uint32_t)a.tokens_per_row);
    k.spans = most_spans(rows, k.a.max_keys);
    const int64_t heads = a.total_tokens * a.H_q, joins = (heads + kThreads / 64 - 1) / (kThreads / 64);
    if (!grid_fits(joins, kThreads)) return hipErrorInvalidConfiguration;
    k.part = static_cast<float*>(a.workspace);
    k.stats = reinterpret_cast<float2*>(k.part + (k.spans > 1 ? heads * k.spans * D : 0));
    // as many row tiles to a wave as the rows fill and the registers hold
    constexpr int most = (sizeof(T) == 2 ? 512 : 256) / D;
    hipError_t e;
    if (sizeof(T) == 2 && rows > 64) e = launch_attention_wide(k, stream);
    else if (rows <= 16 || most == 1) e = launch_rows<T, FORMAT, D, 1>(k, stream);
    else if (rows <= 32 || most == 2) e = launch_rows<T, FORMAT, D, (most > 1 ? 2 : 1)>(k, stream);
    else e = launch_rows<T, FORMAT, D, (most > 2 ? 4 : 1)>(k, stream);
    if (e != hipSuccess || k.spans == 1) return e;
    join_kernel<T, D><<<(unsigned)joins, kThreads, 0, stream>>>(k);
    return hipGetLastError();
}

template <int FORMAT, int D>
hipError_t launch_prompt(const AttentionArgs& a, hipStream_t stream) {
    constexpr int NT = D <= 64 ? 4 : (D <= 128 ? 2 : 1);
    const AttentionKernelArgs k = kernel_args(a);
    const int64_t tiles = a.total_tokens * (int)k.group.d / (16 * NT) + a.num_seqs, blocks = tiles * a.cache.num_heads;
    if (!grid_fits(blocks, kThreads) || a.total_tokens * (int64_t)k.group.d > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    prompt_kernel<float, FORMAT, D, NT><<<(unsigned)blocks, kThreads, Lds<float, D>::kTotal, stream>>>(k);
    return hipGetLastError();
}

template <typename T, int FORMAT, int D>
hipError_t launch(const AttentionArgs& a, hipStream_t stream) {
    if (a.tokens_per_row > 0) return launch_decode<T, FORMAT, D>(a, stream);
    if constexpr (sizeof(T) == 2) return launch_attention_wide(kernel_args(a), stream);
    else return launch_prompt<FORMAT, D>(a, stream);
}

template <typename T, int FORMAT>
hipError_t launch(const AttentionArgs& a, hipStream_t stream) {
    if (a.cache.head_dim == 64) return launch<T, FORMAT, 64>(a, stream);
    if (a.cache.head_dim == 128) return launch<T, FORMAT, 128>(a, stream);
    return launch<T, FORMAT, 256>(a, stream);
}

template <typename T>
hipError_t launch(const AttentionArgs& a, hipStream_t stream) {
    if (a.cache.format == GDN_CACHE_PLAIN) return launch<T, GDN_CACHE_PLAIN>(a, stream);
    if (a.cache.format == GDN_CACHE_E4M3) return launch<T, GDN_CACHE_E4M3>(a, stream);
    return launch<T, GDN_CACHE_INT8>(a, stream);
}

hipError_t launch(const AttentionArgs& a, hipStream_t stream) {
    return a.cache.dtype == GDN_BF16 ? launch<__bf16>(a, stream) : launch<float>(a, stream);
}

}  // namespace

// Partial sums and statistics of every query head's spans; the most over all smaller calls.
size_t attention_workspace_bytes(int H_q, int H_kv, int head_dim, int num_rows, int tokens_per_row, int64_t max_keys) {
    size_t most = 0;
    for (int t = 1; t <= tokens_per_row; ++t) {
        const int spans = most_spans(t * (H_q / H_kv), max_keys);
        if (spans > 1) {
            const size_t n = (size_t)num_rows * t * H_q * spans * (head_dim * sizeof(float) + sizeof(float2));
            most = n > most ? n : most;
        }
    }
    return most;
}

hipError_t launch_attention_prefill(const AttentionArgs& a, hipStream_t stream) { return launch(a, stream); }
hipError_t launch_attention_decode(const AttentionArgs& a, hipStream_t stream) { return launch(a, stream); }

}  // namespace gdn
