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
// never move between lanes and a row's factors are the lane's own.
//
// Memory bounds it: a decode row reads its whole context for a few products.  Loads take
// whole cache rows, neighbouring lanes neighbouring bytes, one tile ahead of the sums in registers, and
// go through the wave's own LDS, so that no wave waits for another.  (Loaded straight into the operands, 16 lanes in
// 16 rows, K took the memory path up to four times as long: 298 us instead of 266 for 64 requests of up to 8192 keys, 136
// instead of 66 for one of 131072 keys in 8 bits.)  Now 240 us, 5.1 TB/s of keys and values, and 58.7 us, 4.7 TB/s.
// fp32 prompts share a staged tile among 16 or 32 rows of one wave only: 4096 tokens of 8 heads over 2, 128 dims, 505 us, 68 TFLOP/s
// of 153 for a large library product; 256 dims 1.26 ms, 55 TFLOP/s, one wave to a SIMD.
//
// With bf16 the weights are rounded to bf16 for the second product.  As two bf16 parts each, in two products, they left only the
// output's rounding: 240.5 us for 240.0, but 17.1 for 16.3 and 41.4 for 38.2 (16 requests of 4096 keys in 8 bits, two heads of
// 128 and 256 dims), where 8-bit values are further off already.
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

// A wave's tiles of K and V in LDS, as values of T, in 16-byte chunks.  Chunks of a key are exchanged by the key, so that operands
// (K: one chunk of 16 keys; V: two chunks of four keys to a group of 16 lanes) do not meet in a bank; V's rows are
// padded instead where the elements are single words.
template <typename T, int D>
struct Tile {
    static constexpr int kRow = D * (int)sizeof(T), kChunks = kRow / 16;                     // of K
    static constexpr int kVRow = sizeof(T) == 2 ? kRow : kRow + 16;
    static constexpr int kSum = 16 * (D + 4) * 4;                                           // 16 rows of a wave's sums
    // Where two tiles fit twice into LDS, V has a place of its own and is loaded and staged beside K, else it takes K's after
    // the scores: 57.6 us beside and 65 after (131072 keys of 128 dims in 8 bits); but 44.5 and 42.1 (16 x 4096 keys of 256
    // dims in bf16), 608 and 362 (a prompt of 2048 tokens, 256 dims in fp32, whose two tiles leave room for two waves).
    static constexpr bool kBeside = kRow <= 256;
    static constexpr int kV = kBeside ? kTile * kRow : 0, kUsed = kV + kTile * kVRow, kBytes = kUsed > kSum ? kUsed : kSum;
    __device__ static __forceinline__ int k(int key, int c) { return key * kRow + (c ^ (kChunks >= 16 ? key & 15 : key >> 1 & 7)) * 16; }
    __device__ static __forceinline__ int v(int key, int c) {
        if constexpr (sizeof(T) == 4) return kV + key * kVRow + c * 16;
        else if constexpr (D >= 128) return kV + key * kVRow + ((c ^ ((2 * key) & 15)) * 16);
        else return kV + key * kVRow + ((c ^ (key & 6)) * 16);
    }
    // first of the lane's eight dims of operand f of the scores; the last four of fp32 stand 16 further
    __device__ static __forceinline__ int dim(int f, int lane) { return f * 32 + lane / 16 * (16 / (int)sizeof(T)); }
    __device__ static __forceinline__ dev::frag_t<T> query(const T* q, int f, int lane) {
        if constexpr (sizeof(T) == 2) return *reinterpret_cast<const dev::bf16x8_t*>(q + dim(f, lane));
        else return __builtin_shufflevector(*reinterpret_cast<const f32x4_t*>(q + dim(f, lane)), *reinterpret_cast<const f32x4_t*>(q + dim(f, lane) + 16), 0, 1, 2, 3, 4, 5, 6, 7);
    }
    __device__ static __forceinline__ dev::frag_t<T> load_k(const char* lds, int key, int f, int lane) {
        if constexpr (sizeof(T) == 2) return *reinterpret_cast<const dev::bf16x8_t*>(lds + k(key, 4 * f + lane / 16));
        else return __builtin_shufflevector(*reinterpret_cast<const f32x4_t*>(lds + k(key, 8 * f + lane / 16)),
                                            *reinterpret_cast<const f32x4_t*>(lds + k(key, 8 * f + 4 + lane / 16)), 0, 1, 2, 3, 4, 5, 6, 7);
    }
    // V^T for dims 16 t .. 16 t + 15: lane % 16 is the dim, the eight keys 4 (lane / 16) + 0..3 of both halves of the tile
    __device__ static __forceinline__ dev::frag_t<T> load_v(const char* lds, int t, int lane) {
        if constexpr (sizeof(T) == 2) {
            const int key = 4 * (lane / 16) + lane % 16 / 4, c = 2 * t + (lane & 3) / 2;
            typedef __attribute__((address_space(3))) dev::s16x4_t* lds_ptr;
            const auto a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(lds + v(key, c) + (lane & 1) * 8));
            const auto b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(lds + v(key + 16, c) + (lane & 1) * 8));
            const dev::bf16x4_t x = __builtin_bit_cast(dev::bf16x4_t, a), y = __builtin_bit_cast(dev::bf16x4_t, b);
            return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
        } else {
            dev::f32x8_t f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int key = 16 * (j / 4) + 4 * (lane / 16) + j % 4;
                f[j] = *reinterpret_cast<const float*>(lds + kV + key * kVRow + (16 * t + lane % 16) * 4);
            }
            return f;
        }
    }
    __device__ static __forceinline__ T& v_at(char* lds, int key, int dim) {
        return *reinterpret_cast<T*>(lds + v(key, dim * (int)sizeof(T) / 16) + dim * (int)sizeof(T) % 16);
    }
};

// LDS of a workgroup: a tile of each wave, which the waves' sums share at the end; then the waves' scales and statistics.
template <typename T, int D>
struct Lds {
    static constexpr int kWave = Tile<T, D>::kBytes;
    static constexpr int kScales = kWaves * 2 * kTile * 4;
    static constexpr int kTotal = kWaves * kWave + kScales + kWaves * 16 * 8;
};

template <typename T, int FORMAT, int D, int NT>
__device__ __forceinline__ void attend(const AttentionKernelArgs& k, const Unit& u, char* lds) {
    using Tl = Tile<T, D>;
    constexpr bool kCodes = FORMAT != GDN_CACHE_PLAIN;
    constexpr int kRowBytes = D * (kCodes ? 1 : (int)sizeof(T));
    constexpr int kPieces = kRowBytes / 16, kKeys = 64 / kPieces, kLoads = kTile / kKeys;        // a load of a wave takes kKeys whole rows
    constexpr int kDims = D / 16, kFrags = D / 32;
    if (u.lo >= u.hi) {        // a table or a cache without rows: no address may be formed
        fill_rows<T, D>(k, u, 16 * NT, kThreads, 0.f);
        return;
    }
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane % 16, quad = lane / 16, G = (int)k.group.d;
    char* const tile = lds + wave * Lds<T, D>::kWave;
    float* const scales = reinterpret_cast<float*>(lds + kWaves * Lds<T, D>::kWave) + wave * 2 * kTile;
    float2* const stats = reinterpret_cast<float2*>(lds + kWaves * Lds<T, D>::kWave + Lds<T, D>::kScales);
    const dev::Pages pages = {k.a.table + (int64_t)u.seq * k.a.table_width, k.a.table_width, k.block, k.a.cache.num_rows};
    const int H = k.a.cache.num_heads;
    const float c = k.a.scale * kLog2e;

    // ---- loads: the lane's key and its page's entry (in flight) two tiles ahead, values one.  Lanes l and l + 32 hold the same key.
    int entry = -1, key = 0, row = -1;
    const auto lookup = [&](int p0) {
        key = p0 + (lane & 31);
        entry = pages.entry(key);
    };
    u32x4_t kp[kLoads], vp[kLoads];
    float scale = 0.f;                                  // of the lane's key: K's in the lower half of the wave, V's in the upper
    const auto load = [&](const void* cache, u32x4_t (&p)[kLoads]) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = __shfl(row, i * kKeys + lane / kPieces);
            const uint64_t at = (uint64_t)(unsigned)(r < 0 ? 0 : r) * (unsigned)(H * kRowBytes) + (unsigned)(u.h * kRowBytes + lane % kPieces * 16);
            p[i] = *reinterpret_cast<const u32x4_t*>(static_cast<const char*>(cache) + at);
        }
    };
    const auto load_scales = [&]() {
        if constexpr (kCodes) scale = row >= 0 ? (lane < 32 ? k.a.cache.k_scale : k.a.cache.v_scale)[(int64_t)row * H + u.h] : 0.f;
    };
    // What was loaded, in LDS as values; with `there`, keys that are absent as zeros.
    const auto stage = [&](const u32x4_t (&p)[kLoads], auto place, uint32_t there) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int n = i * kKeys + lane / kPieces, first = lane % kPieces;
            u32x4_t v = p[i];
            if (there != 0xffffffffu && !(there >> n & 1)) v = u32x4_t{};
            if constexpr (!kCodes) {
                *reinterpret_cast<u32x4_t*>(tile + place(n, first)) = v;
            } else {
                asm volatile("" : "+v"(v));                // (else integers are taken apart where they are loaded, a tile ahead)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const dev::frag_t<T> f = dev::codes8<T, FORMAT>(v[2 * x], v[2 * x + 1]);
                    if constexpr (sizeof(T) == 2) {
                        *reinterpret_cast<dev::bf16x8_t*>(tile + place(n, 2 * first + x)) = f;
                    } else {
                        *reinterpret_cast<f32x4_t*>(tile + place(n, 4 * first + 2 * x)) = __builtin_shufflevector(f, f, 0, 1, 2, 3);
                        *reinterpret_cast<f32x4_t*>(tile + place(n, 4 * first + 2 * x + 1)) = __builtin_shufflevector(f, f, 4, 5, 6, 7);
                    }
                }
            }
        }
    };
    // Whether the lane's share of V in LDS is finite; all of V, what is not as zeros.
    const auto all_finite = [lane](char* lds) {
        constexpr int kOfChunk = 16 / (int)sizeof(T);
        bool fine = true;
        for (int i = lane; i < kTile * Tl::kChunks; i += 64) {
            const T* const v = &Tl::v_at(lds, i / Tl::kChunks, i % Tl::kChunks * kOfChunk);
#pragma unroll
            for (int j = 0; j < kOfChunk; ++j) fine &= dev::finite((float)v[j]);
        }
        return fine;
    };
    const auto zero_others = [lane](char* lds) {
        for (int i = lane; i < kTile * D; i += 64)
            if (!dev::finite((float)Tl::v_at(lds, i / D, i % D))) Tl::v_at(lds, i / D, i % D) = (T)0.f;
    };
    const auto place_k = [](int n, int c) { return Tl::k(n, c); };
    const auto place_v = [](int n, int c) { return Tl::v(n, c); };
    int p0 = u.lo + wave * kTile;
    const bool any = p0 < u.hi;
    if (any) {
        lookup(p0);
        row = pages.row(key, entry, u.hi);
        load_scales();
        load(k.a.cache.k, kp);
        lookup(p0 + kWaves * kTile);
        load(k.a.cache.v, vp);
    }
    uint32_t present = (uint32_t)__ballot(row >= 0);

    dev::frag_t<T> q[NT][kFrags];
    dev::Sees sees[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = u.row0 + 16 * n + col, t = (int)dev::divide(r, k.group);
        sees[n] = {0, 0, 0};
        if (r < u.rows) {
            const T* p = static_cast<const T*>(k.a.q) + (u.first + t) * k.a.q_stride + (int64_t)(u.h * G + (r - t * G)) * D;
#pragma unroll
            for (int f = 0; f < kFrags; ++f) q[n][f] = Tl::query(p, f, lane);
            sees[n] = row_sees(k, u, r);
        } else {
#pragma unroll
            for (int f = 0; f < kFrags; ++f) q[n][f] = dev::frag_t<T>{};
        }
        // waited for here: in the loop the wait would be for the tile on its way as well
#pragma unroll
        for (int f = 0; f < kFrags; ++f) asm volatile("" : "+v"(q[n][f]));
        asm volatile("" : "+v"(sees[n].all), "+v"(sees[n].first), "+v"(sees[n].mask));
    }
    const int some = k.a.tree_mask ? u.past : causal_keys(k, u, u.row0);        // every row sees the keys below

    f32x4_t o[NT][kDims] = {};
    float m[NT], l[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) { m[n] = -INFINITY; l[n] = 0.f; }

    for (; p0 < u.hi; p0 += kWaves * kTile) {
        const uint32_t there = present;
        const bool partial = there != 0xffffffffu || p0 + kTile > some, more = p0 + kWaves * kTile < u.hi;
        stage(kp, place_k, 0xffffffffu);
        if constexpr (kCodes) scales[lane] = lane < 32 ? scale * c : (dev::finite(scale) ? scale : NAN);        // (an infinite scale is a NaN one)
        if (Tl::kBeside) stage(vp, place_v, there);
        if (more) {
            row = pages.row(key, entry, u.hi);
            present = (uint32_t)__ballot(row >= 0);
            load_scales();
            load(k.a.cache.k, kp);
            if (Tl::kBeside) load(k.a.cache.v, vp);
            lookup(p0 + 2 * kWaves * kTile);         // (before V: what waits for it waits for every load before it)
        }
        uint32_t seen[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) seen[n] = partial ? (uint32_t)sees[n].from(p0) & there : 0xffffffffu;

        f32x4_t s[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int b = 0; b < 2; ++b) s[n][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int f = 0; f < kFrags; ++f)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const dev::frag_t<T> kf = Tl::load_k(tile, 16 * b + col, f, lane);
#pragma unroll
                for (int n = 0; n < NT; ++n) s[n][b] = dev::mma16(kf, q[n][f], s[n][b]);
            }
        dev::frag_t<T> w[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float top = -INFINITY;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                f32x4_t by = {c, c, c, c};
                if constexpr (kCodes) by = *reinterpret_cast<const f32x4_t*>(scales + 16 * b + 4 * quad);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[n][b][i] *= by[i];
                    if (partial && !(seen[n] >> (16 * b + 4 * quad + i) & 1)) s[n][b][i] = -INFINITY;
                    top = fmaxf(top, s[n][b][i]);
                }
            }
            top = dev::across_max(top);
            // kept until it is short by 2^8, which sums and weights take as well: the sums are seldom scaled
            const float next = top > m[n] + 8.f ? top : m[n];
            if (__any(next > m[n])) {
                const float keep = m[n] == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m[n] - next);        // (no sums yet)
                l[n] *= keep;
#pragma unroll
                for (int t = 0; t < kDims; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[n][t][i] *= keep;
                m[n] = next;
            }
        }
        if (!Tl::kBeside) {
            stage(vp, place_v, there);
            if (more) load(k.a.cache.v, vp);
        }
        // Where some rows do not see some keys, no value that is not finite may meet a weight of zero that stands for that: it is added to
        // the rows that see it, and is a zero in the product.  Codes and scales can only be NaN.
        if (kCodes && partial) {
            if (__builtin_expect(__any(!(all_finite(tile) && dev::finite(scales[kTile + (lane & 31)]))), 0)) {
                for (int n = 0; n < kTile; ++n) {
                    if (!(there >> n & 1)) continue;
                    const bool no = !dev::finite(scales[kTile + n]);
#pragma unroll
                    for (int t = 0; t < kDims; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float v = no ? NAN : (float)Tl::v_at(tile, n, 16 * t + 4 * quad + i);
#pragma unroll
                            for (int x = 0; x < NT; ++x)
                                if (!dev::finite(v) && (seen[x] >> n & 1)) o[x][t][i] += v;
                        }
                }
                zero_others(tile);
                if (lane >= 32 && !dev::finite(scales[lane])) scales[lane] = 0.f;
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const float base = m[n] == -INFINITY ? 0.f : m[n];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                f32x4_t by = {1.f, 1.f, 1.f, 1.f};
                if constexpr (kCodes) by = *reinterpret_cast<const f32x4_t*>(scales + kTile + 16 * b + 4 * quad);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = __builtin_amdgcn_exp2f(s[n][b][i] - base);
                    if constexpr (kCodes || sizeof(T) == 4) l[n] += x;
                    w[n][4 * b + i] = (T)(x * by[i]);
                }
            }
            // the rounded weights' sum (see gdn_attention_wide.hip)
            if constexpr (!kCodes && sizeof(T) == 2) l[n] += dev::sum8(w[n], 0.f);
        }
        // The same of plain values, infinities among them: they are added times their weights, as the product would take them.
        if (!kCodes && partial) {
            if (__builtin_expect(__any(!all_finite(tile)), 0)) {
                for (int j = 0; j < kTile; ++j) {
                    if (!(there >> j & 1)) continue;
                    float by[NT];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {        // the weight of the lane's row, from the lane that holds the key
                        by[n] = 0.f;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (j == 16 * (i / 4) + 4 * quad + i % 4) by[n] = (float)w[n][i];
                        by[n] = __shfl(by[n], j % 16 / 4 * 16 + col);
                    }
#pragma unroll
                    for (int t = 0; t < kDims; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float v = (float)Tl::v_at(tile, j, 16 * t + 4 * quad + i);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                if (!dev::finite(v) && (seen[n] >> j & 1)) o[n][t][i] += by[n] * v;
                        }
                }
                zero_others(tile);
            }
        }
#pragma unroll
        for (int t = 0; t < kDims; ++t) {
            const dev::frag_t<T> vf = Tl::load_v(tile, t, lane);
#pragma unroll
            for (int n = 0; n < NT; ++n) o[n][t] = dev::mma16(vf, w[n], o[n][t]);
        }
    }

    // the waves' sums, 16 rows at a time
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        l[n] = dev::across_sum(l[n]);
        __syncthreads();
        float* const mine = reinterpret_cast<float*>(tile);
#pragma unroll
        for (int t = 0; t < kDims; ++t) *reinterpret_cast<f32x4_t*>(mine + col * (D + 4) + 16 * t + 4 * quad) = o[n][t];
        if (quad == 0) stats[wave * 16 + col] = {m[n], l[n]};
        __syncthreads();
#pragma unroll
        for (int r = threadIdx.x / 16; r < 16; r += kThreads / 16) {
            const int row = u.row0 + 16 * n + r;
            if (row >= u.rows) break;
            float top = -INFINITY, sum = 0.f, by[kWaves];
#pragma unroll
            for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stats[w * 16 + r].x);
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                by[w] = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(stats[w * 16 + r].x - top);
                sum += by[w] * stats[w * 16 + r].y;
            }
            const int t = (int)dev::divide(row, k.group);
            const int64_t at = (u.first + t) * k.a.H_q + u.h * G + (row - t * G);
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
            for (int e = 0; e < D / 64; ++e) {
                const int dim = 64 * e + threadIdx.x % 16 * 4;
                f32x4_t x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < kWaves; ++w) {
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

// Most tiles of 16 rows to a wave: more spill hundreds of bytes.
template <typename T, int D>
constexpr int row_tiles() { return D == 256 ? 1 : (D == 128 || sizeof(T) == 4 ? 2 : 4); }

// Workgroups of a compute unit, as waves to a SIMD, by the registers that a wave's tile, sums and queries take.
template <typename T, int D>
constexpr int workgroups() { return Tile<T, D>::kBeside ? 2 : 1; }

template <typename T, int FORMAT, int D, int NT>
__global__ __launch_bounds__(kThreads, (workgroups<T, D>())) void decode_kernel(AttentionKernelArgs k) {
    extern __shared__ __align__(16) char lds[];
    Unit u;
    if (decode_unit<T, D>(k, 16 * NT, kThreads, u)) attend<T, FORMAT, D, NT>(k, u, lds);
}

template <typename T, int FORMAT, int D, int NT>
__global__ __launch_bounds__(kThreads, (workgroups<T, D>())) void prompt_kernel(AttentionKernelArgs k) {
    extern __shared__ __align__(16) char lds[];
    const unsigned H = (unsigned)k.a.cache.num_heads, tile = blockIdx.x / H;
    Unit u;
    if (prompt_unit(k, 16 * NT, (int)tile, (int)(blockIdx.x - tile * H), u)) attend<T, FORMAT, D, NT>(k, u, lds);
}

// A row's spans joined, in four sums of every fourth span: a workgroup for each query head of a token, a sum to each wave, or
// (W = 1, up to 16 spans) a wave for it.  Two ways, the same bits: 64 spans took one wave 11 us of dependent
// loads, of a workgroup 3 us; 16384 heads of up to 9 spans 10 us more in a workgroup each.
template <typename T, int D, int W>
__global__ __launch_bounds__(kThreads) void join_kernel(AttentionKernelArgs k) {
#pragma clang fp contract(off)             // a product that one of them fused into the sum of the statistics would round differently
    constexpr int N = D / 64, kHeads = kWaves / W, kSums = 4 / W, kEach = 4 * W;        // heads of a workgroup; sums of a wave, spans of a sum
    static_assert(kWaves == 4 && kMaxSpans == 64, "");
    __shared__ float sums[W == 1 ? 1 : 4][D];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, first = wave % W * kSums;
    const int64_t at = (int64_t)blockIdx.x * kHeads + wave / W;
    if (at >= k.a.total_tokens * k.a.H_q) return;
    const unsigned token = (unsigned)at / (unsigned)k.a.H_q;
    const int keys = row_keys(k.a, k.a.past[dev::divide(token, k.rows)]);
    if (keys <= 0 || keys > k.a.max_keys) return;
    const int span = span_keys(k.a.tokens_per_row * (int)k.group.d, keys), spans = span_count(keys, span);
    if (spans == 1) return;
    const float2 mine = lane < spans ? k.stats[at * k.spans + lane] : float2{-INFINITY, 0.f};
    float x[kSums][N] = {}, v[kEach][kSums][N];
    const float* p = k.part + at * k.spans * D + lane * N;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
#pragma unroll
        for (int w = 0; w < kSums; ++w)
#pragma unroll
            for (int j = 0; j < N; ++j) v[i][w][j] = 4 * i + first + w < spans ? p[(4 * i + first + w) * D + j] : 0.f;
    float top = mine.x;
#pragma unroll
    for (int i = 1; i < 64; i *= 2) top = fmaxf(top, __shfl_xor(top, i));
    const float by = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mine.x - top);
    const float sum = dev::group_sum(by * mine.y, 64), inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < kEach; ++i)
#pragma unroll
        for (int w = 0; w < kSums; ++w) {
            const float f = __shfl(by, 4 * i + first + w);
#pragma unroll
            for (int j = 0; j < N; ++j) x[w][j] = fmaf(f, v[i][w][j], x[w][j]);
        }
    T* const o = static_cast<T*>(k.a.o) + at * D;
    if constexpr (W == 1) {
#pragma unroll
        for (int j = 0; j < N; ++j) o[lane * N + j] = (T)((((x[0][j] + x[1][j]) + x[2][j]) + x[3][j]) * inv);
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) sums[wave][lane * N + j] = x[0][j];
        __syncthreads();
        const int dim = threadIdx.x;
        if (dim < D) o[dim] = (T)((((sums[0][dim] + sums[1][dim]) + sums[2][dim]) + sums[3][dim]) * inv);
    }
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
    const int64_t heads = a.total_tokens * a.H_q, joins = k.spans <= 16 ? (heads + kWaves - 1) / kWaves : heads;
    if (k.spans > 1 && !grid_fits(joins, kThreads)) return hipErrorInvalidConfiguration;
    k.part = static_cast<float*>(a.workspace);
    k.stats = reinterpret_cast<float2*>(k.part + (k.spans > 1 ? heads * k.spans * D : 0));
    // as many row tiles to a wave as the rows fill and the registers hold; more rows share the keys in gdn_attention_wide.hip (two
    // heads of 16 requests with 4096 keys, here / there: 64 dims, 32 rows 15.8 / 16.2 us, 64 rows 22.7 / 19.6, 96 rows 31.7 / 26.0; 128
    // dims, 32 rows 25.6 / 20.8, 48 rows 35.6 / 25.7, 64 rows 36.8 / 26.4; 256 dims, 32 rows 57.3 / 52.9, 64 rows 90.7 / 58.4)
    constexpr int most = row_tiles<T, D>();
    hipError_t e;
    if (sizeof(T) == 2 && rows > 16 * most) e = launch_attention_wide(k, stream);
    else if (rows <= 16 || most == 1) e = launch_rows<T, FORMAT, D, 1>(k, stream);
    else if (rows <= 32 || most == 2) e = launch_rows<T, FORMAT, D, (most > 1 ? 2 : 1)>(k, stream);
    else e = launch_rows<T, FORMAT, D, (most > 2 ? 4 : 1)>(k, stream);
    if (e != hipSuccess || k.spans == 1) return e;
    auto* const join = k.spans <= 16 ? join_kernel<T, D, 1> : join_kernel<T, D, 4>;
    join<<<(unsigned)joins, kThreads, 0, stream>>>(k);
    return hipGetLastError();
}

template <int FORMAT, int D, int NT>
hipError_t launch_prompt(const AttentionKernelArgs& k, hipStream_t stream) {
    const int64_t tiles = k.a.total_tokens * (int)k.group.d / (16 * NT) + k.a.num_seqs, blocks = tiles * k.a.cache.num_heads;
    if (!grid_fits(blocks, kThreads) || k.a.total_tokens * (int64_t)k.group.d > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    prompt_kernel<float, FORMAT, D, NT><<<(unsigned)blocks, kThreads, Lds<float, D>::kTotal, stream>>>(k);
    return hipGetLastError();
}

// One row tile to a wave where two would leave compute units without work (one / two of 128 dims, 8 heads over 2: 512 tokens
// 22.3 / 31.2 us, 1024 59 / 56, 4096 602 / 505; of 64 dims 12.7 / 17.9, 27.6 / 31.3, 235 / 221).
template <int FORMAT, int D>
hipError_t launch_prompt(const AttentionArgs& a, hipStream_t stream) {
    constexpr int most = row_tiles<float, D>();
    const AttentionKernelArgs k = kernel_args(a);
    if (most == 1 || a.total_tokens * a.H_q <= 16 * most * 256) return launch_prompt<FORMAT, D, 1>(k, stream);
    return launch_prompt<FORMAT, D, most>(k, stream);
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
