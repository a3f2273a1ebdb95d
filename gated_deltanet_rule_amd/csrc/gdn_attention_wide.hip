// gdn_attention_wide.hip -- attention of many query rows over a paged cache for gfx950: bf16
// prompts, and decode rows of many tokens.
//
// The same sums as gdn_attention.hip, for rows enough to share the keys: four waves of 32 rows take
// the same tiles of 64 keys from LDS, where two of K and two of V stand in turn.  Plain values
// go there past the registers, codes through them, widened.  The products are transposed here
// too, 32 x 32 tiles with a query row to each pair of lanes, so that weights are the second
// product's operand as they come out of the first.
//
// The matrix cores bound it, as far as they are fed: a wave's products take 1024 cycles of a tile at 128 dims, its softmax 700
// of the vector ALU, which the other wave of the SIMD has to fill.  8 prompts of up to 4096 tokens, 128 dims: 452 to 470
// us, 870 TFLOP/s where a large library product reaches 1150.  (Its clock is what the card's power leaves: 2.06 to 1.83 GHz by the cycles
// counted in 30 calls in a row, 482 to 553 us.)  8192 tokens behind 24576, 256 dims, 8-bit codes: 4.87 ms, 790
// TFLOP/s with one wave to a SIMD.  Trees of 32 tokens (128 rows) of 16 requests: 108 us with the join, 420 TFLOP/s, held by the
// start and end of each span.  A prompt's keys are not split over workgroups: 16 tokens behind 32768, 8 heads, are 8 workgroups, 704
// us (a chain of decoded tokens: 41).  Tried and not better: eight waves in two phases (466 and 463 us), four tiles of
// 32 keys in turn (477), loads behind the scores (511), the next tile's scores beside this one's exponentials (458, but spilling at 256
// dims), wave priorities, a workgroup's heads on one XCD.
//
// Weights are rounded to bf16 for the second product, the one rounding below fp32: as two bf16 parts they would take half as many
// products again, of what bounds the kernel.
#include <hip/hip_runtime.h>

#include "gdn_attention_device.h"
#include "gdn_device.h"
#include "gdn_layer_internal.h"

namespace gdn {
namespace {

using dev::bf16x8_t;
using dev::f32x4_t;
using dev::f32x16_t;
using dev::u32x4_t;

constexpr int kWaves = 4, kThreads = 64 * kWaves, kRowsOfTile = 32 * kWaves, kTile = 64;

__device__ __forceinline__ f32x16_t mma32(bf16x8_t a, bf16x8_t b, f32x16_t acc) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0); }

template <typename V>
using lds_ptr = __attribute__((address_space(3))) V*;
typedef lds_ptr<char> lds_t;

// Tiles of bf16 values in LDS: blocks of 8 keys by 64 dims, 1 KB each, key after key, which one load of a wave fills (16
// bytes a lane, in lanes' order) from 128 bytes of each key: four neighbouring lanes have to stand in the same 64 bytes of
// memory, or a load takes the memory path up to four times as long (1 KB: 17 cycles, or 65).  The 16-byte chunks of a key
// are exchanged: K's operands take one chunk of 16 keys at a time, V's transposing loads 64 bytes of four, and neither
// meets itself in a bank.
template <int D>
struct Tile {
    static constexpr int kBytes = kTile * D * 2;
    __device__ static constexpr int block(int key8, int dim64) { return (key8 * (D / 64) + dim64) * 1024; }
    // where chunk c (eight dims) of a key stands
    __device__ static constexpr int kswap(int key) { return key >> 1 & 7; }
    __device__ static constexpr int vswap(int key) { return 2 * key & 4; }
    __device__ static constexpr int k(int key, int c) { return block(key / 8, c / 8) + key % 8 * 128 + (c % 8 ^ kswap(key)) * 16; }
    __device__ static constexpr int v(int key, int c) { return block(key / 8, c / 8) + key % 8 * 128 + (c % 8 ^ vswap(key)) * 16; }
};

// 16 bytes a lane from memory into LDS, past the registers: lane l's to dst + 16 l.  In assembly, since the
// compiler has every transposing load wait for such a load in flight, whatever tile it fills; landed() waits
// for a wave's own, and a barrier behind that for all.  (The compiler sets m0 right before what needs it and
// takes none of it over an assembly that says it writes it; that it warns of any such register is silenced here.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_to_lds(const void* src, lds_t dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"((unsigned)(uintptr_t)dst), "v"(src) : "memory", "m0");
}
#pragma clang diagnostic pop
__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0)" : : : "memory"); }

// LDS of a workgroup: two tiles of K, two of V, and their keys' factors (scores, values, values as they are
// stored); whether a wave met a value that is not finite where that matters.
template <int D>
struct Lds {
    static constexpr int kFactors = 4 * Tile<D>::kBytes;
    static constexpr int kFlags = kFactors + 6 * kTile * 4;
    static constexpr int kTotal = kFlags + kWaves * 4;
};

template <int FORMAT, int D>
__device__ __forceinline__ void attend(const AttentionKernelArgs& k, const Unit& u, lds_t lds) {
    constexpr bool kCodes = FORMAT != GDN_CACHE_PLAIN;
    constexpr int kRowBytes = D * (kCodes ? 1 : 2);
    // A load of a wave takes kRows keys of a tile, 128 bytes (or all) of each; a wave loads kGroups such groups of keys.
    constexpr int kChunks = kRowBytes < 128 ? kRowBytes / 16 : 8, kRows = 64 / kChunks, kPieces = kRowBytes / (16 * kChunks);
    constexpr int kGroups = kTile / kRows / kWaves;
    constexpr int kSteps = D / 16, kDims = D / 32;
    if (u.lo >= u.hi) {        // a table or a cache without rows: no address may be formed
        fill_rows<__bf16, D>(k, u, kRowsOfTile, kThreads, 0.f);
        return;
    }
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 31, half = lane >> 5, G = (int)k.group.d;
    const int H = k.a.cache.num_heads;
    const dev::Pages pages = {k.a.table + (int64_t)u.seq * k.a.table_width, k.a.table_width, k.block, k.a.cache.num_rows};
    const auto ktile = [&](int t) { return lds + (t & 1) * Tile<D>::kBytes; };
    const auto vtile = [&](int t) { return lds + (2 + (t & 1)) * Tile<D>::kBytes; };
    const auto kfactor = [&](int t) { return (lds_ptr<float>)(lds + Lds<D>::kFactors) + (t & 1) * kTile; };
    const auto vfactor = [&](int t) { return (lds_ptr<float>)(lds + Lds<D>::kFactors) + (2 + (t & 1)) * kTile; };
    const auto vstored = [&](int t) { return (lds_ptr<float>)(lds + Lds<D>::kFactors) + (4 + (t & 1)) * kTile; };
    const lds_ptr<int> flags = (lds_ptr<int>)(lds + Lds<D>::kFlags);
    const int tiles = (u.hi - u.lo + kTile - 1) / kTile;

    // ---- loads: a lane's key and its page's entry (in flight) two tiles ahead, values one
    int entry = -1, key = 0;
    const auto lookup = [&](int t) {
        key = u.lo + t * kTile + lane;
        entry = pages.entry(key);
    };
    u32x4_t kp[kGroups][kPieces], vp[kGroups][kPieces];
    float ks = 0.f, vs = 0.f;
    // Chunk `chunk` of a key's row in the cache; an absent key's values are those of row 0.
    const auto address = [&](const void* cache, int row, int chunk) {
        return static_cast<const char*>(cache) + (int64_t)u.h * kRowBytes + chunk * 16 + (uint64_t)(unsigned)(row < 0 ? 0 : row) * (unsigned)(H * kRowBytes);
    };
    const auto load_k = [&](int t, int row) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int group = wave * kGroups + g, at = lane % kChunks, n = group * kRows + lane / kChunks;
            const char* const from = address(k.a.cache.k, __shfl(row, n), kCodes ? at : at ^ Tile<D>::kswap(n));
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                if constexpr (kCodes) kp[g][i] = *reinterpret_cast<const u32x4_t*>(from + 128 * i);
                else load_to_lds(from + 128 * i, ktile(t) + Tile<D>::block(group, i));
            }
        }
        if constexpr (kCodes)
            if (wave == 0) {
                ks = row >= 0 ? k.a.cache.k_scale[(int64_t)row * H + u.h] : 0.f;
                vs = row >= 0 ? k.a.cache.v_scale[(int64_t)row * H + u.h] : 0.f;
            }
    };
    const auto load_v = [&](int t, int row) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const int group = wave * kGroups + g, at = lane % kChunks, n = group * kRows + lane / kChunks;
            const char* const from = address(k.a.cache.v, __shfl(row, n), kCodes ? at : at ^ Tile<D>::vswap(n));
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                if constexpr (kCodes) vp[g][i] = *reinterpret_cast<const u32x4_t*>(from + 128 * i);
                else load_to_lds(from + 128 * i, vtile(t) + Tile<D>::block(group, i));
            }
        }
    };
    lookup(0);

    // the scale's sign goes into the queries (exactly), so that the largest product is the largest score
    const float c = k.a.scale == 0.f ? 1.f : fabsf(k.a.scale) * kLog2e, sign = k.a.scale == 0.f ? 0.f : copysignf(1.f, k.a.scale);
    const int first_row = u.row0 + 32 * wave, r = first_row + col, token = (int)dev::divide(r, k.group);
    const bool live = r < u.rows;
    bf16x8_t q[kSteps] = {};
    dev::Sees sees = {0, 0, 0};
    if (live) {
        const __bf16* p = static_cast<const __bf16*>(k.a.q) + (u.first + token) * k.a.q_stride + (int64_t)(u.h * G + (r - token * G)) * D + half * 8;
#pragma unroll
        for (int x = 0; x < kSteps; ++x) q[x] = *reinterpret_cast<const bf16x8_t*>(p + 16 * x);
        if (sign != 1.f)
#pragma unroll
            for (int x = 0; x < kSteps; ++x)
#pragma unroll
                for (int i = 0; i < 8; ++i) q[x][i] = (__bf16)((float)q[x][i] * sign);
        sees = row_sees(k, u, r);
    }
    // every row of the workgroup (of the wave) sees the keys below `some` (`mine`), no row of the wave one from `end` on
    const bool tree = k.a.tree_mask != nullptr;
    const int some = tree ? u.past : causal_keys(k, u, u.row0);
    const int last_row = (first_row + 32 < u.rows ? first_row + 32 : u.rows) - 1;
    const int mine = tree ? u.past : causal_keys(k, u, first_row);
    const int end = first_row >= u.rows ? 0 : (tree ? u.hi : causal_keys(k, u, last_row));
    const auto works = [&](int t) { return t < tiles && u.lo + t * kTile < end; };
    // Whether keys of a tile are absent, or some rows of the workgroup do not see some.
    const auto special = [&](int t, uint64_t there) { return there != ~0ull || u.lo + (t + 1) * kTile > some; };

    // What was loaded, in LDS: codes as values.
    const auto land_k = [&](int t, uint64_t there) {
        if constexpr (kCodes) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        *(lds_ptr<bf16x8_t>)(ktile(t) + Tile<D>::k((wave * kGroups + g) * kRows + lane / kChunks, 16 * i + 2 * (lane % kChunks) + x)) =
                            dev::codes8<__bf16, FORMAT>(kp[g][i][2 * x], kp[g][i][2 * x + 1]);
            if (wave == 0) {
                kfactor(t)[lane] = ks * c;
                vfactor(t)[lane] = dev::finite(vs) ? vs : (special(t, there) ? 0.f : NAN);       // (an infinite scale is a NaN one)
                vstored(t)[lane] = vs;
            }
        }
    };
    const auto land_v = [&](int t) {
        if constexpr (kCodes) {
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int i = 0; i < kPieces; ++i)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        *(lds_ptr<bf16x8_t>)(vtile(t) + Tile<D>::v((wave * kGroups + g) * kRows + lane / kChunks, 16 * i + 2 * (lane % kChunks) + x)) =
                            dev::codes8<__bf16, FORMAT>(vp[g][i][2 * x], vp[g][i][2 * x + 1]);
        }
    };
    uint64_t there[2] = {0, 0};                    // which keys of tiles t and t + 1 are there, after issue(t)
    const auto issue = [&](int t) {                // the next tile, into the buffers of the one before
        const int next = t + 1 < tiles ? pages.row(key, entry, u.hi) : -1;
        there[0] = there[1];
        there[1] = __ballot(next >= 0);
        if (t + 1 < tiles) {
            load_k(t + 1, next);
            load_v(t + 1, next);
            lookup(t + 2);
        }
    };
    const auto land = [&](int t) {
        if (t + 1 < tiles) {
            land_k(t + 1, there[1]);
            land_v(t + 1);
        }
        if (!kCodes) landed();
    };

    // ---- a tile
    f32x16_t o[kDims] = {};
    float m = -INFINITY, l = 0.f;
    bf16x8_t w[4];
    // A head of 256 dims needs the accumulation registers for its sums: here they are said to be there.
    const auto accumulate = [&]() {
        if constexpr (D == 256)
#pragma unroll
            for (int d = 0; d < kDims; ++d) asm volatile("" : "+a"(o[d]));
    };
    f32x16_t s[2];
    const auto scores = [&](int t) {
        // chunk 2 x + half of key 32 b + col: fixed distances from the lane's first four
        lds_t kt[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) kt[x] = ktile(t) + Tile<D>::k(col, 2 * x + half);
        s[0] = f32x16_t{};
        s[1] = f32x16_t{};
#pragma unroll
        for (int x = 0; x < kSteps; ++x)
#pragma unroll
            for (int b = 0; b < 2; ++b) s[b] = mma32(*(lds_ptr<bf16x8_t>)(kt[x & 3] + Tile<D>::block(4 * b, x / 4)), q[x], s[b]);
    };
    // Masks, the running maximum, and the sums scaled where it rose.
    const auto maximum = [&](int t, uint64_t now) {
        const int p0 = u.lo + t * kTile;
        if constexpr (kCodes)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4_t by = *(lds_ptr<f32x4_t>)(kfactor(t) + 32 * b + 8 * i + 4 * half);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[b][4 * i + j] *= by[j];
                }
        if (now != ~0ull || p0 + kTile > mine) {
            const uint64_t seen = sees.from(p0) & now;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                const unsigned bits = (unsigned)(seen >> (32 * b)) >> (4 * half);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (!(bits >> (8 * (i / 4) + i % 4) & 1)) s[b][i] = -INFINITY;
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
        float x, y;
        dev::pair32(top, x, y);
        top = fmaxf(x, y);
        if constexpr (!kCodes) top *= c;
        // the maximum is kept until it is short by 2^8, which fp32 sums and bf16 weights take as well, so that the sums are
        // seldom scaled; each row goes by its own
        const float next = top > m + 8.f ? top : m;
        if (__any(next > m)) {
            const float keep = m == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m - next);      // (no sums yet)
            l *= keep;
            accumulate();
#pragma unroll
            for (int d = 0; d < kDims; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[d][i] *= keep;
            accumulate();
            m = next;
        }
    };
    const auto weights = [&](int t) {
        const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f32x4_t by = {1.f, 1.f, 1.f, 1.f};
                if constexpr (kCodes) by = *(lds_ptr<f32x4_t>)(vfactor(t) + 32 * b + 8 * i + 4 * half);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = __builtin_amdgcn_exp2f(kCodes ? s[b][4 * i + j] - base : fmaf(s[b][4 * i + j], c, -base));
                    if constexpr (kCodes) l += e;
                    w[2 * b + i / 2][4 * (i & 1) + j] = (__bf16)(e * by[j]);
                }
            }
        // The rounded weights' sum: a row's largest weight may be up to 2^8, not 1, and where it has nearly all of the sum its rounding
        // then cancels.  (With codes the weights carry the values' scales, and what they are rounded by is not the sum's.)
        if constexpr (!kCodes) {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int g = 0; g < 4; g += 2) {
                x = dev::sum8(w[g], x);
                y = dev::sum8(w[g + 1], y);
            }
            l += x + y;
        }
    };
    const auto sums = [&](int t) {
        // chunk 4 d + piece of four keys: fixed distances too, from one first for the even d and one for the odd
        const int vkey = 4 * half + lane % 16 / 4, piece = 2 * (lane >> 4 & 1) + (lane >> 1 & 1);
        const lds_t vt[2] = {vtile(t) + Tile<D>::v(vkey, piece) + (lane & 1) * 8, vtile(t) + Tile<D>::v(vkey, 4 + piece) + (lane & 1) * 8};
#pragma unroll
        for (int g = 0; g < 4; ++g)
#pragma unroll
            for (int d = 0; d < kDims; ++d) {
                const auto a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr<dev::s16x4_t>)(vt[d & 1] + Tile<D>::block(2 * g, d / 2)));
                const auto b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr<dev::s16x4_t>)(vt[d & 1] + Tile<D>::block(2 * g + 1, d / 2)));
                const dev::bf16x4_t x = __builtin_bit_cast(dev::bf16x4_t, a), y = __builtin_bit_cast(dev::bf16x4_t, b);
                o[d] = mma32(__builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7), w[g], o[d]);
            }
    };
    // Where keys are absent, or some rows do not see some, no value that is not finite may meet a weight of zero that stands for
    // that: absent keys' values are zeroed here, between the landing of the tile's V and its sums, where all waves come
    // together; whether others are left, for part().
    const auto inspect = [&](int t, uint64_t now) {
        if (!special(t, now)) return false;
        const lds_t vt = vtile(t);
        bool fine = true;
        for (int i = threadIdx.x; i < kTile * D / 8; i += kThreads) {
            const int n = i / D * 8 + i % 64 / 8;                 // chunks as they lie: D to eight keys
            const lds_ptr<bf16x8_t> at = (lds_ptr<bf16x8_t>)vt + i;
            if (now >> n & 1) {
                const bf16x8_t v = *at;
#pragma unroll
                for (int j = 0; j < 8; ++j) fine &= dev::finite((float)v[j]);
            } else {
                *at = bf16x8_t{};
            }
        }
        if (kCodes && threadIdx.x < kTile) fine &= dev::finite(vstored(t)[threadIdx.x]);
        const bool wrong = __any(!fine);
        if (lane == 0) flags[wave] = wrong;
        dev::lds_barrier();
        int bad = 0;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) bad |= flags[i];
        dev::lds_barrier();
        return __builtin_amdgcn_readfirstlane(bad) != 0;
    };
    // Values that are not finite, added to the rows that see them, and zeros in the product.  Plain ones (infinities among them) are
    // added times their weights, as the product would take them, which are formed here for themselves: the tile's own, in the
    // loop, then find the maximum where it has to be.  Codes and scales can only be NaN.
    const auto part = [&](int t, uint64_t now) {
        const lds_t vt = vtile(t);
        if (works(t)) {
            if constexpr (!kCodes) {
                scores(t);
                maximum(t, now);
                const float sum = l;
                weights(t);
                l = sum;
            }
            const uint64_t seen = sees.from(u.lo + t * kTile) & now;
            for (int n = 0; n < kTile; ++n) {
                if (!(now >> n & 1)) continue;
                float scale = 1.f, by = 1.f;                  // by: the row's weight, from the lane of its pair that holds the key
                if constexpr (kCodes) {
                    scale = vstored(t)[n];
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (n == 16 * (i / 8) + 8 * (i / 4 & 1) + 4 * half + i % 4) by = (float)w[i / 8][i % 8];
                    by = __shfl(by, 32 * (n >> 2 & 1) + col);
                }
#pragma unroll
                for (int d = 0; d < kDims; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int dim = 32 * d + 8 * (i / 4) + 4 * half + i % 4;
                        float v = (float)*(lds_ptr<__bf16>)(vt + Tile<D>::v(n, dim / 8) + dim % 8 * 2);
                        if (!dev::finite(scale)) v = NAN;
                        if (!dev::finite(v) && (seen >> n & 1)) o[d][i] += kCodes ? v : by * v;
                    }
            }
        }
        dev::lds_barrier();
        for (int i = threadIdx.x; i < kTile * D / 8; i += kThreads) {
            const lds_ptr<bf16x8_t> at = (lds_ptr<bf16x8_t>)vt + i;
            bf16x8_t v = *at;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (!dev::finite((float)v[j])) v[j] = (__bf16)0.f;
            *at = v;
        }
        dev::lds_barrier();
    };
    {
        const int row = pages.row(key, entry, u.hi);
        there[1] = __ballot(row >= 0);
        load_k(0, row);
        load_v(0, row);
        lookup(1);
    }
    // The compiler's own loads are waited for here: it does not see the waits in assembly, and would otherwise place its own
    // where the queries are first used, in the loop, for whatever is on its way there.
#pragma unroll
    for (int x = 0; x < kSteps; ++x) asm volatile("" : "+v"(q[x]));
    asm volatile("" : "+v"(sees.all), "+v"(sees.first), "+v"(sees.mask));
    land(-1);
    dev::lds_barrier();
    // (right behind the barrier, where no other tile's loads or scores are live, and marked as seldom: 4.87 ms for 8192 tokens of 256 dims in 8
    // bits, 5.1 to 9.1 in other places)
    if (__builtin_expect(inspect(0, there[1]), 0)) part(0, there[1]);
    for (int t = 0; t < tiles; ++t) {
        issue(t);
        if (works(t)) {
            scores(t);
            maximum(t, there[0]);
            weights(t);
            sums(t);
        }
        land(t);
        dev::lds_barrier();
        if (t + 1 < tiles && __builtin_expect(inspect(t + 1, there[1]), 0)) part(t + 1, there[1]);
    }

    float x, y;
    dev::pair32(l, x, y);
    l = x + y;
    if (!live) return;
    const int64_t at = (u.first + token) * k.a.H_q + u.h * G + (r - token * G);
    if (u.spans > 1) {
        float* const part = k.part + (at * k.spans + u.span) * D + 4 * half;
#pragma unroll
        for (int d = 0; d < kDims; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<f32x4_t*>(part + 32 * d + 8 * i) = f32x4_t{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
        if (half == 0) k.stats[at * k.spans + u.span] = {m, l};
        return;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __bf16* const out = static_cast<__bf16*>(k.a.o) + at * D + 4 * half;
#pragma unroll
    for (int d = 0; d < kDims; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dev::bf16x4_t v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = (__bf16)(o[d][4 * i + j] * inv);
            *reinterpret_cast<dev::bf16x4_t*>(out + 32 * d + 8 * i) = v;
        }
}

// Two workgroups to a compute unit; one where a head of 256 dims takes 512 registers and 128 KB of LDS.
template <int FORMAT, int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void wide_decode_kernel(AttentionKernelArgs k) {
    extern __shared__ __align__(16) char lds[];
    Unit u;
    if (decode_unit<__bf16, D>(k, kRowsOfTile, kThreads, u)) attend<FORMAT, D>(k, u, (lds_t)lds);
}

// Tiles from the last to the first: those with the most keys start first.
template <int FORMAT, int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void wide_prompt_kernel(AttentionKernelArgs k) {
    extern __shared__ __align__(16) char lds[];
    const unsigned H = (unsigned)k.a.cache.num_heads, at = blockIdx.x / H;
    Unit u;
    if (prompt_unit(k, kRowsOfTile, k.row_tiles - 1 - (int)at, (int)(blockIdx.x - at * H), u)) attend<FORMAT, D>(k, u, (lds_t)lds);
}

template <int FORMAT, int D>
hipError_t launch(AttentionKernelArgs k, hipStream_t stream) {
    const int H = k.a.cache.num_heads;
    const bool decode = k.a.tokens_per_row > 0;
    const int64_t tiles = decode ? (k.a.tokens_per_row * (int)k.group.d + kRowsOfTile - 1) / kRowsOfTile : k.a.total_tokens * (int)k.group.d / kRowsOfTile + k.a.num_seqs;
    const int64_t units = decode ? ((int64_t)k.a.num_seqs * k.spans * H + 7) / 8 * 8 : H;
    if (!grid_fits(tiles * units, kThreads) || k.a.total_tokens * (int64_t)k.group.d > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    k.row_tiles = (int)tiles;
    auto* const kernel = decode ? wide_decode_kernel<FORMAT, D> : wide_prompt_kernel<FORMAT, D>;
    kernel<<<(unsigned)(tiles * units), kThreads, Lds<D>::kTotal, stream>>>(k);
    return hipGetLastError();
}

template <int FORMAT>
hipError_t launch(const AttentionKernelArgs& k, hipStream_t stream) {
    if (k.a.cache.head_dim == 64) return launch<FORMAT, 64>(k, stream);
    if (k.a.cache.head_dim == 128) return launch<FORMAT, 128>(k, stream);
    return launch<FORMAT, 256>(k, stream);
}

}  // namespace

hipError_t launch_attention_wide(const AttentionKernelArgs& k, hipStream_t stream) {
    if (k.a.cache.format == GDN_CACHE_PLAIN) return launch<GDN_CACHE_PLAIN>(k, stream);
    if (k.a.cache.format == GDN_CACHE_E4M3) return launch<GDN_CACHE_E4M3>(k, stream);
    return launch<GDN_CACHE_INT8>(k, stream);
}

}  // namespace gdn
