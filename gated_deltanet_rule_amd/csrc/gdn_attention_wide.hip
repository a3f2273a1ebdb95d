// gdn_attention_wide.hip -- attention of many query rows over a paged cache for gfx950: bf16
// prompts, and decode rows with large trees.
//
// The same sums as gdn_attention.hip, for rows enough to share the keys: four waves of 32 rows
// take the same tile of 64 keys from LDS, two tiles of which stand there in turn: while one is
// worked on, the next is loaded into registers and widened, if it holds codes, on its way into
// the other.  The products are transposed here too, 32 x 32 tiles with a query row to each pair of
// lanes, so that weights are the second product's operand as they come out of the first.
#include <hip/hip_runtime.h>

#include "gdn_attention_device.h"
#include "gdn_layer_internal.h"

namespace gdn {
namespace {

using dev::bf16x8_t;
using dev::f32x4_t;
using dev::f32x16_t;
using dev::u32x4_t;

constexpr int kThreads = 256, kWaves = 4, kTile = 64, kRows = 128;

__device__ __forceinline__ f32x16_t mma32(bf16x8_t a, bf16x8_t b, f32x16_t acc) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0); }

// Tiles of bf16 values in LDS: blocks of 16 keys by 32 dims, 1 KB each, which one load of a wave fills (16 bytes a
// lane, in lanes' order).  K's operands take one 16-byte chunk of 16 keys at a time: a block of K holds chunk after
// chunk.  V's transposing loads take 64 bytes of four keys at a time: a block of V holds key after key.  Neither
// meets itself in a bank, and all of a tile's operands stand at fixed distances from a lane's first.
template <int D>
struct Tile {
    static constexpr int kBytes = kTile * D * 2;
    __device__ static constexpr int block(int key16, int dim32) { return (key16 * (D / 32) + dim32) * 1024; }
    // chunk c (eight dims) of a key
    __device__ static constexpr int k(int key, int c) { return block(key / 16, c / 4) + c % 4 * 256 + key % 16 * 16; }
    __device__ static constexpr int v(int key, int c) { return block(key / 16, c / 4) + key % 16 * 64 + c % 4 * 16; }
};

// 16 bytes a lane from memory into LDS, past the registers: lane l's to dst + 16 l.  In assembly, since the
// compiler has every transposing load wait for such a load in flight, whatever tile it fills; landed() waits
// for a wave's own, and a barrier behind that for all.  (m0 holds nothing between instructions: whatever needs it
// sets it.)
__device__ __forceinline__ void load_to_lds(const void* src, char* dst) {
    const unsigned to = __builtin_amdgcn_readfirstlane((unsigned)(uintptr_t)(__attribute__((address_space(3))) char*)dst);
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(to), "v"(src) : "memory");
}
__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0)" : : : "memory"); }

// LDS of a workgroup: two tiles each of K and V; for each, the keys' factors (score, value); whether a wave met a
// value that is not finite where that matters.
template <int D>
struct Lds {
    static constexpr int kTiles = 4 * Tile<D>::kBytes;
    static constexpr int kFactors = 2 * 2 * kTile * 4;
    static constexpr int kTotal = kTiles + kFactors + kWaves * 4;
};

template <int FORMAT, int D>
__device__ __forceinline__ void attend(const AttentionKernelArgs& k, const Unit& u, char* lds) {
    constexpr bool kCodes = FORMAT != GDN_CACHE_PLAIN;
    constexpr int kRowBytes = D * (kCodes ? 1 : 2), kPieces = kRowBytes / 64;      // 64 bytes of 16 keys to a load of a wave
    constexpr int kSteps = D / 16, kDims = D / 32;
    if (u.lo >= u.hi) {        // a table or a cache without rows: no address may be formed
        fill_rows<__bf16, D>(k, u, kRows, kThreads, 0.f);
        return;
    }
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 31, half = lane >> 5, G = (int)k.group.d;
    const int H = k.a.cache.num_heads;
    const dev::Pages pages = {k.a.table + (int64_t)u.seq * k.a.table_width, k.a.table_width, k.block, k.a.cache.num_rows};
    float* const factors = reinterpret_cast<float*>(lds + Lds<D>::kTiles);
    int* const flags = reinterpret_cast<int*>(lds + Lds<D>::kTiles + Lds<D>::kFactors);
    // the scale's sign goes into the queries (exactly), so that the largest product is the largest score
    const float c = k.a.scale == 0.f ? 1.f : fabsf(k.a.scale) * kLog2e, sign = k.a.scale == 0.f ? 0.f : copysignf(1.f, k.a.scale);

    const int r = u.row0 + 32 * wave + col, t = (int)dev::divide(r, k.group);
    const bool live = r < u.rows;
    const bool busy = u.row0 + 32 * wave < u.rows;       // whether the wave has any rows
    bf16x8_t q[kSteps] = {};
    dev::Sees sees = {0, 0, 0};
    if (live) {
        const __bf16* p = static_cast<const __bf16*>(k.a.q) + (u.first + t) * k.a.q_stride + (int64_t)(u.h * G + (r - t * G)) * D + half * 8;
#pragma unroll
        for (int s = 0; s < kSteps; ++s) q[s] = *reinterpret_cast<const bf16x8_t*>(p + 16 * s);
        if (sign != 1.f)
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int i = 0; i < 8; ++i) q[s][i] = (__bf16)((float)q[s][i] * sign);
        sees = row_sees(k, u, r);
    }
    // every row of the workgroup (of the wave) sees the keys below `some` (`mine`), no row of the wave one from `end` on
    const bool tree = k.a.tree_mask != nullptr;
    const int some = tree ? u.past : u.past + (int)dev::divide(u.row0, k.group) + 1;
    const int first_row = u.row0 + 32 * wave, last_row = (first_row + 32 < u.rows ? first_row + 32 : u.rows) - 1;
    const int mine = tree ? u.past : u.past + (int)dev::divide(first_row, k.group) + 1;
    const int end = !busy ? 0 : (tree ? u.hi : u.past + (int)dev::divide(last_row, k.group) + 1);

    f32x16_t o[kDims] = {};
    float m = -INFINITY, l = 0.f;

    // ---- one tile ahead: the keys' rows, then what they hold.  A wave loads 16 of the tile's keys.
    int entry = -1, key = 0;            // a lane's key two tiles ahead: its page's entry, in flight, and itself
    const auto lookup = [&](int p0) {
        key = p0 + lane;
        const unsigned page = dev::divide((unsigned)key, k.block);
        entry = pages.table[page < (unsigned)pages.width ? page : (unsigned)pages.width - 1];
    };
    const auto row_of = [&]() {
        const unsigned page = dev::divide((unsigned)key, k.block);
        const int64_t row = (int64_t)entry * k.block.d + ((unsigned)key - page * k.block.d);
        return key < u.hi && page < (unsigned)pages.width && entry >= 0 && row < pages.num_rows ? (int)row : -1;
    };
    u32x4_t kp[kCodes ? kPieces : 1], vp[kCodes ? kPieces : 1];
    float ks = 0.f, vs = 0.f;
    // Plain values go into `buf` directly, codes into registers.  An absent key's are those of row 0.
    const auto load = [&](int row, int buf) {
        const int krow = __shfl(row, 16 * wave + lane % 16), vrow = __shfl(row, 16 * wave + lane / 4);
        const char* const kc = static_cast<const char*>(k.a.cache.k) + (int64_t)u.h * kRowBytes + lane / 16 * 16 + (uint64_t)(unsigned)(krow < 0 ? 0 : krow) * (unsigned)(H * kRowBytes);
        const char* const vc = static_cast<const char*>(k.a.cache.v) + (int64_t)u.h * kRowBytes + lane % 4 * 16 + (uint64_t)(unsigned)(vrow < 0 ? 0 : vrow) * (unsigned)(H * kRowBytes);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            if constexpr (kCodes) {
                kp[i] = *reinterpret_cast<const u32x4_t*>(kc + 64 * i);
                vp[i] = *reinterpret_cast<const u32x4_t*>(vc + 64 * i);
            } else {
                char* const to = lds + buf * 2 * Tile<D>::kBytes + Tile<D>::block(wave, i);
                load_to_lds(kc + 64 * i, to);
                load_to_lds(vc + 64 * i, to + Tile<D>::kBytes);
            }
        }
        if constexpr (kCodes) {
            ks = row >= 0 ? k.a.cache.k_scale[(int64_t)row * H + u.h] : 0.f;
            vs = row >= 0 ? k.a.cache.v_scale[(int64_t)row * H + u.h] : 0.f;
        }
    };
    // Codes as values into the tiles of `buf`.
    const auto store = [&](int buf) {
        if constexpr (kCodes) {
            char* const kt = lds + buf * 2 * Tile<D>::kBytes;
            char* const vt = kt + Tile<D>::kBytes;
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int kchunk = 2 * (4 * i + lane / 16) + x, vchunk = 2 * (4 * i + lane % 4) + x;
                    *reinterpret_cast<bf16x8_t*>(kt + Tile<D>::k(16 * wave + lane % 16, kchunk)) = dev::codes8<__bf16, FORMAT>(kp[i][2 * x], kp[i][2 * x + 1]);
                    *reinterpret_cast<bf16x8_t*>(vt + Tile<D>::v(16 * wave + lane / 4, vchunk)) = dev::codes8<__bf16, FORMAT>(vp[i][2 * x], vp[i][2 * x + 1]);
                }
            if (wave == 0) {
                factors[buf * 2 * kTile + lane] = ks * c;
                factors[buf * 2 * kTile + kTile + lane] = vs;
            }
        }
    };

    lookup(u.lo);
    int row = row_of();
    uint64_t present = __ballot(row >= 0);
    load(row, 0);
    lookup(u.lo + kTile);
    store(0);
    if (!kCodes) landed();
    __syncthreads();

    int buf = 0;
    for (int p0 = u.lo; p0 < u.hi; p0 += kTile, buf ^= 1) {
        const bool more = p0 + kTile < u.hi;
        const uint64_t now = present;
        if (more) {
            row = row_of();
            present = __ballot(row >= 0);
            load(row, buf ^ 1);
            lookup(p0 + 2 * kTile);
        }
        char* const kt = lds + buf * 2 * Tile<D>::kBytes;
        char* const vt = kt + Tile<D>::kBytes;
        float* const factor = factors + buf * 2 * kTile;
        const bool work = p0 < end;
        const bool partial = now != ~0ull || p0 + kTile > mine;
        f32x16_t s[2] = {};
        uint64_t seen = ~0ull;
        if (work) {
#pragma unroll
            for (int x = 0; x < kSteps; ++x)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const bf16x8_t kf = *reinterpret_cast<const bf16x8_t*>(kt + Tile<D>::k(32 * b + col, 2 * x + half));
                    s[b] = mma32(kf, q[x], s[b]);
                }
            if constexpr (kCodes)
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const f32x4_t by = *reinterpret_cast<const f32x4_t*>(factor + 32 * b + 8 * i + 4 * half);
#pragma unroll
                        for (int j = 0; j < 4; ++j) s[b][4 * i + j] *= by[j];
                    }
            if (partial) {
                seen = sees.from(p0) & now;
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
                const float keep = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - next);
                l *= keep;
#pragma unroll
                for (int d = 0; d < kDims; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[d][i] *= keep;
                m = next;
            }
        }
        // Where keys are absent, or some rows do not see some, no value that is not finite may meet a weight of zero:
        // absent keys' values are zeroed; others are added to the rows that see them, and are zeros in the product.
        if (now != ~0ull || p0 + kTile > some) {
            constexpr int kChunks = kTile * D / 8;
            bool fine = true;
            for (int i = threadIdx.x; i < kChunks; i += kThreads) {
                const int n = i / (D * 2) * 16 + i % 64 / 4;          // chunks as they lie
                bf16x8_t* const at = reinterpret_cast<bf16x8_t*>(vt) + i;
                if (now >> n & 1) {
                    const bf16x8_t v = *at;
#pragma unroll
                    for (int j = 0; j < 8; ++j) fine &= dev::finite((float)v[j]);
                } else {
                    *at = bf16x8_t{};
                }
            }
            if (kCodes && threadIdx.x < kTile) fine &= dev::finite(factor[kTile + threadIdx.x]);
            const bool wrong = __any(!fine);
            if (lane == 0) flags[wave] = wrong;
            __syncthreads();
            int bad = 0;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) bad |= flags[w];
            if (bad) {
                if (work) {
                    for (int n = 0; n < kTile; ++n) {
                        if (!(now >> n & 1)) continue;
                        float by = 1.f;
                        if constexpr (kCodes) by = factor[kTile + n];
#pragma unroll
                        for (int d = 0; d < kDims; ++d)
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int dim = 32 * d + 8 * (i / 4) + 4 * half + i % 4;
                                float v = (float)*reinterpret_cast<const __bf16*>(vt + Tile<D>::v(n, dim / 8) + dim % 8 * 2);
                                if (!dev::finite(by)) v = NAN;
                                if (!dev::finite(v) && (seen >> n & 1)) o[d][i] += v;
                            }
                    }
                }
                __syncthreads();
                for (int i = threadIdx.x; i < kChunks; i += kThreads) {
                    bf16x8_t* const at = reinterpret_cast<bf16x8_t*>(vt) + i;
                    bf16x8_t v = *at;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (!dev::finite((float)v[j])) v[j] = (__bf16)0.f;
                    *at = v;
                }
                if (kCodes && threadIdx.x < kTile && !dev::finite(factor[kTile + threadIdx.x])) factor[kTile + threadIdx.x] = 0.f;
                __syncthreads();
            }
        }
        if (work) {
            const float base = m == -INFINITY ? 0.f : m;
            bf16x8_t w[4];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x4_t by = {1.f, 1.f, 1.f, 1.f};
                    if constexpr (kCodes) by = *reinterpret_cast<const f32x4_t*>(factor + kTile + 32 * b + 8 * i + 4 * half);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = __builtin_amdgcn_exp2f(kCodes ? s[b][4 * i + j] - base : fmaf(s[b][4 * i + j], c, -base));
                        l += x;
                        w[2 * b + i / 2][4 * (i & 1) + j] = (__bf16)(x * by[j]);
                    }
                }
            typedef __attribute__((address_space(3))) dev::s16x4_t* lds_ptr;
            const int vkey = 4 * half + lane % 16 / 4, piece = 2 * (lane >> 4 & 1) + (lane >> 1 & 1);
#pragma unroll
            for (int d = 0; d < kDims; ++d)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const auto a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(vt + Tile<D>::v(16 * g + vkey, 4 * d + piece) + (lane & 1) * 8));
                    const auto b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(vt + Tile<D>::v(16 * g + 8 + vkey, 4 * d + piece) + (lane & 1) * 8));
                    const dev::bf16x4_t x = __builtin_bit_cast(dev::bf16x4_t, a), y = __builtin_bit_cast(dev::bf16x4_t, b);
                    o[d] = mma32(__builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7), w[g], o[d]);
                }
        }
        if (more) store(buf ^ 1);
        if (!kCodes) landed();
        __syncthreads();
    }

    float x, y;
    dev::pair32(l, x, y);
    l = x + y;
    if (!live) return;
    const int64_t at = (u.first + t) * k.a.H_q + u.h * G + (r - t * G);
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

template <int FORMAT, int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void wide_decode_kernel(AttentionKernelArgs k) {
    extern __shared__ __align__(16) char lds[];
    Unit u;
    if (decode_unit<__bf16, D>(k, kRows, kThreads, u)) attend<FORMAT, D>(k, u, lds);
}

// Tiles from the last to the first: those with the most keys start first.
template <int FORMAT, int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void wide_prompt_kernel(AttentionKernelArgs k) {
    extern __shared__ __align__(16) char lds[];
    const unsigned H = (unsigned)k.a.cache.num_heads, at = blockIdx.x / H;
    Unit u;
    if (prompt_unit(k, kRows, k.row_tiles - 1 - (int)at, (int)(blockIdx.x - at * H), u)) attend<FORMAT, D>(k, u, lds);
}

template <int FORMAT, int D>
hipError_t launch(AttentionKernelArgs k, hipStream_t stream) {
    const int H = k.a.cache.num_heads;
    const bool decode = k.a.tokens_per_row > 0;
    const int64_t tiles = decode ? (k.a.tokens_per_row * (int)k.group.d + kRows - 1) / kRows : k.a.total_tokens * (int)k.group.d / kRows + k.a.num_seqs;
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
