// gdn_attention_wide.hip -- attention of many query rows over a paged cache for gfx950: bf16
// prompts, and decode rows with large trees.
//
// The same sums as gdn_attention.hip, for rows enough to share the keys: waves of 32 rows each take
// the same tiles of keys from LDS.  The products are transposed here too, 32 x 32 tiles with a
// query row to each pair of lanes, so that weights are the second product's operand as they
// come out of the first.
//
// Everything comes from memory into LDS past the registers, three tiles ahead: the pages' entries, then K
// and V.  That is what it takes: the waves of all workgroups that share keys run along them together, so
// every tile is new to the cache when the first of them asks for it, and a tile is worked off in less
// time than memory takes to answer.  Codes wait in LDS as they are stored, each wave's own, and become
// bf16 tiles just before they are needed.
//
// A tile is two phases to a wave: matrix products (the weights of the tile before times V, then K
// times the queries) and the softmax, which keeps the vector ALU as long as the products keep the
// matrix cores.  In a workgroup of eight waves the second four run one phase behind the first: each
// SIMD holds a wave of either, and one's products run beside the other's softmax.
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

// Keys of a tile: where LDS has to hold two workgroups, or heads of 256 dims, half of them.
template <int WAVES>
constexpr int kKeys = WAVES == 8 ? 64 : 32;

__device__ __forceinline__ f32x16_t mma32(bf16x8_t a, bf16x8_t b, f32x16_t acc) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0); }

template <typename V>
using lds_ptr = __attribute__((address_space(3))) V*;
typedef lds_ptr<char> lds_t;

// Tiles of bf16 values in LDS: blocks of 8 keys by 64 dims, 1 KB each, key after key, which one load of a wave fills (16
// bytes a lane, in lanes' order) from 128 bytes of each key: four neighbouring lanes have to stand in the same 64 bytes of
// memory, or a load takes the memory path up to four times as long.  The 16-byte chunks of a key are exchanged: K's operands
// take one chunk of 16 keys at a time, V's transposing loads 64 bytes of four, and neither meets itself in a bank.
template <int D>
struct Tile {
    __device__ static constexpr int block(int key8, int dim64) { return (key8 * (D / 64) + dim64) * 1024; }
    // where chunk c (eight dims) of a key stands
    __device__ static constexpr int kswap(int key) { return key >> 1 & 7; }
    __device__ static constexpr int vswap(int key) { return 2 * key & 4; }
    __device__ static constexpr int k(int key, int c) { return block(key / 8, c / 8) + key % 8 * 128 + (c % 8 ^ kswap(key)) * 16; }
    __device__ static constexpr int v(int key, int c) { return block(key / 8, c / 8) + key % 8 * 128 + (c % 8 ^ vswap(key)) * 16; }
};

// From memory into LDS, past the registers: lane l's 16 (4) bytes to dst + 16 l (4 l).  In assembly, since the compiler
// has every transposing load wait for all such loads in flight.  landed<N>() waits for a wave's own but the last N, and
// a barrier behind that for all.  (m0 holds nothing between instructions: whatever needs it sets it.)
__device__ __forceinline__ void load_to_lds(const void* src, lds_t dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"((unsigned)(uintptr_t)dst), "v"(src) : "memory");
}
__device__ __forceinline__ void load_word_to_lds(const void* src, lds_t dst) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" : : "s"((unsigned)(uintptr_t)dst), "v"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void landed() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "i"(N) : "memory");
}

// How a workgroup's waves load a tile.  A load of a wave takes kRows keys, 128 bytes (or all) of each.  Every wave takes
// kRows keys of K and of V, or, where a load takes twice as many, the first half of the waves K and the others V.
template <int FORMAT, int D, int WAVES>
struct Plan {
    static constexpr bool kCodes = FORMAT != GDN_CACHE_PLAIN;
    static constexpr int kTile = kKeys<WAVES>;
    static constexpr int kRowBytes = D * (kCodes ? 1 : 2);
    static constexpr int kChunks = kRowBytes < 128 ? kRowBytes / 16 : 8, kRows = 64 / kChunks, kPieces = kRowBytes / (16 * kChunks);
    static constexpr bool kSplit = kTile / kRows < WAVES;
    static_assert(kTile / kRows == (kSplit ? WAVES / 2 : WAVES), "one group of keys to a wave");
    static constexpr int kLoads = kPieces * (kSplit ? 1 : 2) + 1;      // a wave's, a tile; wave 0 of codes loads two scales more
    // LDS: tiles of K, of V; codes on their way; the waves' page entries; scales on their way, factors of the keys (scores,
    // values, values as they are stored); whether a wave met a value that is not finite where that matters
    static constexpr int kRing = kCodes ? 2 : 4, kWaiting = 3, kEntries = 4;
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kV = kRing * kTileBytes, kRaw = 2 * kV, kRawWave = kPieces * 1024 * 2;
    static constexpr int kEntry = kRaw + (kCodes ? kWaiting * WAVES * kRawWave : 0);
    static constexpr int kScales = kEntry + WAVES * kEntries * 256, kFactors = kScales + (kCodes ? kWaiting * 2 * 256 : 0);
    static constexpr int kFlags = kFactors + (kCodes ? 6 * kTile * 4 : 0), kTotal = kFlags + WAVES * 4;
    static_assert(kTotal <= 160 * 1024, "LDS of a compute unit");
};

template <int FORMAT, int D, int WAVES>
__device__ __forceinline__ void attend(const AttentionKernelArgs& k, const Unit& u, lds_t lds) {
    using P = Plan<FORMAT, D, WAVES>;
    constexpr bool kCodes = P::kCodes, kPair = WAVES == 8;
    constexpr int kThreads = 64 * WAVES, kTile = P::kTile, kBlocks = kTile / 32, kRows = P::kRows, kChunks = P::kChunks, kPieces = P::kPieces;
    constexpr int kSteps = D / 16, kDims = D / 32;
    constexpr uint64_t kAll = ~0ull >> (64 - kTile);
    if (u.lo >= u.hi) {        // a table or a cache without rows: no address may be formed
        fill_rows<__bf16, D>(k, u, 32 * WAVES, kThreads, 0.f);
        return;
    }
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), col = lane & 31, half = lane >> 5, G = (int)k.group.d;
    const int H = k.a.cache.num_heads;
    const int32_t* const table = k.a.table + (int64_t)u.seq * k.a.table_width;
    // tile numbers from -3 on; 12 is a multiple of every ring's length
    const auto ktile = [&](int t) { return lds + (unsigned)(t + 12) % P::kRing * P::kTileBytes; };
    const auto vtile = [&](int t) { return lds + P::kV + (unsigned)(t + 12) % P::kRing * P::kTileBytes; };
    const auto raw = [&](int t) { return lds + P::kRaw + ((unsigned)(t + 12) % P::kWaiting * WAVES + wave) * P::kRawWave; };
    const auto entries = [&](int t) { return lds + P::kEntry + (wave * P::kEntries + (unsigned)(t + 12) % P::kEntries) * 256; };
    const auto scales = [&](int t) { return lds + P::kScales + (unsigned)(t + 12) % P::kWaiting * 512; };
    const auto kfactor = [&](int t) { return (lds_ptr<float>)(lds + P::kFactors) + (t & 1) * kTile; };
    const auto vfactor = [&](int t) { return (lds_ptr<float>)(lds + P::kFactors) + (2 + (t & 1)) * kTile; };
    const auto vstored = [&](int t) { return (lds_ptr<float>)(lds + P::kFactors) + (4 + (t & 1)) * kTile; };
    const lds_ptr<int> flags = (lds_ptr<int>)(lds + P::kFlags);
    // the scale's sign goes into the queries (exactly), so that the largest product is the largest score
    const float c = k.a.scale == 0.f ? 1.f : fabsf(k.a.scale) * kLog2e, sign = k.a.scale == 0.f ? 0.f : copysignf(1.f, k.a.scale);

    const auto load_entries = [&](int t) {
        const unsigned page = dev::divide((unsigned)(u.lo + t * kTile + lane), k.block);
        load_word_to_lds(table + (page < (unsigned)k.a.table_width ? page : (unsigned)k.a.table_width - 1), entries(t));
    };
    for (int t = 0; t < 4; ++t) load_entries(t);

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
    // The compiler's own loads are waited for here: it does not see the waits in assembly below, and would otherwise place its
    // own where the queries are first used, in the loop, for whatever is on its way there.
#pragma unroll
    for (int x = 0; x < kSteps; ++x) asm volatile("" : "+v"(q[x]));
    asm volatile("" : "+v"(sees.all), "+v"(sees.first), "+v"(sees.mask));
    // every row of the workgroup (of the wave) sees the keys below `some` (`mine`), no row of the wave one from `end` on
    const bool tree = k.a.tree_mask != nullptr;
    const int some = tree ? u.past : u.past + (int)dev::divide(u.row0, k.group) + 1;
    const int first_row = u.row0 + 32 * wave, last_row = (first_row + 32 < u.rows ? first_row + 32 : u.rows) - 1;
    const int mine = tree ? u.past : u.past + (int)dev::divide(first_row, k.group) + 1;
    const int end = !busy ? 0 : (tree ? u.hi : u.past + (int)dev::divide(last_row, k.group) + 1);

    const bool behind = kPair && wave >= 4;       // one phase behind the others
    const int tiles = (u.hi - u.lo + kTile - 1) / kTile;

    f32x16_t o[kDims] = {};
    float m = -INFINITY, l = 0.f;

    // ---- loads
    const bool loads_k = !P::kSplit || wave < WAVES / 2, loads_v = !P::kSplit || wave >= WAVES / 2;
    const int group = P::kSplit ? wave % (WAVES / 2) : wave;      // of kRows keys
    // Chunk `chunk` of a key's row in the cache; an absent key's values are those of row 0.
    const auto address = [&](const void* cache, int row, int chunk) {
        return static_cast<const char*>(cache) + (int64_t)u.h * P::kRowBytes + chunk * 16 + (uint64_t)(unsigned)(row < 0 ? 0 : row) * (unsigned)(H * P::kRowBytes);
    };
    const auto row_of = [&](int t) {      // the cache row of the lane's key of tile t, or -1
        const int key = u.lo + t * kTile + lane, entry = ((lds_ptr<int>)entries(t))[lane];
        const unsigned page = dev::divide((unsigned)key, k.block);
        const int64_t at = (int64_t)entry * k.block.d + ((unsigned)key - page * k.block.d);
        return (kTile == 64 || lane < kTile) && key < u.hi && page < (unsigned)k.a.table_width && entry >= 0 && at < k.a.cache.num_rows ? (int)at : -1;
    };
    // What is issued with tile t: the entries seven tiles ahead, K (and the scales) three, V two.  Where they come from is worked out
    // one issue earlier (prepare(t)), in the shadow of the loads before.
    int next = -1;                          // the cache row of the lane's key of tile t + 3, from prepare(t) on
    uint64_t there[5] = {0, 0, 0, 0, 0};    // which keys of tiles t .. t + 4 are there, after issue(t)
    const char *kfrom = nullptr, *vfrom = nullptr;
    const int chunk = lane % kChunks, mykey = group * kRows + lane / kChunks;
    const auto prepare = [&](int t) {
        if (loads_v) vfrom = address(k.a.cache.v, __shfl(next, mykey), kCodes ? chunk : chunk ^ Tile<D>::vswap(mykey));
        next = row_of(t + 3);
        there[4] = __ballot(next >= 0);
        if (loads_k) kfrom = address(k.a.cache.k, __shfl(next, mykey), kCodes ? chunk : chunk ^ Tile<D>::kswap(mykey));
    };
    const auto issue = [&](int t) {
        there[0] = there[1];
        there[1] = there[2];
        there[2] = there[3];
        there[3] = there[4];
        if (loads_v)
#pragma unroll
            for (int i = 0; i < kPieces; ++i) load_to_lds(vfrom + 128 * i, kCodes ? raw(t + 2) + (kPieces + i) * 1024 : vtile(t + 2) + Tile<D>::block(group, i));
        if (loads_k)
#pragma unroll
            for (int i = 0; i < kPieces; ++i) load_to_lds(kfrom + 128 * i, kCodes ? raw(t + 3) + i * 1024 : ktile(t + 3) + Tile<D>::block(group, i));
        if (kCodes && wave == 0) {
            const int64_t head = (int64_t)(next < 0 ? 0 : next) * H + u.h;
            load_word_to_lds(k.a.cache.k_scale + head, scales(t + 3));
            load_word_to_lds(k.a.cache.v_scale + head, scales(t + 3) + 256);
        }
        load_entries(t + 7);
        prepare(t + 1);
    };
    // Whether keys of a tile are absent, or some rows of the workgroup do not see some.
    const auto special = [&](int t, uint64_t now) { return now != kAll || u.lo + (t + 1) * kTile > some; };
    // K of the next tile and V of tile t (the loads of issue(t - 2)) are there; codes as values.
    const auto land = [&](int t) {
        if (kCodes && wave == 0) landed<2 * (P::kLoads + 2)>();
        else landed<2 * P::kLoads>();
        if constexpr (kCodes) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                if (loads_k) {
                    const u32x4_t w = *(lds_ptr<u32x4_t>)(raw(t + 1) + i * 1024 + lane * 16);
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        *(lds_ptr<bf16x8_t>)(ktile(t + 1) + Tile<D>::k(group * kRows + lane / kChunks, 16 * i + 2 * (lane % kChunks) + x)) =
                            dev::codes8<__bf16, FORMAT>(w[2 * x], w[2 * x + 1]);
                }
                if (loads_v) {
                    const u32x4_t w = *(lds_ptr<u32x4_t>)(raw(t) + (kPieces + i) * 1024 + lane * 16);
#pragma unroll
                    for (int x = 0; x < 2; ++x)
                        *(lds_ptr<bf16x8_t>)(vtile(t) + Tile<D>::v(group * kRows + lane / kChunks, 16 * i + 2 * (lane % kChunks) + x)) =
                            dev::codes8<__bf16, FORMAT>(w[2 * x], w[2 * x + 1]);
                }
            }
            if (wave == 0 && (kTile == 64 || lane < kTile)) {
                const float ks = ((lds_ptr<float>)scales(t + 1))[lane], vs = ((lds_ptr<float>)(scales(t + 1) + 256))[lane];
                const bool here = there[1] >> lane & 1;
                kfactor(t + 1)[lane] = here ? ks * c : 0.f;
                vfactor(t + 1)[lane] = !here || (special(t + 1, there[1]) && !dev::finite(vs)) ? 0.f : vs;
                vstored(t + 1)[lane] = here ? vs : 0.f;
            }
        }
    };

    // ---- the phases of a tile
    f32x16_t s[kBlocks];
    bf16x8_t w[2 * kBlocks];
    const auto scores = [&](int t) {
        // chunk 2 x + half of key 32 b + col: fixed distances from the lane's first four
        lds_t kt[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) kt[x] = ktile(t) + Tile<D>::k(col, 2 * x + half);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) s[b] = f32x16_t{};
#pragma unroll
        for (int x = 0; x < kSteps; ++x)
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) s[b] = mma32(*(lds_ptr<bf16x8_t>)(kt[x & 3] + Tile<D>::block(4 * b, x / 4)), q[x], s[b]);
    };
    const auto softmax = [&](int t, uint64_t now) {
        const int p0 = u.lo + t * kTile;
        if constexpr (kCodes)
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4_t by = *(lds_ptr<f32x4_t>)(kfactor(t) + 32 * b + 8 * i + 4 * half);
#pragma unroll
                    for (int j = 0; j < 4; ++j) s[b][4 * i + j] *= by[j];
                }
        if (now != kAll || p0 + kTile > mine) {
            const uint64_t seen = sees.from(p0) & now;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const unsigned bits = (unsigned)(seen >> (32 * b)) >> (4 * half);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (!(bits >> (8 * (i / 4) + i % 4) & 1)) s[b][i] = -INFINITY;
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
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
#pragma unroll
            for (int d = 0; d < kDims; ++d)
#pragma unroll
                for (int i = 0; i < 16; ++i) o[d][i] *= keep;
            m = next;
        }
        const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f32x4_t by = {1.f, 1.f, 1.f, 1.f};
                if constexpr (kCodes) by = *(lds_ptr<f32x4_t>)(vfactor(t) + 32 * b + 8 * i + 4 * half);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = __builtin_amdgcn_exp2f(kCodes ? s[b][4 * i + j] - base : fmaf(s[b][4 * i + j], c, -base));
                    l += e;
                    w[2 * b + i / 2][4 * (i & 1) + j] = (__bf16)(e * by[j]);
                }
            }
    };
    const auto sums = [&](int t) {
        // chunk 4 d + piece of four keys: fixed distances too, from one first for the even d and one for the odd
        const int vkey = 4 * half + lane % 16 / 4, piece = 2 * (lane >> 4 & 1) + (lane >> 1 & 1);
        const lds_t vt[2] = {vtile(t) + Tile<D>::v(vkey, piece) + (lane & 1) * 8, vtile(t) + Tile<D>::v(vkey, 4 + piece) + (lane & 1) * 8};
#pragma unroll
        for (int g = 0; g < 2 * kBlocks; ++g)
#pragma unroll
            for (int d = 0; d < kDims; ++d) {
                const auto a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr<dev::s16x4_t>)(vt[d & 1] + Tile<D>::block(2 * g, d / 2)));
                const auto b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr<dev::s16x4_t>)(vt[d & 1] + Tile<D>::block(2 * g + 1, d / 2)));
                const dev::bf16x4_t x = __builtin_bit_cast(dev::bf16x4_t, a), y = __builtin_bit_cast(dev::bf16x4_t, b);
                o[d] = mma32(__builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7), w[g], o[d]);
            }
    };
    // Where keys are absent, or some rows do not see some, no value that is not finite may meet a weight of zero: absent
    // keys' values are zeroed; others are added to the rows that see them, and are zeros in the product.  All waves
    // come here together, between the landing of the tile's V and its sums.
    const auto mend = [&](int t, uint64_t now) {
        const int p0 = u.lo + t * kTile;
        if (!special(t, now)) return;
        constexpr int kCount = kTile * D / 8;
        const lds_t vt = vtile(t);
        bool fine = true;
        for (int i = threadIdx.x; i < kCount; i += kThreads) {
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
        for (int i = 0; i < WAVES; ++i) bad |= flags[i];
        if (bad) {
            if (p0 < end) {
                const uint64_t seen = sees.from(p0) & now;
                for (int n = 0; n < kTile; ++n) {
                    if (!(now >> n & 1)) continue;
                    float by = 1.f;
                    if constexpr (kCodes) by = vstored(t)[n];
#pragma unroll
                    for (int d = 0; d < kDims; ++d)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int dim = 32 * d + 8 * (i / 4) + 4 * half + i % 4;
                            float v = (float)*(lds_ptr<__bf16>)(vt + Tile<D>::v(n, dim / 8) + dim % 8 * 2);
                            if (!dev::finite(by)) v = NAN;
                            if (!dev::finite(v) && (seen >> n & 1)) o[d][i] += v;
                        }
                }
            }
            dev::lds_barrier();
            for (int i = threadIdx.x; i < kCount; i += kThreads) {
                const lds_ptr<bf16x8_t> at = (lds_ptr<bf16x8_t>)vt + i;
                bf16x8_t v = *at;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (!dev::finite((float)v[j])) v[j] = (__bf16)0.f;
                *at = v;
            }
        }
        dev::lds_barrier();
    };

    // ---- slot 2 t: the first waves' products of tile t (their sums of t - 1); slot 2 t + 1: their softmax.  The waves behind do the
    // same one slot later.  A wave issues behind its softmax, where it has time to wait for the memory path: the first waves
    // issue(t) in slot 2 t + 1, the others in slot 2 t; all land(t) in slot 2 t + 1, where issue(t - 2) is behind any of them.  K of tile t
    // is read in slots 2 t and 2 t + 1, V in 2 t + 2 and 2 t + 3; K of t + 3 and V of t + 2 take the places of t - 1 and t - 2, last read in
    // slot 2 t - 1; so do codes' tiles, K of t + 1 and V of t made in slot 2 t + 1.  A wave reads its entries of t + 4 in issue(t), behind
    // land(t - 1), to which those of issue(t - 3) have come.
    landed<0>();               // the first four tiles' entries (and the queries)
    prepare(-3);
    for (int t = -3; t < 0; ++t) issue(t);
    land(-1);
    dev::lds_barrier();
    if (behind) {
        issue(0);
        dev::lds_barrier();
    }
    for (int t = 0; t < tiles; ++t) {
        const bool work = u.lo + t * kTile < end;
        const uint64_t now = behind ? there[0] : there[1];
        if (t > 0 && u.lo + (t - 1) * kTile < end) sums(t - 1);
        if (work) scores(t);
        if (behind) land(t);
        if (kPair) dev::lds_barrier();
        if (behind) mend(t, now);
        if (work) softmax(t, now);
        if (!behind || t + 1 < tiles) issue(behind ? t + 1 : t);
        if (!behind) land(t);
        if (!behind || t + 1 < tiles) dev::lds_barrier();
        if (!behind) mend(t, now);
    }
    if (u.lo + (tiles - 1) * kTile < end) sums(tiles - 1);
    landed<0>();               // nothing may be on its way into LDS that is another workgroup's by then

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

// Eight waves of 256 registers, or four of 512: a head of 256 dims has sums of 128 registers a wave.
template <int FORMAT, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, D == 256 ? 1 : 2) void wide_decode_kernel(AttentionKernelArgs k) {
    extern __shared__ __align__(16) char lds[];
    Unit u;
    if (decode_unit<__bf16, D>(k, 32 * WAVES, 64 * WAVES, u)) attend<FORMAT, D, WAVES>(k, u, (lds_t)lds);
}

// Tiles from the last to the first: those with the most keys start first.
template <int FORMAT, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, D == 256 ? 1 : 2) void wide_prompt_kernel(AttentionKernelArgs k) {
    extern __shared__ __align__(16) char lds[];
    const unsigned H = (unsigned)k.a.cache.num_heads, at = blockIdx.x / H;
    Unit u;
    if (prompt_unit(k, 32 * WAVES, k.row_tiles - 1 - (int)at, (int)(blockIdx.x - at * H), u)) attend<FORMAT, D, WAVES>(k, u, (lds_t)lds);
}

template <int FORMAT, int D, int WAVES>
hipError_t launch(AttentionKernelArgs k, hipStream_t stream) {
    constexpr int kThreads = 64 * WAVES, kRows = 32 * WAVES;
    const int H = k.a.cache.num_heads;
    const bool decode = k.a.tokens_per_row > 0;
    const int64_t tiles = decode ? (k.a.tokens_per_row * (int)k.group.d + kRows - 1) / kRows : k.a.total_tokens * (int)k.group.d / kRows + k.a.num_seqs;
    const int64_t units = decode ? ((int64_t)k.a.num_seqs * k.spans * H + 7) / 8 * 8 : H;
    if (!grid_fits(tiles * units, kThreads) || k.a.total_tokens * (int64_t)k.group.d > 0x7fffffffLL) return hipErrorInvalidConfiguration;
    k.row_tiles = (int)tiles;
    auto* const kernel = decode ? wide_decode_kernel<FORMAT, D, WAVES> : wide_prompt_kernel<FORMAT, D, WAVES>;
    kernel<<<(unsigned)(tiles * units), kThreads, (Plan<FORMAT, D, WAVES>::kTotal), stream>>>(k);
    return hipGetLastError();
}

template <int FORMAT, int D>
hipError_t launch(const AttentionKernelArgs& k, hipStream_t stream) {
    if constexpr (D < 256)
        if (k.a.tokens_per_row == 0 || k.a.tokens_per_row * (int)k.group.d > 128) return launch<FORMAT, D, 8>(k, stream);
    return launch<FORMAT, D, 4>(k, stream);
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
