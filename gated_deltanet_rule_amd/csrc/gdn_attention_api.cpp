// gdn_attention_api.cpp -- the C ABI of the attention layers' operators
// (include/gdn_attention.h): host-side validation and dispatch to the gfx950 launchers, by
// the same rules as gdn_api.cpp and gdn_layer_api.cpp.
#include <cmath>
#include <cstddef>

#include "gdn_attention.h"
#include "gdn_attention_internal.h"
#include "gdn_check.h"

namespace {

using gdn::aligned;
using gdn::check_ptrs;
using gdn::fail;
using gdn::hip_status;

constexpr int64_t kMaxTokens = 0x7fffffffLL - 2 * GDN_CHUNK;
constexpr int kMaxHeadDim = 512;
constexpr int kMaxRowTokens = 64;

// A launcher's result: a call too large for one launch is the caller's to split.
gdn_status launched(hipError_t e, const char* what) {
    if (e == hipErrorInvalidConfiguration) return fail(GDN_ERR_UNSUPPORTED, "%s exceeds the launch grid of 2^32 - 1 threads", what);
    return hip_status(e, what);
}

size_t elem(int32_t dtype) { return dtype == GDN_BF16 ? 2 : 4; }

gdn_status check_dtype(int32_t dtype) {
    if (dtype != GDN_F32 && dtype != GDN_BF16)
        return fail(GDN_ERR_UNSUPPORTED, "dtype %d is neither GDN_F32 (0) nor GDN_BF16 (1)", dtype);
    return GDN_OK;
}

gdn_status check_tokens(int64_t n, const char* name) {
    if (n < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "%s %lld is negative", name, (long long)n);
    if (n > kMaxTokens) return fail(GDN_ERR_UNSUPPORTED, "%s %lld exceeds the supported 2^31 - 129", name, (long long)n);
    return GDN_OK;
}

gdn_status check_stride(int64_t stride, int64_t row, const char* name) {
    if (stride < row || stride % 8 != 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s %lld must be a multiple of 8 of at least the %lld values of a row", name,
                    (long long)stride, (long long)row);
    return GDN_OK;
}

// The cache's scalars and, unless it has no rows, its pointers.
gdn_status check_cache_shape(const gdn_kv_cache* c) {
    if (!c) return fail(GDN_ERR_INVALID_ARGUMENT, "cache is NULL");
    if (c->num_heads <= 0) return fail(GDN_ERR_INVALID_ARGUMENT, "num_heads %d is not positive", c->num_heads);
    if (c->head_dim <= 0) return fail(GDN_ERR_INVALID_ARGUMENT, "head_dim %d is not positive", c->head_dim);
    if (c->head_dim % 8 != 0 || c->head_dim > kMaxHeadDim)
        return fail(GDN_ERR_UNSUPPORTED, "head_dim %d is not a multiple of 8 up to %d", c->head_dim, kMaxHeadDim);
    if ((int64_t)c->num_heads * c->head_dim > (1 << 20))
        return fail(GDN_ERR_UNSUPPORTED, "rows of num_heads %d x head_dim %d values exceed the supported 2^20", c->num_heads, c->head_dim);
    gdn_status st = check_dtype(c->dtype);
    if (st != GDN_OK) return st;
    if (c->format != GDN_CACHE_PLAIN && c->format != GDN_CACHE_E4M3 && c->format != GDN_CACHE_INT8)
        return fail(GDN_ERR_UNSUPPORTED, "format %d: must be GDN_CACHE_PLAIN (0), GDN_CACHE_E4M3 (1) or GDN_CACHE_INT8 (2)", c->format);
    return GDN_OK;
}

gdn_status check_cache(const gdn_kv_cache* c) {
    gdn_status st = check_cache_shape(c);
    if (st != GDN_OK) return st;
    if (c->num_rows < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "num_rows %lld is negative", (long long)c->num_rows);
    if (c->num_rows > 0x7fffffffLL) return fail(GDN_ERR_UNSUPPORTED, "num_rows %lld exceeds the supported 2^31 - 1", (long long)c->num_rows);
    if (c->num_rows == 0) return GDN_OK;
    st = check_ptrs({{"cache k", c->k, 16}, {"cache v", c->v, 16}});
    if (st != GDN_OK || c->format == GDN_CACHE_PLAIN) return st;
    return check_ptrs({{"k_scale", c->k_scale, 4}, {"v_scale", c->v_scale, 4}});
}

gdn_status check_heads(const gdn_kv_cache* c, int32_t num_q_heads, float scale) {
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return fail(GDN_ERR_UNSUPPORTED, "head_dim %d: the attention takes 64, 128 or 256", c->head_dim);
    if (num_q_heads <= 0 || num_q_heads % c->num_heads != 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "num_q_heads %d is not a positive multiple of num_heads %d", num_q_heads, c->num_heads);
    if ((int64_t)num_q_heads * c->head_dim > (1 << 20))
        return fail(GDN_ERR_UNSUPPORTED, "rows of num_q_heads %d x head_dim %d values exceed the supported 2^20", num_q_heads, c->head_dim);
    if (!std::isfinite(scale)) return fail(GDN_ERR_INVALID_ARGUMENT, "scale is not finite");
    return GDN_OK;
}

gdn_status check_table(int32_t width, int32_t kv_block) {
    if (width < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "kv_table_width %d is negative", width);
    if (kv_block <= 0) return fail(GDN_ERR_INVALID_ARGUMENT, "kv_block %d is not positive", kv_block);
    return GDN_OK;
}

// Keys that a table holds.  The kernels look up to 512 positions past the last key.
int table_capacity(int32_t width, int32_t kv_block) {
    const int64_t keys = (int64_t)width * kv_block, most = 0x7fffffffLL - 1024;
    return (int)(keys < most ? keys : most);
}

gdn::AttentionArgs attention_args(const gdn_kv_cache* cache, int32_t num_q_heads, float scale, int32_t num_seqs, int64_t total_tokens,
                                  const void* q, int64_t q_stride, const int32_t* kv_table, int32_t width, int32_t kv_block, void* o) {
    gdn::AttentionArgs a = {};
    a.cache = *cache;
    a.H_q = num_q_heads;
    a.scale = scale;
    a.num_seqs = num_seqs;
    a.total_tokens = total_tokens;
    a.q = q;
    a.q_stride = q_stride;
    a.table = kv_table;
    a.table_width = width;
    a.kv_block = kv_block;
    a.capacity = table_capacity(width, kv_block);
    a.o = o;
    return a;
}

}  // namespace

extern "C" {

gdn_status gdn_rotary(const gdn_rotary_shape* shape, int64_t num_tokens, const int32_t* positions, const float* inv_freq,
                      const void* q, int64_t q_stride, const void* k, int64_t k_stride, void* q_out, int64_t q_out_stride,
                      void* k_out, int64_t k_out_stride, hipStream_t stream) {
    gdn::clear_error();
    if (!shape) return fail(GDN_ERR_INVALID_ARGUMENT, "shape is NULL");
    const int heads[2] = {shape->num_q_heads, shape->num_k_heads}, d = shape->head_dim, r = shape->rotary_dim;
    if (heads[0] < 0 || heads[1] < 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "num_q_heads %d or num_k_heads %d is negative", heads[0], heads[1]);
    if (d <= 0) return fail(GDN_ERR_INVALID_ARGUMENT, "head_dim %d is not positive", d);
    if (d > kMaxHeadDim) return fail(GDN_ERR_UNSUPPORTED, "head_dim %d exceeds %d", d, kMaxHeadDim);
    if (r < 2 || r % 2 != 0 || r > d)
        return fail(GDN_ERR_INVALID_ARGUMENT, "rotary_dim %d is not an even number from 2 to head_dim %d", r, d);
    if (((int64_t)heads[0] + heads[1]) * d > (1 << 20))
        return fail(GDN_ERR_UNSUPPORTED, "rows of %d + %d heads of %d values exceed the supported 2^20", heads[0], heads[1], d);
    if (!std::isfinite(shape->factor)) return fail(GDN_ERR_INVALID_ARGUMENT, "factor is not finite");
    gdn_status st = check_dtype(shape->dtype);
    if (st != GDN_OK) return st;
    st = check_tokens(num_tokens, "num_tokens");
    if (st != GDN_OK || num_tokens == 0 || heads[0] + heads[1] == 0) return st;
    st = check_ptrs({{"positions", positions, 4}, {"inv_freq", inv_freq, 4}});
    if (st != GDN_OK) return st;
    gdn::RotaryArgs a = {*shape, num_tokens, positions, inv_freq, {q, k}, {q_stride, k_stride}, {q_out, k_out}, {q_out_stride, k_out_stride}};
    const char* names[2][4] = {{"q", "q_stride", "q_out", "q_out_stride"}, {"k", "k_stride", "k_out", "k_out_stride"}};
    const size_t es = elem(shape->dtype);
    for (int i = 0; i < 2; ++i) {
        if (heads[i] == 0) continue;
        const int64_t row = (int64_t)heads[i] * d;
        if (a.in_stride[i] < row)
            return fail(GDN_ERR_INVALID_ARGUMENT, "%s %lld is smaller than a row of %lld", names[i][1], (long long)a.in_stride[i], (long long)row);
        if (a.out_stride[i] < row)
            return fail(GDN_ERR_INVALID_ARGUMENT, "%s %lld is smaller than a row of %lld", names[i][3], (long long)a.out_stride[i], (long long)row);
        if (a.in[i] && a.in[i] == a.out[i] && a.in_stride[i] != a.out_stride[i])
            return fail(GDN_ERR_INVALID_ARGUMENT, "%s is in place with %s %lld and %s %lld", names[i][0], names[i][1],
                        (long long)a.in_stride[i], names[i][3], (long long)a.out_stride[i]);
        st = check_ptrs({{names[i][0], a.in[i], es}, {names[i][2], a.out[i], es}});
        if (st != GDN_OK) return st;
    }
    return launched(gdn::launch_rotary(a, stream), "rotary launch");
}

gdn_status gdn_kv_cache_write(const gdn_kv_cache* cache, int64_t num_tokens, const void* k, int64_t k_stride, const void* v,
                              int64_t v_stride, const int64_t* slots, hipStream_t stream) {
    gdn::clear_error();
    gdn_status st = check_cache(cache);
    if (st != GDN_OK) return st;
    st = check_tokens(num_tokens, "num_tokens");
    if (st != GDN_OK || num_tokens == 0) return st;
    const int64_t row = (int64_t)cache->num_heads * cache->head_dim;
    st = check_stride(k_stride, row, "k_stride");
    if (st != GDN_OK) return st;
    st = check_stride(v_stride, row, "v_stride");
    if (st != GDN_OK) return st;
    st = check_ptrs({{"k", k, 16}, {"v", v, 16}, {"slots", slots, 8}});
    if (st != GDN_OK) return st;
    gdn::CacheCopyArgs a = {*cache, num_tokens, slots, {k, v}, {k_stride, v_stride}, {nullptr, nullptr}};
    return launched(gdn::launch_cache_write(a, stream), "cache write launch");
}

gdn_status gdn_kv_cache_read(const gdn_kv_cache* cache, int64_t num_tokens, const int64_t* slots, void* k_out, void* v_out,
                             hipStream_t stream) {
    gdn::clear_error();
    gdn_status st = check_cache(cache);
    if (st != GDN_OK) return st;
    st = check_tokens(num_tokens, "num_tokens");
    if (st != GDN_OK || num_tokens == 0) return st;
    st = check_ptrs({{"slots", slots, 8}, {"k_out", k_out, 16}, {"v_out", v_out, 16}});
    if (st != GDN_OK) return st;
    gdn::CacheCopyArgs a = {*cache, num_tokens, slots, {nullptr, nullptr}, {0, 0}, {k_out, v_out}};
    return launched(gdn::launch_cache_read(a, stream), "cache read launch");
}

gdn_status gdn_attention_prefill(const gdn_kv_cache* cache, int32_t num_q_heads, float scale, int32_t num_seqs, int64_t total_tokens,
                                 const int32_t* cu_seqlens, const int32_t* start_pos, const void* q, int64_t q_stride,
                                 const int32_t* kv_table, int32_t kv_table_width, int32_t kv_block, void* o, hipStream_t stream) {
    gdn::clear_error();
    gdn_status st = check_cache(cache);
    if (st != GDN_OK) return st;
    st = check_heads(cache, num_q_heads, scale);
    if (st != GDN_OK) return st;
    if (num_seqs < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "num_seqs %d is negative", num_seqs);
    st = check_tokens(total_tokens, "total_tokens");
    if (st != GDN_OK) return st;
    st = check_table(kv_table_width, kv_block);
    if (st != GDN_OK || num_seqs == 0 || total_tokens == 0) return st;
    st = check_stride(q_stride, (int64_t)num_q_heads * cache->head_dim, "q_stride");
    if (st != GDN_OK) return st;
    if (!aligned(start_pos, 4)) return fail(GDN_ERR_INVALID_ARGUMENT, "start_pos is not 4-byte aligned");
    if (kv_table_width > 0) {
        st = check_ptrs({{"kv_table", kv_table, 4}});
        if (st != GDN_OK) return st;
    }
    st = check_ptrs({{"cu_seqlens", cu_seqlens, 4}, {"q", q, 16}, {"o", o, 16}});
    if (st != GDN_OK) return st;
    gdn::AttentionArgs a = attention_args(cache, num_q_heads, scale, num_seqs, total_tokens, q, q_stride, kv_table, kv_table_width, kv_block, o);
    a.cu_seqlens = cu_seqlens;
    a.past = start_pos;
    return launched(gdn::launch_attention_prefill(a, stream), "attention launch");
}

size_t gdn_attention_decode_workspace_size(const gdn_kv_cache* cache, int32_t num_q_heads, int32_t num_rows, int32_t tokens_per_row,
                                           int64_t max_keys) {
    if (check_cache_shape(cache) != GDN_OK || check_heads(cache, num_q_heads, 1.f) != GDN_OK || num_rows < 0 || tokens_per_row < 1 ||
        tokens_per_row > kMaxRowTokens || (int64_t)num_rows * tokens_per_row > kMaxTokens || max_keys < 0)
        return 0;
    return gdn::attention_workspace_bytes(num_q_heads, cache->num_heads, cache->head_dim, num_rows, tokens_per_row,
                                          max_keys < kMaxTokens ? max_keys : kMaxTokens);
}

gdn_status gdn_attention_decode(const gdn_kv_cache* cache, int32_t num_q_heads, float scale, int32_t num_rows, int32_t tokens_per_row,
                                const int32_t* computed, const int64_t* tree_mask, const void* q, int64_t q_stride,
                                const int32_t* kv_table, int32_t kv_table_width, int32_t kv_block, int64_t max_keys, void* o,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
    gdn::clear_error();
    gdn_status st = check_cache(cache);
    if (st != GDN_OK) return st;
    st = check_heads(cache, num_q_heads, scale);
    if (st != GDN_OK) return st;
    if (num_rows < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "num_rows %d is negative", num_rows);
    if (tokens_per_row < 1) return fail(GDN_ERR_INVALID_ARGUMENT, "tokens_per_row %d is not positive", tokens_per_row);
    if (tokens_per_row > kMaxRowTokens)
        return fail(GDN_ERR_UNSUPPORTED, "tokens_per_row %d exceeds the %d bits of a mask", tokens_per_row, kMaxRowTokens);
    const int64_t tokens = (int64_t)num_rows * tokens_per_row;
    st = check_tokens(tokens, "num_rows x tokens_per_row");
    if (st != GDN_OK) return st;
    if (max_keys < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "max_keys %lld is negative", (long long)max_keys);
    st = check_table(kv_table_width, kv_block);
    if (st != GDN_OK || num_rows == 0) return st;
    st = check_stride(q_stride, (int64_t)num_q_heads * cache->head_dim, "q_stride");
    if (st != GDN_OK) return st;
    if (!aligned(tree_mask, 8)) return fail(GDN_ERR_INVALID_ARGUMENT, "tree_mask is not 8-byte aligned");
    if (kv_table_width > 0) {
        st = check_ptrs({{"kv_table", kv_table, 4}});
        if (st != GDN_OK) return st;
    }
    gdn::AttentionArgs a = attention_args(cache, num_q_heads, scale, num_rows, tokens, q, q_stride, kv_table, kv_table_width, kv_block, o);
    a.past = computed;
    a.tokens_per_row = tokens_per_row;
    a.tree_mask = tree_mask;
    a.max_keys = max_keys > 0 && max_keys < a.capacity ? (int)max_keys : a.capacity;
    const size_t need = gdn::attention_workspace_bytes(num_q_heads, cache->num_heads, cache->head_dim, num_rows, tokens_per_row, a.max_keys);
    if (workspace_bytes < need)
        return fail(GDN_ERR_INVALID_ARGUMENT, "workspace_bytes %zu is smaller than the %zu bytes required", workspace_bytes, need);
    if (need > 0) {
        st = check_ptrs({{"workspace", workspace, 256}});
        if (st != GDN_OK) return st;
    }
    a.workspace = workspace;
    st = check_ptrs({{"computed", computed, 4}, {"q", q, 16}, {"o", o, 16}});
    if (st != GDN_OK) return st;
    return launched(gdn::launch_attention_decode(a, stream), "attention decode launch");
}

}  // extern "C"
