// rq_attn_api.cpp -- entry points around the linears: head norm with rotation and
// cache store, paged single-token attention, eviction; the residual stream with its
// norms, attention to states of another length, attention behind a shared prefix.
// Argument validation and dispatch.  Every check runs before the first launch;
// sizes of workspaces and grids follow the device's number of CUs (read once).

#include <hip/hip_runtime.h>

#include <cmath>
#include <string>

#include "rq_internal.h"

using namespace rq;

namespace {

rq_status hip_status(int err, const char *what) {
    if (err == (int)hipSuccess) return RQ_OK;
    return fail(RQ_ERR_HIP, std::string(what) + ": " + hipGetErrorString((hipError_t)err));
}

bool head_dim_ok(int D) { return D >= 16 && D <= 256 && D % 8 == 0; }

// rows of `ld` elements that start 16-byte aligned
bool rows_aligned(const void *p, int64_t ld, int dtype) {
    return aligned16(p) && ld % (dtype == RQ_BF16 ? 8 : 4) == 0;
}

rq_status check_cache(const rq_kv_cache *c, bool need_buffers) {
    if (!c) return fail(RQ_ERR_NULL, "cache descriptor is NULL");
    if (c->dtype != RQ_BF16 && c->dtype != RQ_I8)
        return fail(RQ_ERR_DTYPE, "the cache must be RQ_BF16 or RQ_I8");
    if (c->heads < 1 || c->heads > 1024) return fail(RQ_ERR_SHAPE, "cache heads out of range [1, 1024]");
    if (!head_dim_ok(c->head_dim))
        return fail(RQ_ERR_SHAPE, "head_dim must satisfy 16 <= D <= 256 and D % 8 == 0, got " +
                                      std::to_string(c->head_dim));
    if (c->page < 16 || c->page > 1024 || !is_pow2(c->page))
        return fail(RQ_ERR_SHAPE, "page must be a power of two in [16, 1024], got " + std::to_string(c->page));
    if (c->batch < 0 || c->batch > 65535) return fail(RQ_ERR_SHAPE, "cache batch out of range [0, 65535]");
    if (c->table_ld < 1 || (int64_t)c->table_ld * c->page > (int64_t(1) << 24))
        return fail(RQ_ERR_SHAPE, "a sequence holds 1 page to 2^24 slots");
    if (c->pages < 1 || c->pages > 0x7fffffff) return fail(RQ_ERR_SHAPE, "pages out of range");
    if (!need_buffers || c->batch == 0) return RQ_OK;
    if (!c->k || !c->v || !c->table) return fail(RQ_ERR_NULL, "cache k, v and table must not be NULL");
    if (c->dtype == RQ_I8 && (!c->k_scale || !c->v_scale))
        return fail(RQ_ERR_NULL, "an RQ_I8 cache needs k_scale and v_scale");
    if (!aligned16(c->k) || !aligned16(c->v) || (c->k_scale && !aligned16(c->k_scale)) ||
        (c->v_scale && !aligned16(c->v_scale)) || !aligned16(c->table) ||
        (c->weight && !aligned16(c->weight)) || (c->pos && !aligned16(c->pos)))
        return fail(RQ_ERR_ALIGN, "cache buffers must be 16-byte aligned");
    return RQ_OK;
}

rq_status check_max_len(const rq_kv_cache *c, int64_t max_len) {
    if (max_len < 0 || max_len > (int64_t)c->table_ld * c->page)
        return fail(RQ_ERR_SHAPE, "max_len must lie in [0, table_ld * page]");
    return RQ_OK;
}

rq_status check_attention(const rq_kv_cache *c, int q_heads, int64_t max_len, int track, bool buffers) {
    rq_status st = check_cache(c, buffers);
    if (st != RQ_OK) return st;
    if (q_heads < 1 || q_heads > 1024 || q_heads % c->heads != 0)
        return fail(RQ_ERR_SHAPE, "q_heads must be a multiple of the cache's heads, at most 1024");
    if (track != 0 && track != 1) return fail(RQ_ERR_SHAPE, "track must be 0 or 1");
    if ((st = check_max_len(c, max_len)) != RQ_OK) return st;
    if (!attend_fits(c, q_heads, max_len, track))
        return fail(RQ_ERR_SHAPE, "batch, heads and max_len of a tracked call need more workgroups than a launch holds");
    return RQ_OK;
}

rq_status check_evict(const rq_kv_cache *c, int keep, int64_t max_len, bool buffers) {
    rq_status st = check_cache(c, buffers);
    if (st != RQ_OK) return st;
    if (keep < 1) return fail(RQ_ERR_SHAPE, "keep must be at least 1");
    if ((st = check_max_len(c, max_len)) != RQ_OK) return st;
    if (!evict_fits(c, keep, max_len))
        return fail(RQ_ERR_SHAPE, "batch, heads and moves need more workgroups than a launch holds");
    return RQ_OK;
}

bool io_dtype(int dtype) { return dtype == RQ_F32 || dtype == RQ_BF16; }

rq_status check_norm(const rq_norm *n, const char *name) {
    if (!n) return RQ_OK;
    if (n->kind != RQ_NORM_RMS && n->kind != RQ_NORM_LAYER)
        return fail(RQ_ERR_SHAPE, std::string(name) + ": unknown kind of norm");
    if (!(n->eps >= 0.0f) || std::isinf(n->eps)) return fail(RQ_ERR_SHAPE, std::string(name) + ": eps must be finite and >= 0");
    if ((n->weight && !aligned16(n->weight)) || (n->bias && !aligned16(n->bias)))
        return fail(RQ_ERR_ALIGN, std::string(name) + ": weight and bias must be 16-byte aligned");
    return RQ_OK;
}

rq_status check_cross(const rq_states *s, int64_t queries, int q_heads, int dtype) {
    if (!s) return fail(RQ_ERR_NULL, "states descriptor is NULL");
    if (!io_dtype(dtype)) return fail(RQ_ERR_DTYPE, "q must be RQ_F32 or RQ_BF16");
    if (s->heads < 1 || s->heads > 1024) return fail(RQ_ERR_SHAPE, "the states' heads out of range [1, 1024]");
    if (!head_dim_ok(s->head_dim))
        return fail(RQ_ERR_SHAPE, "head_dim must satisfy 16 <= D <= 256 and D % 8 == 0, got " + std::to_string(s->head_dim));
    if (s->batch < 0 || s->batch > 65535) return fail(RQ_ERR_SHAPE, "batch out of range [0, 65535]");
    if (s->keys < 0 || s->keys > (int64_t(1) << 24)) return fail(RQ_ERR_SHAPE, "keys out of range [0, 2^24]");
    if (q_heads < 1 || q_heads > 1024 || q_heads % s->heads != 0)
        return fail(RQ_ERR_SHAPE, "q_heads must be a multiple of the states' heads, at most 1024");
    if (queries < 0 || queries > (int64_t(1) << 24)) return fail(RQ_ERR_SHAPE, "queries out of range [0, 2^24]");
    if (!cross_fits(s, queries, q_heads, dtype == RQ_BF16))
        return fail(RQ_ERR_SHAPE, "batch * queries * q_heads must be below 2^25");
    return RQ_OK;
}

rq_status check_prefix(const rq_kv_cache *c, int q_heads, int dtype, int64_t prefix, int64_t max_len, bool buffers) {
    rq_status st = check_cache(c, buffers);
    if (st != RQ_OK) return st;
    if (!io_dtype(dtype)) return fail(RQ_ERR_DTYPE, "q must be RQ_F32 or RQ_BF16");
    if (q_heads < 1 || q_heads > 1024 || q_heads % c->heads != 0)
        return fail(RQ_ERR_SHAPE, "q_heads must be a multiple of the cache's heads, at most 1024");
    if ((st = check_max_len(c, max_len)) != RQ_OK) return st;
    if (prefix < 0 || prefix > max_len) return fail(RQ_ERR_SHAPE, "prefix must lie in [0, max_len]");
    if (!prefix_fits(c, q_heads, dtype == RQ_BF16, prefix, max_len))
        return fail(RQ_ERR_SHAPE, "batch * q_heads must be below 2^25");
    return RQ_OK;
}

// (the kernels multiply by scale log2(e), which has to be finite, too)
rq_status check_scale(float scale) {
    if (!(std::fabs(scale) <= 0x1p127f)) return fail(RQ_ERR_SHAPE, "scale must be finite, at most 2^127 in magnitude");
    return RQ_OK;
}

rq_status check_workspace(const char *what, size_t need, const void *workspace, size_t have) {
    if (need == 0) return RQ_OK;
    if (!workspace || have < need)
        return fail(RQ_ERR_SHAPE, std::string(what) + " needs a workspace of " + std::to_string(need) + " bytes");
    if (!aligned16(workspace)) return fail(RQ_ERR_ALIGN, "workspace must be 16-byte aligned");
    return RQ_OK;
}

}  // namespace

extern "C" {

rq_status rq_qk_norm_rope(const rq_qk_norm *d, const void *qkv, int32_t dtype, int64_t ld,
                          int64_t T, const int32_t *positions, void *q_out, int64_t q_ld,
                          void *k_out, int64_t k_ld, const rq_kv_cache *cache,
                          const int32_t *seq, const int32_t *place, void *stream) {
    clear_error();
    if (!d) return fail(RQ_ERR_NULL, "head norm descriptor is NULL");
    if (d->q_heads < 1 || d->q_heads > 1024 || d->kv_heads < 0 || d->kv_heads > 1024)
        return fail(RQ_ERR_SHAPE, "q_heads must lie in [1, 1024] and kv_heads in [0, 1024]");
    const int D = d->head_dim;
    if (!head_dim_ok(D))
        return fail(RQ_ERR_SHAPE, "head_dim must satisfy 16 <= D <= 256 and D % 8 == 0, got " + std::to_string(D));
    if (d->rot_dim < 0 || d->rot_dim > D || d->rot_dim % 8 != 0)
        return fail(RQ_ERR_SHAPE, "rot_dim must be a multiple of 8 in [0, head_dim]");
    if (d->interleaved != 0 && d->interleaved != 1) return fail(RQ_ERR_SHAPE, "interleaved must be 0 or 1");
    if (d->rot_dim > 0 && d->table_rows < 1) return fail(RQ_ERR_SHAPE, "table_rows must be at least 1");
    if (!(d->eps >= 0.0f) || std::isinf(d->eps)) return fail(RQ_ERR_SHAPE, "eps must be finite and >= 0");
    if (dtype != RQ_F32 && dtype != RQ_BF16) return fail(RQ_ERR_DTYPE, "qkv must be RQ_F32 or RQ_BF16");
    if (T < 0 || T >= (int64_t(1) << 31)) return fail(RQ_ERR_SHAPE, "T out of range");
    const int64_t qw = (int64_t)d->q_heads * D, kw = (int64_t)d->kv_heads * D;
    // (rows of at most 2^31 elements keep every offset below 2^63)
    const int64_t wide = int64_t(1) << 31;
    if (ld < qw + kw * (cache ? 2 : 1) || ld > wide)
        return fail(RQ_ERR_SHAPE, "ld is shorter than a row of qkv");
    if (q_ld < qw || q_ld > wide) return fail(RQ_ERR_SHAPE, "q_ld is shorter than a row of queries");
    if (k_out && (k_ld < kw || k_ld > wide)) return fail(RQ_ERR_SHAPE, "k_ld is shorter than a row of keys");
    if (cache) {
        rq_status st = check_cache(cache, T > 0);
        if (st != RQ_OK) return st;
        if (cache->heads != d->kv_heads || cache->head_dim != D)
            return fail(RQ_ERR_SHAPE, "the cache's heads and head_dim are not the descriptor's");
    }
    if (T == 0) return RQ_OK;
    if (!qkv || !q_out) return fail(RQ_ERR_NULL, "qkv and q_out must not be NULL");
    if (d->kv_heads > 0 && !k_out && !cache)
        return fail(RQ_ERR_NULL, "key heads need k_out or a cache");
    if (cache && !place) return fail(RQ_ERR_NULL, "a cache needs place");
    if (d->rot_dim > 0 && (!d->cos || !d->sin)) return fail(RQ_ERR_NULL, "cos and sin must not be NULL");
    if (!rows_aligned(qkv, ld, dtype) || !rows_aligned(q_out, q_ld, dtype) ||
        (k_out && !rows_aligned(k_out, k_ld, dtype)) || (d->cos && !aligned16(d->cos)) ||
        (d->sin && !aligned16(d->sin)) || (d->q_weight && !aligned16(d->q_weight)) ||
        (d->k_weight && !aligned16(d->k_weight)))
        return fail(RQ_ERR_ALIGN, "rows of qkv, q_out and k_out, and the tables, must be 16-byte aligned");
    return hip_status(launch_qk_norm_rope(d, qkv, dtype == RQ_BF16, ld, T, positions, q_out, q_ld, k_out,
                                          k_ld, cache, seq, place, stream),
                      "qk_norm_rope launch");
}

rq_status rq_paged_attention_workspace_bytes(const rq_kv_cache *cache, int32_t q_heads,
                                             int64_t max_len, int32_t track, size_t *bytes) {
    clear_error();
    rq_status st = check_attention(cache, q_heads, max_len, track, false);
    if (st != RQ_OK) return st;
    if (!bytes) return fail(RQ_ERR_NULL, "bytes is NULL");
    *bytes = attend_workspace_bytes(cache, q_heads, max_len, track);
    return RQ_OK;
}

rq_status rq_paged_attention(const rq_kv_cache *cache, const void *q, int32_t dtype, int64_t q_ld,
                             int32_t q_heads, float scale, const int32_t *lens, int64_t max_len,
                             const uint8_t *mask, int64_t mask_ld, void *out, int64_t out_ld,
                             float *lse, int32_t track, float *weight_out, void *workspace,
                             size_t workspace_bytes, void *stream) {
    clear_error();
    rq_status st = check_attention(cache, q_heads, max_len, track, true);
    if (st != RQ_OK) return st;
    if (dtype != RQ_F32 && dtype != RQ_BF16) return fail(RQ_ERR_DTYPE, "q must be RQ_F32 or RQ_BF16");
    if (!std::isfinite(scale)) return fail(RQ_ERR_SHAPE, "scale must be finite");
    const int64_t row = (int64_t)q_heads * cache->head_dim, wide = int64_t(1) << 31;
    if (q_ld < row || q_ld > wide || out_ld < row || out_ld > wide)
        return fail(RQ_ERR_SHAPE, "q_ld and out_ld must hold a row of q_heads * head_dim");
    if (mask && (mask_ld < max_len || mask_ld > wide)) return fail(RQ_ERR_SHAPE, "mask_ld is shorter than max_len");
    if (cache->batch == 0) return RQ_OK;
    if (!q || !lens || !out) return fail(RQ_ERR_NULL, "q, lens and out must not be NULL");
    if (track && (!cache->weight || !weight_out))
        return fail(RQ_ERR_NULL, "track needs the cache's weight and weight_out");
    if (!rows_aligned(q, q_ld, dtype) || !rows_aligned(out, out_ld, dtype) ||
        (track && !aligned16(weight_out)))
        return fail(RQ_ERR_ALIGN, "rows of q and out, and weight_out, must be 16-byte aligned");
    const size_t need = attend_workspace_bytes(cache, q_heads, max_len, track);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(RQ_ERR_SHAPE, "paged attention needs a workspace of " + std::to_string(need) + " bytes");
        if (!aligned16(workspace)) return fail(RQ_ERR_ALIGN, "workspace must be 16-byte aligned");
    }
    return hip_status(launch_paged_attention(cache, q, dtype == RQ_BF16, q_ld, q_heads, scale, lens, max_len,
                                             mask, mask_ld, out, out_ld, lse, track, weight_out, workspace,
                                             stream),
                      "paged attention launch");
}

rq_status rq_cache_evict_workspace_bytes(const rq_kv_cache *cache, int32_t keep, int64_t max_len,
                                         size_t *bytes) {
    clear_error();
    rq_status st = check_evict(cache, keep, max_len, false);
    if (st != RQ_OK) return st;
    if (!bytes) return fail(RQ_ERR_NULL, "bytes is NULL");
    *bytes = evict_workspace_bytes(cache, keep, max_len);
    return RQ_OK;
}

rq_status rq_cache_evict(const rq_kv_cache *cache, const int32_t *lens, int64_t max_len,
                         int32_t keep, int32_t recent, int32_t sink, int32_t *lens_out,
                         float *weight_out, int32_t *pos_out, void *workspace,
                         size_t workspace_bytes, void *stream) {
    clear_error();
    rq_status st = check_evict(cache, keep, max_len, true);
    if (st != RQ_OK) return st;
    if (recent < 0 || sink < 0) return fail(RQ_ERR_SHAPE, "recent and sink must not be negative");
    if (cache->batch == 0) return RQ_OK;
    if (!lens || !lens_out || !weight_out || !pos_out || !cache->weight || !cache->pos)
        return fail(RQ_ERR_NULL, "lens, lens_out, weight_out, pos_out and the cache's weight and pos must not be NULL");
    if (!aligned16(weight_out) || !aligned16(pos_out))
        return fail(RQ_ERR_ALIGN, "weight_out and pos_out must be 16-byte aligned");
    const size_t need = evict_workspace_bytes(cache, keep, max_len);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(RQ_ERR_SHAPE, "eviction needs a workspace of " + std::to_string(need) + " bytes");
        if (!aligned16(workspace)) return fail(RQ_ERR_ALIGN, "workspace must be 16-byte aligned");
    }
    return hip_status(launch_cache_evict(cache, lens, max_len, keep, recent, sink, lens_out, weight_out,
                                         pos_out, workspace, stream),
                      "cache evict launch");
}

rq_status rq_block_norm(const rq_norm *post, const rq_norm *pre, const rq_modulation *mod,
                        int32_t width, const void *x, int32_t x_dtype, int64_t x_ld, const void *y,
                        int32_t dtype, int64_t y_ld, int64_t T, float alpha, float beta, void *h,
                        int64_t h_ld, void *z, int64_t z_ld, void *stream) {
    clear_error();
    rq_status st = check_norm(post, "post");
    if (st == RQ_OK) st = check_norm(pre, "pre");
    if (st != RQ_OK) return st;
    if (width < 8 || width > 16384 || width % 8 != 0)
        return fail(RQ_ERR_SHAPE, "width must satisfy 8 <= K <= 16384 and K % 8 == 0, got " + std::to_string(width));
    if (!io_dtype(x_dtype) || !io_dtype(dtype)) return fail(RQ_ERR_DTYPE, "x and y must be RQ_F32 or RQ_BF16");
    if (T < 0 || T >= (int64_t(1) << 31)) return fail(RQ_ERR_SHAPE, "T out of range");
    if (!std::isfinite(alpha) || !std::isfinite(beta)) return fail(RQ_ERR_SHAPE, "alpha and beta must be finite");
    const int64_t wide = int64_t(1) << 31;
    auto row_ok = [&](const void *p, int64_t ld) { return !p || (ld >= width && ld <= wide); };
    if (x_ld < width || x_ld > wide || !row_ok(y, y_ld) || !row_ok(h, h_ld) || !row_ok(z, z_ld))
        return fail(RQ_ERR_SHAPE, "x_ld, y_ld, h_ld and z_ld must hold a row of width");
    if (mod) {
        if (mod->rows < 1) return fail(RQ_ERR_SHAPE, "modulations have at least one row");
        if (mod->rows > 1 && (mod->ld < width || mod->ld > wide))
            return fail(RQ_ERR_SHAPE, "the modulations' ld is shorter than a row of width");
        if (!mod->index && (mod->per < 1 || (T > 0 && (T - 1) / mod->per >= mod->rows)))
            return fail(RQ_ERR_SHAPE, "the modulations have no row for every token: rows * per < T");
    }
    if (T == 0) return RQ_OK;
    if (!x || (!h && !z)) return fail(RQ_ERR_NULL, "x, and h or z, must not be NULL");
    if (post && !y) return fail(RQ_ERR_NULL, "post needs y");
    if (pre && !z) return fail(RQ_ERR_NULL, "pre needs z");
    if (!rows_aligned(x, x_ld, x_dtype) || (y && !rows_aligned(y, y_ld, dtype)) ||
        (h && !rows_aligned(h, h_ld, x_dtype)) || (z && !rows_aligned(z, z_ld, dtype)))
        return fail(RQ_ERR_ALIGN, "rows of x, y, h and z must be 16-byte aligned");
    if (mod && ((mod->rows > 1 && mod->ld % 4 != 0) || (mod->gate && !aligned16(mod->gate)) ||
                (mod->shift && !aligned16(mod->shift)) || (mod->scale && !aligned16(mod->scale))))
        return fail(RQ_ERR_ALIGN, "rows of gate, shift and scale must be 16-byte aligned");
    return hip_status(launch_block_norm(post, pre, mod, width, x, x_dtype == RQ_BF16, x_ld, y, dtype == RQ_BF16,
                                        y_ld, T, alpha, beta, h, h_ld, z, z_ld, stream),
                      "block norm launch");
}

rq_status rq_cross_attention_workspace_bytes(const rq_states *states, int64_t queries, int32_t q_heads,
                                             int32_t dtype, size_t *bytes) {
    clear_error();
    rq_status st = check_cross(states, queries, q_heads, dtype);
    if (st != RQ_OK) return st;
    if (!bytes) return fail(RQ_ERR_NULL, "bytes is NULL");
    *bytes = cross_workspace_bytes(states, queries, q_heads, dtype == RQ_BF16);
    return RQ_OK;
}

rq_status rq_cross_attention(const rq_states *states, const void *q, int32_t dtype, int64_t q_ld,
                             int64_t q_stride, int64_t queries, int32_t q_heads, float scale,
                             const int32_t *q_lens, void *out, int64_t out_ld, int64_t out_stride,
                             float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    clear_error();
    rq_status st = check_cross(states, queries, q_heads, dtype);
    if (st != RQ_OK) return st;
    if ((st = check_scale(scale)) != RQ_OK) return st;
    const int D = states->head_dim;
    const int64_t row = (int64_t)q_heads * D, kv = (int64_t)states->heads * D;
    // (rows of at most 2^31 elements and sequences of 2^46 keep every offset below 2^63)
    const int64_t wide = int64_t(1) << 31, far = int64_t(1) << 46;
    if (q_ld < row || q_ld > wide || out_ld < row || out_ld > wide)
        return fail(RQ_ERR_SHAPE, "q_ld and out_ld must hold a row of q_heads * head_dim");
    if (q_stride < 0 || q_stride > far || out_stride < 0 || out_stride > far)
        return fail(RQ_ERR_SHAPE, "q_stride and out_stride must lie in [0, 2^46]");
    if (states->batch == 0 || queries == 0) return RQ_OK;
    // (sequences one after another, or their tokens in turn)
    if (states->batch > 1 && out_stride < (queries - 1) * out_ld + row &&
        (out_stride < row || out_ld < (states->batch - 1) * out_stride + row))
        return fail(RQ_ERR_SHAPE, "sequences of out overlap");
    if (!q || !out) return fail(RQ_ERR_NULL, "q and out must not be NULL");
    if (!rows_aligned(q, q_ld, dtype) || !rows_aligned(out, out_ld, dtype) ||
        q_stride % (dtype == RQ_BF16 ? 8 : 4) != 0 || out_stride % (dtype == RQ_BF16 ? 8 : 4) != 0)
        return fail(RQ_ERR_ALIGN, "rows of q and out must be 16-byte aligned");
    if (states->keys > 0) {
        if (!states->k || !states->v) return fail(RQ_ERR_NULL, "the states' k and v must not be NULL");
        // (16 rows of at most 2^22 elements keep the offsets of one load below 2^31 bytes)
        const int64_t most = int64_t(1) << 22;
        if (states->k_ld < kv || states->k_ld > most || states->v_ld < kv || states->v_ld > most)
            return fail(RQ_ERR_SHAPE, "k_ld and v_ld must hold a row of heads * head_dim, and 2^22 elements at most");
        if (states->k_stride < 0 || states->k_stride > far || states->v_stride < 0 || states->v_stride > far)
            return fail(RQ_ERR_SHAPE, "k_stride and v_stride must lie in [0, 2^46]");
        if (states->mask && states->mask_ld != 0 && (states->mask_ld < states->keys || states->mask_ld > wide))
            return fail(RQ_ERR_SHAPE, "mask_ld is shorter than keys");
        if (!rows_aligned(states->k, states->k_ld, RQ_BF16) || !rows_aligned(states->v, states->v_ld, RQ_BF16) ||
            states->k_stride % 8 != 0 || states->v_stride % 8 != 0)
            return fail(RQ_ERR_ALIGN, "rows of the states' k and v must be 16-byte aligned");
    }
    st = check_workspace("cross attention", cross_workspace_bytes(states, queries, q_heads, dtype == RQ_BF16), workspace, workspace_bytes);
    if (st != RQ_OK) return st;
    return hip_status(launch_cross_attention(states, q, dtype == RQ_BF16, q_ld, q_stride, queries, q_heads, scale, q_lens,
                                             out, out_ld, out_stride, lse, workspace, stream),
                      "cross attention launch");
}

rq_status rq_prefix_attention_workspace_bytes(const rq_kv_cache *cache, int32_t q_heads, int32_t dtype,
                                              int64_t prefix, int64_t max_len, size_t *bytes) {
    clear_error();
    rq_status st = check_prefix(cache, q_heads, dtype, prefix, max_len, false);
    if (st != RQ_OK) return st;
    if (!bytes) return fail(RQ_ERR_NULL, "bytes is NULL");
    *bytes = prefix_workspace_bytes(cache, q_heads, dtype == RQ_BF16, prefix, max_len);
    return RQ_OK;
}

rq_status rq_prefix_attention(const rq_kv_cache *cache, const int32_t *prefix_table, int64_t prefix,
                              const void *q, int32_t dtype, int64_t q_ld, int32_t q_heads, float scale,
                              const int32_t *lens, int64_t max_len, const uint8_t *mask, int64_t mask_ld,
                              void *out, int64_t out_ld, float *lse, void *workspace,
                              size_t workspace_bytes, void *stream) {
    clear_error();
    rq_status st = check_prefix(cache, q_heads, dtype, prefix, max_len, true);
    if (st != RQ_OK) return st;
    if ((st = check_scale(scale)) != RQ_OK) return st;
    const int64_t row = (int64_t)q_heads * cache->head_dim, wide = int64_t(1) << 31;
    if (q_ld < row || q_ld > wide || out_ld < row || out_ld > wide)
        return fail(RQ_ERR_SHAPE, "q_ld and out_ld must hold a row of q_heads * head_dim");
    if (mask && (mask_ld < max_len || mask_ld > wide)) return fail(RQ_ERR_SHAPE, "mask_ld is shorter than max_len");
    if (cache->batch == 0) return RQ_OK;
    if (!q || !lens || !out || (prefix > 0 && !prefix_table))
        return fail(RQ_ERR_NULL, "q, lens, out and prefix_table must not be NULL");
    if (!rows_aligned(q, q_ld, dtype) || !rows_aligned(out, out_ld, dtype) || (prefix_table && !aligned16(prefix_table)))
        return fail(RQ_ERR_ALIGN, "rows of q and out, and prefix_table, must be 16-byte aligned");
    st = check_workspace("prefix attention", prefix_workspace_bytes(cache, q_heads, dtype == RQ_BF16, prefix, max_len),
                         workspace, workspace_bytes);
    if (st != RQ_OK) return st;
    return hip_status(launch_prefix_attention(cache, prefix_table, prefix, q, dtype == RQ_BF16, q_ld, q_heads, scale, lens,
                                              max_len, mask, mask_ld, out, out_ld, lse, workspace, stream),
                      "prefix attention launch");
}

}  // extern "C"
