// rq_attn_api.cpp -- entry points of the attention around the linears: head
// norm with rotation and cache store, paged single-token attention, eviction.
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

}  // extern "C"
