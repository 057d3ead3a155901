// rq_attn_util.h -- the paged cache as the attention kernels take it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "rq_internal.h"

namespace rq {
namespace attn {

// A cache as the kernels take it: slot j of (sequence b, head h) is row
// (page * heads + h) * 2^page_log + j % 2^page_log of k and v.
struct Cache {
    void *k, *v;
    float *k_scale, *v_scale;
    const int32_t *table;
    float *weight;
    int32_t *pos;
    int32_t heads, D, page_log, batch, table_ld, pages;

    // row of slot j, or -1 where no page is there
    __device__ __forceinline__ int64_t row(int b, int h, int j) const {
        const int32_t pg = table[(int64_t)b * table_ld + (j >> page_log)];
        if ((uint32_t)pg >= (uint32_t)pages) return -1;
        return (((int64_t)pg * heads + h) << page_log) + (j & ((1 << page_log) - 1));
    }
    __device__ __forceinline__ int64_t slots() const { return (int64_t)table_ld << page_log; }
};

}  // namespace attn

inline attn::Cache device_cache(const rq_kv_cache *c) {
    return {c->k, c->v, c->k_scale, c->v_scale, c->table, c->weight, c->pos,
            c->heads, c->head_dim, ilog2(c->page), c->batch, c->table_ld, (int32_t)c->pages};
}
}  // namespace rq
