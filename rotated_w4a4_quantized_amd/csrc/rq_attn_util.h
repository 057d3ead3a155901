// rq_attn_util.h -- device helpers shared by the attention kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "rq_internal.h"

namespace rq {
namespace attn {

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }
// round to nearest even
__device__ __forceinline__ uint16_t f32_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

template <bool BF16>
__device__ __forceinline__ float load1(const void *p, int64_t i) {
    if constexpr (BF16) return bf16_f32(static_cast<const uint16_t *>(p)[i]);
    else return static_cast<const float *>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store1(void *p, int64_t i, float v) {
    if constexpr (BF16) static_cast<uint16_t *>(p)[i] = f32_bf16(v);
    else static_cast<float *>(p)[i] = v;
}

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
