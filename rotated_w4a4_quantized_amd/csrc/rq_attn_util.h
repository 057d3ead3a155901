// rq_attn_util.h -- the paged cache as the attention kernels take it, and what
// they share: vector types, rounding to bf16, sums over a wave, joined statistics.
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

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const f2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));
}
__device__ __forceinline__ float lo_of(uint32_t p) { return __builtin_bit_cast(float, p << 16); }
__device__ __forceinline__ float hi_of(uint32_t p) { return __builtin_bit_cast(float, p & 0xffff0000u); }
constexpr float kLn2 = 0.69314718055994531f;
template <bool BF16>
__device__ __forceinline__ void store4(void *p, int64_t at, f4 v) {
    if constexpr (BF16) *reinterpret_cast<u2 *>(static_cast<uint16_t *>(p) + at) = u2{pack2(v[0], v[1]), pack2(v[2], v[3])};
    else *reinterpret_cast<f4 *>(static_cast<float *>(p) + at) = v;
}
// x as `parts` bf16 numbers whose sum carries 8 bits of x each
template <int PARTS>
__device__ __forceinline__ void split2(float x, float y, uint32_t (&p)[PARTS]) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        p[i] = pack2(x, y);
        x -= lo_of(p[i]);
        y -= hi_of(p[i]);
    }
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float from_lane(float x, float none) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, none), __builtin_bit_cast(int, x), CTRL, ROWS, 0xf, false));
}
// (shifts within rows of 16 lanes, then the rows' last lanes passed on: lane 63 has all)
__device__ __forceinline__ float wave_max(float x) {
    x = fmaxf(x, from_lane<0x111, 0xf>(x, -INFINITY));
    x = fmaxf(x, from_lane<0x112, 0xf>(x, -INFINITY));
    x = fmaxf(x, from_lane<0x114, 0xf>(x, -INFINITY));
    x = fmaxf(x, from_lane<0x118, 0xf>(x, -INFINITY));
    x = fmaxf(x, from_lane<0x142, 0xa>(x, -INFINITY));
    x = fmaxf(x, from_lane<0x143, 0xc>(x, -INFINITY));
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}
__device__ __forceinline__ float wave_sum(float x) {
    x += from_lane<0x111, 0xf>(x, 0.0f);
    x += from_lane<0x112, 0xf>(x, 0.0f);
    x += from_lane<0x114, 0xf>(x, 0.0f);
    x += from_lane<0x118, 0xf>(x, 0.0f);
    x += from_lane<0x142, 0xa>(x, 0.0f);
    x += from_lane<0x143, 0xc>(x, 0.0f);
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}
// Statistics of a head over its n parts, by one wave: all lanes get the maximum
// and the sum relative to it.
__device__ __forceinline__ void join_stats(const f2 *st, int n, int64_t stride, int lane, float &M, float &L) {
    f2 mine = {-INFINITY, 0.0f};             // (a lane's own parts first)
    for (int i = lane; i < n; i += 64) {
        const f2 x = st[i * stride];
        const float top = fmaxf(mine[0], x[0]);
        if (top == -INFINITY) continue;
        mine = f2{top, mine[1] * __builtin_amdgcn_exp2f(mine[0] - top) + x[1] * __builtin_amdgcn_exp2f(x[0] - top)};
    }
    M = wave_max(mine[0]);
    L = wave_sum(mine[0] == -INFINITY ? 0.0f : mine[1] * __builtin_amdgcn_exp2f(mine[0] - M));
}

}  // namespace attn

inline attn::Cache device_cache(const rq_kv_cache *c) {
    return {c->k, c->v, c->k_scale, c->v_scale, c->table, c->weight, c->pos,
            c->heads, c->head_dim, ilog2(c->page), c->batch, c->table_ld, (int32_t)c->pages};
}
}  // namespace rq
