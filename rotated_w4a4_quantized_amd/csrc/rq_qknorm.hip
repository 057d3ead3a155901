// rq_qknorm.hip -- RMS norm of query and key heads with the position rotation,
// and the store of keys and values into a paged cache, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w;  pair (a, b) of angle i becomes
//   (y_a c_i - y_b s_i, y_b c_i + y_a s_i).  fp32, rounded once at the store.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rq_attn_util.h"
#include "rq_internal.h"

namespace rq {
namespace {

using attn::Cache;

struct Args {
    const void *qkv;
    const int32_t *positions, *seq, *place;
    void *q_out, *k_out;
    const float *qw, *kw, *cos, *sin;
    int64_t ld, q_ld, k_ld, T;
    int32_t hq, hkv, D, rot, table_rows;
    float eps;
    Cache c;
};

// One wave per (token, head); lane l holds the pairs l and l + 64.
template <bool BF16, bool I8>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(Args a, int inter, int has_cache) {
    const int lane = threadIdx.x & 63;
    const int nh = a.hq + a.hkv * (has_cache ? 2 : 1);
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (id >= a.T * nh) return;
    const int64_t t = id / nh;
    const int h = (int)(id - t * nh);
    const bool is_q = h < a.hq, is_v = h >= a.hq + a.hkv;
    const int64_t in = t * a.ld + (int64_t)h * a.D;
    const int pairs = a.D / 2, rp = is_v ? 0 : a.rot / 2;
    float x[2][2];
    int ia[2], ib[2];
    float ss = 0.0f;
    for (int u = 0; u < 2; ++u) {
        const int i = lane + 64 * u;
        ia[u] = 2 * i;
        ib[u] = 2 * i + 1;
        if (i < rp && !inter) {
            ia[u] = i;
            ib[u] = i + rp;
        }
        x[u][0] = i < pairs ? attn::load1<BF16>(a.qkv, in + ia[u]) : 0.0f;
        x[u][1] = i < pairs ? attn::load1<BF16>(a.qkv, in + ib[u]) : 0.0f;
        ss += x[u][0] * x[u][0] + x[u][1] * x[u][1];
    }
    const int64_t p = a.positions ? a.positions[t] : t;
    if (!is_v) {
        for (int o = 1; o < 64; o *= 2) ss += __shfl_xor(ss, o);
        const float r = 1.0f / sqrtf(ss / (float)a.D + a.eps);
        const float *w = is_q ? a.qw : a.kw;
        for (int u = 0; u < 2; ++u) {
            const int i = lane + 64 * u;
            if (i >= pairs) continue;
            const float y0 = x[u][0] * r * (w ? w[ia[u]] : 1.0f), y1 = x[u][1] * r * (w ? w[ib[u]] : 1.0f);
            x[u][0] = y0;
            x[u][1] = y1;
            if (i < rp) {
                const bool in_table = p >= 0 && p < a.table_rows;
                const float c = in_table ? a.cos[p * rp + i] : __builtin_nanf("");
                const float s = in_table ? a.sin[p * rp + i] : __builtin_nanf("");
                x[u][0] = y0 * c - y1 * s;
                x[u][1] = y1 * c + y0 * s;
            }
        }
    }
    if (!is_v) {
        void *out = is_q ? a.q_out : a.k_out;
        const int64_t o = is_q ? t * a.q_ld + (int64_t)h * a.D : t * a.k_ld + (int64_t)(h - a.hq) * a.D;
        if (out)
            for (int u = 0; u < 2; ++u)
                if (lane + 64 * u < pairs) {
                    attn::store1<BF16>(out, o + ia[u], x[u][0]);
                    attn::store1<BF16>(out, o + ib[u], x[u][1]);
                }
    }
    if (is_q || !has_cache) return;
    const int64_t b = a.seq ? a.seq[t] : t;
    const int32_t pl = a.place[t];
    if (b < 0 || b >= a.c.batch || pl < 0 || pl >= a.c.slots()) return;
    const int kh = h - a.hq - (is_v ? a.hkv : 0);
    const int64_t row = a.c.row((int)b, kh, pl);
    if (row < 0) return;
    if (!is_v && lane == 0) {
        const int64_t m = (b * a.hkv + kh) * a.c.slots() + pl;
        if (a.c.weight) a.c.weight[m] = 0.0f;
        if (a.c.pos) a.c.pos[m] = (int32_t)p;
    }
    float inv = 0.0f;
    if (I8) {
        float amax = 0.0f;
        for (int u = 0; u < 2; ++u) amax = fmaxf(amax, fmaxf(fabsf(x[u][0]), fabsf(x[u][1])));
        for (int o = 1; o < 64; o *= 2) amax = fmaxf(amax, __shfl_xor(amax, o));
        inv = amax > 0.0f ? 127.0f / amax : 0.0f;
        if (lane == 0) (is_v ? a.c.v_scale : a.c.k_scale)[row] = amax / 127.0f;
    }
    for (int u = 0; u < 2; ++u) {
        if (lane + 64 * u >= pairs) continue;
        for (int e = 0; e < 2; ++e) {
            const int64_t o = row * a.D + (e ? ib[u] : ia[u]);
            if (I8)
                static_cast<int8_t *>(is_v ? a.c.v : a.c.k)[o] = (int8_t)fminf(fmaxf(rintf(x[u][e] * inv), -127.0f), 127.0f);
            else
                static_cast<uint16_t *>(is_v ? a.c.v : a.c.k)[o] = attn::f32_bf16(x[u][e]);
        }
    }
}

}  // namespace

int launch_qk_norm_rope(const rq_qk_norm *d, const void *qkv, int bf16, int64_t ld, int64_t T,
                        const int32_t *positions, void *q_out, int64_t q_ld, void *k_out,
                        int64_t k_ld, const rq_kv_cache *cache, const int32_t *seq,
                        const int32_t *place, void *stream) {
    Args a{};
    a.qkv = qkv, a.positions = positions, a.seq = seq, a.place = place, a.q_out = q_out, a.k_out = k_out;
    a.qw = d->q_weight, a.kw = d->k_weight, a.cos = d->cos, a.sin = d->sin;
    a.ld = ld, a.q_ld = q_ld, a.k_ld = k_ld, a.T = T;
    a.hq = d->q_heads, a.hkv = d->kv_heads, a.D = d->head_dim, a.rot = d->rot_dim, a.table_rows = d->table_rows;
    a.eps = d->eps;
    const bool i8 = cache && cache->dtype == RQ_I8;
    if (cache && d->kv_heads > 0) a.c = device_cache(cache);
    const int has_cache = cache && d->kv_heads > 0;
    const int64_t waves = T * (a.hq + a.hkv * (has_cache ? 2 : 1));
    // (at most 2^31 tokens of 3072 heads: checked against the grid's limit)
    if ((waves + 3) / 4 > 0x7fffffff) return (int)hipErrorInvalidValue;
    auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, static_cast<hipStream_t>(stream),
                           a, (int)d->interleaved, has_cache);
    };
    if (bf16) {
        if (i8) go(qk_norm_rope_kernel<true, true>);
        else go(qk_norm_rope_kernel<true, false>);
    } else {
        if (i8) go(qk_norm_rope_kernel<false, true>);
        else go(qk_norm_rope_kernel<false, false>);
    }
    return (int)hipGetLastError();
}

}  // namespace rq
