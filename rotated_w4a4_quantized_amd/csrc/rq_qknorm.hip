// rq_qknorm.hip -- RMS norm of query and key heads with the position rotation,
// and the store of keys and values into a paged cache, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * w;  pair (a, b) of angle i becomes
//   (y_a c_i - y_b s_i, y_b c_i + y_a s_i).  fp32, rounded once at the store.
//
// Everything is read and written once: HBM bounds long calls (32760 tokens of 24
// heads x 128 in bf16, 419 MB: 83 us, 5.06 TB/s, what a copy reaches), launch and
// three dependent loads (place, page, and positions before cosines) the short ones
// (one token of 40 heads: 4.0 us).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rq_attn_util.h"
#include "rq_internal.h"

namespace rq {
namespace {

using attn::Cache;

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

struct Args {
    const void *qkv;
    const int32_t *positions, *seq, *place;
    void *q_out, *k_out;
    const float *qw, *kw, *cos, *sin;
    int64_t ld, q_ld, k_ld, T;
    int32_t hq, hkv, nh, D, rot, table_rows;
    int32_t per, chunks;   // head groups of a wave's visit to a token; visits of a token
    float eps;
    Cache c;               // (k is NULL: no cache)
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const f2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));
}

// Eight values of a lane's item as they lie in memory, at a .. a + 3 and at
// b .. b + 3 (b = a + 4 unless the item is rotated by halves).
template <bool BF16>
struct Raw {
    u4 v[BF16 ? 1 : 2];
};
template <bool BF16, bool WHOLE>
__device__ __forceinline__ Raw<BF16> load8(const void *p, int64_t a, int64_t b) {
    Raw<BF16> r;
    if constexpr (!BF16) {
        r.v[0] = *reinterpret_cast<const u4 *>(static_cast<const float *>(p) + a);
        r.v[1] = *reinterpret_cast<const u4 *>(static_cast<const float *>(p) + b);
    } else if constexpr (WHOLE) {
        r.v[0] = *reinterpret_cast<const u4 *>(static_cast<const uint16_t *>(p) + a);
    } else {
        const u2 l = *reinterpret_cast<const u2 *>(static_cast<const uint16_t *>(p) + a);
        const u2 h = *reinterpret_cast<const u2 *>(static_cast<const uint16_t *>(p) + b);
        r.v[0] = u4{l[0], l[1], h[0], h[1]};
    }
    return r;
}
template <bool BF16>
__device__ __forceinline__ void widen8(const Raw<BF16> &r, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            x[2 * i] = __builtin_bit_cast(float, r.v[0][i] << 16);
            x[2 * i + 1] = __builtin_bit_cast(float, r.v[0][i] & 0xffff0000u);
        } else {
            // (by value: a bit cast of a vector's element in place reads element 0)
            const uint32_t lo = r.v[0][i], hi = r.v[1][i];
            x[i] = __builtin_bit_cast(float, lo);
            x[4 + i] = __builtin_bit_cast(float, hi);
        }
    }
}
template <bool BF16, bool WHOLE>
__device__ __forceinline__ void store8(void *p, int64_t a, int64_t b, const float (&x)[8]) {
    if constexpr (BF16) {
        const u4 v = {pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7])};
        if constexpr (WHOLE) *reinterpret_cast<u4 *>(static_cast<uint16_t *>(p) + a) = v;
        else {
            *reinterpret_cast<u2 *>(static_cast<uint16_t *>(p) + a) = u2{v[0], v[1]};
            *reinterpret_cast<u2 *>(static_cast<uint16_t *>(p) + b) = u2{v[2], v[3]};
        }
    } else {
        *reinterpret_cast<f4 *>(static_cast<float *>(p) + a) = f4{x[0], x[1], x[2], x[3]};
        *reinterpret_cast<f4 *>(static_cast<float *>(p) + b) = f4{x[4], x[5], x[6], x[7]};
    }
}
// four codes of the symmetric 8-bit rule
__device__ __forceinline__ uint32_t codes4(const float *x, float inv) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // (|x inv| <= 127 but for rounding; NaN, from a value or from 0 times an
        // infinity, gives 0)
        const float y = x[i] * inv;
        const int c = y == y ? (int)fminf(fmaxf(rintf(y), -127.0f), 127.0f) : 0;
        r |= (uint32_t)(c & 0xff) << (8 * i);
    }
    return r;
}

// 1 / sqrt(x).  The instruction takes numbers below 2^-126 for 0, which a small
// eps lets through; scaling by powers of two is exact.
__device__ __forceinline__ float inv_root(float x) {
    const bool tiny = x < 0x1p-100f;
    const float r = __builtin_amdgcn_rsqf(tiny ? x * 0x1p64f : x);
    return tiny ? r * 0x1p32f : r;
}

// A head is LP lanes (a power of two, 8 D's values each); a wave holds 64 / LP
// heads of one token at a time and walks over the token's heads, with the
// token's cosines and sines and both weights in registers.  LP divides a wave,
// so the sum over a head is an exchange between lanes, without LDS or barrier.
// U heads' loads are issued before the first is used.  Pairs live within a lane:
// neighbours of one 16-byte load, or the same places of two 8-byte loads half a
// rotation apart.
template <bool BF16, bool I8, bool INTER, int LP>
__global__ void __launch_bounds__(256) qk_norm_rope_kernel(Args a) {
    constexpr int HPW = 64 / LP, U = BF16 ? 8 : 4;
    const int lane = threadIdx.x & 63, item = lane % LP, slot = lane / LP;
    const int D = a.D;
    const bool live = item * 8 < D, turned = item * 8 < a.rot;
    const int half = a.rot / 2;
    const int ia = !INTER && turned ? item * 4 : item * 8, ib = !INTER && turned ? ia + half : ia + 4;

    // (visits may touch any memory, so the weights are read before them)
    float wq[8], wk[8];
    const f4 one = {1, 1, 1, 1};
    const int da = live ? ia : 0, db = live ? ib : 0;
    const f4 q0 = a.qw ? *reinterpret_cast<const f4 *>(a.qw + da) : one, q1 = a.qw ? *reinterpret_cast<const f4 *>(a.qw + db) : one;
    const f4 k0 = a.kw ? *reinterpret_cast<const f4 *>(a.kw + da) : one, k1 = a.kw ? *reinterpret_cast<const f4 *>(a.kw + db) : one;
#pragma unroll
    for (int i = 0; i < 4; ++i) wq[i] = q0[i], wq[4 + i] = q1[i], wk[i] = k0[i], wk[4 + i] = k1[i];
    const float inv_d = 1.0f / (float)D;
    const int64_t visits = a.T * a.chunks, stride = (int64_t)gridDim.x * 4;
    for (int64_t id = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); id < visits; id += stride) {
        const int64_t t = a.chunks == 1 ? id : id / a.chunks;
        const int first = a.chunks == 1 ? 0 : (int)(id - t * a.chunks) * a.per * HPW;
        const int last = min(a.nh, first + a.per * HPW);
        Raw<BF16> raw[U];
        auto load = [&](int h0) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * HPW;
                if (live && h < last) {
                    const int64_t in = t * a.ld + (int64_t)h * D;
                    raw[u] = load8<BF16, INTER>(a.qkv, in + ia, in + ib);
                } else raw[u] = {};
            }
        };
        // The heads are asked for before anything is waited for, then the three
        // numbers of the token, then what depends on them.
        load(first + slot);
        const int64_t p = a.positions ? a.positions[t] : t;
        const int64_t b = a.c.k && a.seq ? a.seq[t] : t;
        const int32_t place = a.c.k ? a.place[t] : -1;
        float c[4] = {1, 1, 1, 1}, s[4] = {0, 0, 0, 0};
        if (turned) {
            const bool in_table = p >= 0 && p < a.table_rows;
            const int64_t at = (in_table ? p : 0) * half + item * 4;
            const f4 cv = *reinterpret_cast<const f4 *>(a.cos + at), sv = *reinterpret_cast<const f4 *>(a.sin + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                c[i] = in_table ? cv[i] : __builtin_nanf("");
                s[i] = in_table ? sv[i] : __builtin_nanf("");
            }
        }
        // the row of the cache that head 0 goes to, -1: none
        int64_t row0 = -1, meta = 0;
        const int page = 1 << a.c.page_log;
        if (b >= 0 && b < a.c.batch && place >= 0 && place < a.c.slots()) {
            row0 = a.c.row((int)b, 0, place);
            meta = b * a.hkv * a.c.slots() + place;
        }
        for (int h0 = first + slot; h0 - slot < last; h0 += HPW * U) {
            if (h0 != first + slot) load(h0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = h0 + u * HPW;
                if (h - slot >= last) break;   // (the same in every lane)
                const bool is_q = h < a.hq, is_v = h >= a.hq + a.hkv;
                float x[8], y[8];
                widen8<BF16>(raw[u], x);
                if (!is_v) {
                    float ss = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                    for (int o = 1; o < LP; o *= 2) ss += __shfl_xor(ss, o);
                    const float r = inv_root(fmaf(ss, inv_d, a.eps));
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = x[i] * r * (is_q ? wq[i] : wk[i]);
                    if (turned) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            constexpr int S = INTER ? 2 : 1, O = INTER ? 1 : 4;
                            const float ya = y[i * S], yb = y[i * S + O];
                            y[i * S] = ya * c[i] - yb * s[i];
                            y[i * S + O] = yb * c[i] + ya * s[i];
                        }
                    }
                    if (live && h < last) {
                        if (is_q) {
                            const int64_t o = t * a.q_ld + (int64_t)h * D;
                            store8<BF16, INTER>(a.q_out, o + ia, o + ib, y);
                        } else if (a.k_out) {
                            const int64_t o = t * a.k_ld + (int64_t)(h - a.hq) * D;
                            store8<BF16, INTER>(a.k_out, o + ia, o + ib, y);
                        }
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = x[i];
                }
                const int kh = h - a.hq - (is_v ? a.hkv : 0);
                const bool kept = !is_q && row0 >= 0 && h < last;
                const int64_t row = row0 + (int64_t)kh * page;
                void *store = is_v ? a.c.v : a.c.k;
                if (I8) {
                    // the largest magnitude by its bits: they are ordered, with NaN above
                    // all, which the scale then carries (a float maximum would drop it)
                    uint32_t top = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = max(top, __builtin_bit_cast(uint32_t, y[i]) & 0x7fffffffu);
#pragma unroll
                    for (int o = 1; o < LP; o *= 2) top = max(top, (uint32_t)__shfl_xor((int)top, o));
                    const float amax = __builtin_bit_cast(float, top);
                    const float inv = amax > 0.0f ? 127.0f / amax : 0.0f;
                    if (kept && live) {
                        char *o = static_cast<char *>(store) + row * D;
                        const uint32_t lo = codes4(y, inv), hi = codes4(y + 4, inv);
                        if constexpr (INTER) *reinterpret_cast<u2 *>(o + ia) = u2{lo, hi};
                        else {
                            *reinterpret_cast<uint32_t *>(o + ia) = lo;
                            *reinterpret_cast<uint32_t *>(o + ib) = hi;
                        }
                        if (item == 0) (is_v ? a.c.v_scale : a.c.k_scale)[row] = amax / 127.0f;
                    }
                } else if (kept && live)
                    store8<true, INTER>(store, row * D + ia, row * D + ib, y);
                if (kept && item == 0 && !is_v) {
                    const int64_t m = meta + (int64_t)kh * a.c.slots();
                    if (a.c.weight) a.c.weight[m] = 0.0f;
                    if (a.c.pos) a.c.pos[m] = (int32_t)p;
                }
            }
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
    const bool stored = cache && d->kv_heads > 0 && cache->batch > 0;
    if (stored) a.c = device_cache(cache);
    a.nh = a.hq + a.hkv * (stored ? 2 : 1);
    const bool i8 = stored && cache->dtype == RQ_I8;
    const int lp = a.D <= 16 ? 2 : a.D <= 32 ? 4 : a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32;
    // A token's heads are dealt out to as many waves as make one round of what is
    // resident (16 a CU): 1999 fp32 tokens of 24 small heads take 8.7 us, and 10.5
    // with a wave a group of heads; 2000 tokens of 24 x 128 in bf16 8.9 against 11.4.
    const int groups = (a.nh + 64 / lp - 1) / (64 / lp);
    const int64_t full = (int64_t)device_cus() * 16;
    a.per = (int)std::min<int64_t>(groups, std::max<int64_t>(1, (T * groups + full - 1) / full));
    a.chunks = (groups + a.per - 1) / a.per;
    // Twice what is resident, then waves walk over visits: 32760 tokens of 24 heads
    // take 83 us, with a single round of waves 85, with one visit a wave 80.
    const int64_t wgs = std::min<int64_t>((T * a.chunks + 3) / 4, (int64_t)device_cus() * 8);
    auto go = [&](auto kern) {
        hipLaunchKernelGGL(kern, dim3((unsigned)wgs), dim3(256), 0, static_cast<hipStream_t>(stream), a);
    };
    auto lanes = [&](auto b, auto q, auto n) {
        constexpr bool B = decltype(b)::value, Q = decltype(q)::value, N = decltype(n)::value;
        if (lp == 2) go(qk_norm_rope_kernel<B, Q, N, 2>);
        else if (lp == 4) go(qk_norm_rope_kernel<B, Q, N, 4>);
        else if (lp == 8) go(qk_norm_rope_kernel<B, Q, N, 8>);
        else if (lp == 16) go(qk_norm_rope_kernel<B, Q, N, 16>);
        else go(qk_norm_rope_kernel<B, Q, N, 32>);
    };
    auto pairs = [&](auto b, auto q) {
        if (d->interleaved) lanes(b, q, std::true_type{});
        else lanes(b, q, std::false_type{});
    };
    if (bf16) {
        if (i8) pairs(std::true_type{}, std::true_type{});
        else pairs(std::true_type{}, std::false_type{});
    } else {
        if (i8) pairs(std::false_type{}, std::true_type{});
        else pairs(std::false_type{}, std::false_type{});
    }
    return (int)hipGetLastError();
}

}  // namespace rq
