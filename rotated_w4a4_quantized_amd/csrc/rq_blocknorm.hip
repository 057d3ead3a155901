// rq_blocknorm.hip -- what lies between two blocks of a transformer, in one pass:
//
//   h = alpha x + beta gate (.) post(y);   z = pre(h) (.) (1 + scale) + shift
//
// with post and pre an RMS norm, a layer norm or nothing.  x and y are read once,
// h and z written once: HBM bounds it (32760 x 1536, fp32 stream, 604 MB in 124 us: 4.9
// TB/s, a copy's rate; 8192 x 1152 in bf16 75 MB in 18 us, of which 15 are the bytes'),
// but for the widths whose registers do not suffice (below).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "rq_attn_util.h"
#include "rq_internal.h"

namespace rq {
namespace {

using namespace attn;

struct Norm {
    const float *weight, *bias;
    float eps;
    int kind;   // rq_norm_kind, or -1: none
};
struct Args {
    Norm post, pre;
    const float *gate, *shift, *scale;
    const int32_t *index;
    const void *x, *y;
    void *h, *z;
    int64_t x_ld, y_ld, h_ld, z_ld, mod_ld, per;
    int T, K, rows, run;
    float alpha, beta;
};

// 8 elements as they lie in memory
template <bool BF16>
struct Raw { u4 v[BF16 ? 1 : 2]; };

template <bool BF16>
__device__ __forceinline__ Raw<BF16> load8(const void *p, int64_t at) {
    Raw<BF16> r;
    const u4 *q = reinterpret_cast<const u4 *>(static_cast<const char *>(p) + at * (BF16 ? 2 : 4));
    r.v[0] = q[0];
    if constexpr (!BF16) r.v[1] = q[1];
    return r;
}
template <bool BF16>
__device__ __forceinline__ void values(const Raw<BF16> &r, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
            const uint32_t p = r.v[0][i];
            f[2 * i] = lo_of(p);
            f[2 * i + 1] = hi_of(p);
        } else {
            const uint32_t a = r.v[0][i], b = r.v[1][i];
            f[i] = __builtin_bit_cast(float, a);
            f[4 + i] = __builtin_bit_cast(float, b);
        }
    }
}
template <bool BF16>
__device__ __forceinline__ void store8(void *p, int64_t at, const float (&f)[8]) {
    if constexpr (BF16)
        *reinterpret_cast<u4 *>(static_cast<uint16_t *>(p) + at) =
            u4{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
    else {
        store4<false>(p, at, f4{f[0], f[1], f[2], f[3]});
        store4<false>(p, at + 4, f4{f[4], f[5], f[6], f[7]});
    }
}

// WAVES waves take a token; a lane holds CH pieces of 8 of its values in registers,
// always the same channels, so that the modulations stay in registers while the
// tokens walk by (read again for each token they would be more bytes, from the caches,
// than the rows).  The next token's rows are on their way meanwhile.  Two waves a SIMD:
// with one, 8192 x 1152 took 25 us against 20, 32760 x 1536 132 against 130; three have
// too few registers (63 and 307).  They hold up to three pieces (at most 32 registers
// are spilled); with four, widths of 1537 to 2048, 6145 to 8192 and 12289 to 16384, 99 to
// 177 are, and come from scratch for every token: 33.5 M bf16 values of the stream, modulated
// and gated, take 88 us at a width of 2048, 94 at 8192 and 106 at 16384, against 57 at 1536,
// 56 at 4096 and 57 at 12288 (fp32: 170, 181, 180 against 116, 107, 117).  Rows of up to
// 2048 values take one wave and no barrier.  RB, IB: x and h, y and z are bf16 (else fp32).
template <bool RB, bool IB, int WAVES, int CH>
__global__ void __launch_bounds__(WAVES == 1 ? 256 : WAVES * 64) __attribute__((amdgpu_waves_per_eu(2))) block_norm_kernel(Args a) {
    constexpr int GROUPS = WAVES == 1 ? 4 : 1;   // tokens of a workgroup at a time
    __shared__ float s_sum[2][WAVES];
    const int lane = threadIdx.x % (WAVES * 64), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t group = (int64_t)blockIdx.x * GROUPS + (WAVES == 1 ? wave : 0);
    const int64_t t0 = group * a.run;
    if (t0 >= a.T) return;   // (whole waves; with WAVES > 1 whole workgroups)
    const int t1 = (int)min((int64_t)a.T, t0 + a.run);

    int buffer = 0;
    auto sum = [&](float x) {
        x = wave_sum(x);
        if constexpr (WAVES > 1) {
            if ((threadIdx.x & 63) == 0) s_sum[buffer][wave] = x;
            __syncthreads();
            x = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) x += s_sum[buffer][w];
            buffer ^= 1;   // (the next sum's barrier lies between these reads and the next writes here)
        }
        return x;
    };
    const float inv_k = 1.0f / (float)a.K;
    bool in[CH];
    int at[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        at[c] = (c * WAVES * 64 + lane) * 8;
        in[c] = at[c] < a.K;
    }
    // the mean off every value (layer norm), and the reciprocal root of the mean square
    auto normalize = [&](float (&f)[CH][8], const Norm &n) {
        if (n.kind == RQ_NORM_LAYER) {
            float s = 0.0f;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) s += f[c][i];
            const float mean = sum(s) * inv_k;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) f[c][i] = in[c] ? f[c][i] - mean : 0.0f;
        }
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(f[c][i], f[c][i], s);
        return 1.0f / sqrtf(sum(s) * inv_k + n.eps);
    };

    // z = pre(h) to_z + add_z and branch = post(y) to_h, the modulations, weights and beta multiplied out
    float to_h[CH][8], to_z[CH][8], add_z[CH][8];
    int row = -1;
    auto load_mod = [&](int r) {
        row = r;
        const bool ok = (uint32_t)r < (uint32_t)a.rows;
        const float none = ok ? 0.0f : NAN;
        const int64_t base = ok ? (int64_t)r * a.mod_ld : 0;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = in[c] ? at[c] : 0;
            float g[8], s[8], b[8], w[8];
            auto vec = [&](const float *p, int64_t from, float other, float (&v)[8]) {
                if (p) values<false>(load8<false>(p, from), v);
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = other;
            };
            vec(a.gate, base + k, 1.0f, g);
            vec(a.scale, base + k, 0.0f, s);
            vec(a.shift, base + k, 0.0f, b);
            vec(a.post.weight, k, 1.0f, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) to_h[c][i] = a.beta * (g[i] + (a.gate ? none : 0.0f)) * w[i];
            vec(a.pre.weight, k, 1.0f, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[i] = 1.0f + (s[i] + (a.scale ? none : 0.0f));
                to_z[c][i] = s[i] * w[i];
            }
            vec(a.pre.bias, k, 0.0f, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) add_z[c][i] = fmaf(w[i], s[i], b[i] + (a.shift ? none : 0.0f));
        }
    };
    Raw<RB> x[CH];
    Raw<IB> y[CH];
    auto load = [&](int t) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
            if (in[c]) x[c] = load8<RB>(a.x, t * a.x_ld + at[c]);
        if (a.y)
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (in[c]) y[c] = load8<IB>(a.y, t * a.y_ld + at[c]);
    };
    load((int)t0);
    int64_t turn = t0 / a.per;   // row by position, and the token at which it changes
    int64_t change = (turn + 1) * a.per;
    for (int t = (int)t0; t < t1; ++t) {
        if (t == change) {
            ++turn;
            change += a.per;
        }
        const int r = a.index ? a.index[t] : (int)turn;
        if (r != row || t == t0) load_mod(r);
        float h[CH][8], f[CH][8];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            values<RB>(x[c], h[c]);
            if (a.y) values<IB>(y[c], f[c]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[c][i] = in[c] ? h[c][i] * a.alpha : 0.0f;
                f[c][i] = in[c] && a.y ? f[c][i] : 0.0f;
            }
        }
        if (t + 1 < t1) load(t + 1);
        if (a.y) {
            const float n = a.post.kind >= 0 ? normalize(f, a.post) : 1.0f;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) h[c][i] = fmaf(f[c][i] * n, to_h[c][i], h[c][i]);
            if (a.post.bias) {   // (rare: not worth registers of its own)
                const bool ok = (uint32_t)r < (uint32_t)a.rows;
                for (int c = 0; c < CH; ++c)
                    for (int i = 0; i < 8; ++i)
                        if (in[c]) h[c][i] = fmaf(a.beta * (a.gate && ok ? a.gate[(int64_t)r * a.mod_ld + at[c] + i] : 1.0f),
                                                  a.post.bias[at[c] + i], h[c][i]);
            }
        }
        if (a.h)
#pragma unroll
            for (int c = 0; c < CH; ++c)
                if (in[c]) store8<RB>(a.h, t * a.h_ld + at[c], h[c]);
        if (!a.z) continue;
        const float n = a.pre.kind >= 0 ? normalize(h, a.pre) : 1.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] = fmaf(h[c][i] * n, to_z[c][i], add_z[c][i]);
            if (in[c]) store8<IB>(a.z, t * a.z_ld + at[c], h[c]);
        }
    }
}

}  // namespace

int launch_block_norm(const rq_norm *post, const rq_norm *pre, const rq_modulation *mod, int width,
                      const void *x, int x_bf16, int64_t x_ld, const void *y, int io_bf16, int64_t y_ld,
                      int64_t T, float alpha, float beta, void *h, int64_t h_ld, void *z, int64_t z_ld,
                      void *stream) {
    Args a{};
    auto take = [](const rq_norm *n) { return n ? Norm{n->weight, n->bias, n->eps, n->kind} : Norm{nullptr, nullptr, 0.0f, -1}; };
    a.post = take(post), a.pre = take(pre);
    a.rows = 1, a.per = T;
    if (mod) {
        a.gate = mod->gate, a.shift = mod->shift, a.scale = mod->scale, a.index = mod->index;
        a.rows = mod->rows, a.mod_ld = mod->ld;
        if (!mod->index) a.per = mod->per;
    }
    a.x = x, a.y = y, a.h = h, a.z = z;
    a.x_ld = x_ld, a.y_ld = y_ld, a.h_ld = h_ld, a.z_ld = z_ld;
    a.T = (int)T, a.K = width, a.alpha = alpha, a.beta = beta;
    hipStream_t s = static_cast<hipStream_t>(stream);
    auto go = [&](auto kern, int waves) {
        // (runs of tokens for twice the waves that are resident, or a wave where there are fewer)
        const int64_t most = (int64_t)device_cus() * (waves == 1 ? 16 : waves == 4 ? 4 : 2);
        a.run = (int)((T + most - 1) / most);
        const int64_t groups = (T + a.run - 1) / a.run, per_block = waves == 1 ? 4 : 1;
        hipLaunchKernelGGL(kern, dim3((unsigned)((groups + per_block - 1) / per_block)), dim3(waves == 1 ? 256 : waves * 64), 0, s, a);
    };
    auto sized = [&](auto rb, auto ib) {
        constexpr bool R = decltype(rb)::value, I = decltype(ib)::value;
        if (width <= 512) go(block_norm_kernel<R, I, 1, 1>, 1);
        else if (width <= 1024) go(block_norm_kernel<R, I, 1, 2>, 1);
        else if (width <= 1536) go(block_norm_kernel<R, I, 1, 3>, 1);
        else if (width <= 2048) go(block_norm_kernel<R, I, 1, 4>, 1);
        else if (width <= 4096) go(block_norm_kernel<R, I, 4, 2>, 4);
        else if (width <= 6144) go(block_norm_kernel<R, I, 4, 3>, 4);
        else if (width <= 8192) go(block_norm_kernel<R, I, 4, 4>, 4);
        else if (width <= 12288) go(block_norm_kernel<R, I, 8, 3>, 8);
        else go(block_norm_kernel<R, I, 8, 4>, 8);
    };
    if (x_bf16 && io_bf16) sized(std::true_type{}, std::true_type{});
    else if (x_bf16) sized(std::true_type{}, std::false_type{});
    else if (io_bf16) sized(std::false_type{}, std::true_type{});
    else sized(std::false_type{}, std::false_type{});
    return (int)hipGetLastError();
}

}  // namespace rq
