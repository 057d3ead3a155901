// rq_attend.hip -- attention of one new token per sequence over a paged cache.
//
//   s_j = scale q . k_j;  lse = log sum exp s_j;  out = sum exp(s_j - lse) v_j
//
// The cache is read once and nothing else is large, so HBM bounds it.  The
// length is split into chunks, one workgroup per (chunk, key-value head,
// sequence), joined by a second kernel where there is more than one chunk.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "rq_attn_util.h"
#include "rq_internal.h"

namespace rq {
namespace {

using attn::Cache;

typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));

struct Args {
    Cache c;
    const void *q;
    void *out;
    const int32_t *lens;
    const uint8_t *mask;
    const float *weight;
    float *lse, *weight_out;
    float *scores;   // [batch][q heads][score_ld], base-2 scores (tracked calls)
    float *part;     // [batch][q heads][splits][D], unnormalized outputs of the chunks
    float *stat;     // [batch][q heads][splits][2], their maxima and sums
    int64_t q_ld, out_ld, mask_ld;
    int32_t hq, G, max_len, chunk, splits, score_ld;
    float scale2;    // scale * log2(e)
};

constexpr int kWaves = 4;      // waves of a workgroup
constexpr int kTile = 32;      // tokens of one wave's step

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const f2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, b2));
}
__device__ __forceinline__ float lo_of(uint32_t p) { return __builtin_bit_cast(float, p << 16); }
__device__ __forceinline__ float hi_of(uint32_t p) { return __builtin_bit_cast(float, p & 0xffff0000u); }
__device__ __forceinline__ f4 mfma(u4 a, u4 b, f4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
}
// the largest of the lanes l, l ^ 16, l ^ 32, l ^ 48, in all four
__device__ __forceinline__ float max_of_four(float x) {
    x = fmaxf(x, __shfl_xor(x, 16));
    return fmaxf(x, __shfl_xor(x, 32));
}
// four int8 codes -> four bf16 (exact)
__device__ __forceinline__ u2 widen4(uint32_t c) {
    const float a = (float)(int8_t)c, b = (float)(int8_t)(c >> 8), d = (float)(int8_t)(c >> 16), e = (float)((int32_t)c >> 24);
    return u2{pack2(a, b), pack2(d, e)};
}
__device__ __forceinline__ u4 widen8(u2 c) {
    const u2 a = widen4(c[0]), b = widen4(c[1]);
    return u4{a[0], a[1], b[0], b[1]};
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

// One chunk of one (sequence, key-value head, tile of 16 query heads).
//
// A wave takes 32 tokens a step, straight from memory into the operands of
// v_mfma_f32_16x16x32_bf16, with no LDS:
//   S [token][head] = K Q^T: lane (m, g4) = (lane % 16, lane / 16) loads 16-byte
//     pieces of token m's key, the order of d being free as long as Q has the same;
//   the result lies in lane (head, g4) for tokens 4 g4 .. 4 g4 + 3 of each half
//     of the step, which are the 8 tokens that this lane feeds to
//   O^T [d][head] = V^T P^T as k of its slice g4: P needs no exchange between
//     lanes.  Lane (m, g4) loads the same 8 tokens' values, W = 8 (4 for D <= 64)
//     d at W m each; v_perm pairs tokens, and product j covers d = W m + j.
// The 16 columns are query heads of one key-value head; fewer leave columns
// unused, at no cost next to the loads.
//
// Rounding: K, V and bf16 queries enter exactly; fp32 queries as three bf16
// parts (24 bits).  Weights enter as two bf16 parts (2^-17) for bf16 outputs
// and three for fp32: with one part their rounding would be as large as the
// output's own.  Sums and statistics are fp32.
template <int DP, bool EXACT, bool I8, bool BF16, bool MASKED, bool TRACK>
__global__ void __launch_bounds__(kWaves * 64) attend_kernel(Args a) {
    constexpr int QP = BF16 ? 1 : 3, PP = BF16 ? 2 : 3;
    constexpr int KS = DP / 32;                  // products along d
    constexpr int W = DP == 64 ? 4 : 8;          // d of one value load
    constexpr int NU = DP / (16 * W);            // value loads of a token
    __shared__ float s_m[kWaves][16], s_l[kWaves][16];
    __shared__ float s_o[kWaves][16][DP + 4];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g4 = lane >> 4;
    const int tiles = (a.G + 15) / 16;
    const int h = blockIdx.y / tiles, g0 = (blockIdx.y % tiles) * 16, b = blockIdx.z, sp = blockIdx.x;
    const int len = min(max(a.lens[b], 0), a.max_len);
    const int begin = sp * a.chunk, end = min(len, begin + a.chunk);
    if (begin >= len && a.splits > 1) return;
    const int D = EXACT ? DP : a.c.D;
    const int heads = min(16, a.G - g0);
    const int64_t head0 = (int64_t)b * a.hq + h * a.G + g0;

    // queries: piece s of lane (head, g4) holds d_of(s) .. + 7
    auto d_of = [&](int s) { return I8 && EXACT ? (s >> 1) * 64 + g4 * 16 + (s & 1) * 8 : s * 32 + g4 * 8; };
    u4 q[QP][KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const int d = d_of(s);
        const bool in = col < heads && (EXACT || d < D);
        const int64_t at = (int64_t)b * a.q_ld + (int64_t)(h * a.G + g0 + (in ? col : 0)) * D + (in ? d : 0);
        if constexpr (BF16) {
            u4 v = *reinterpret_cast<const u4 *>(static_cast<const uint16_t *>(a.q) + at);
            q[0][s] = in ? v : u4{0, 0, 0, 0};
        } else {
            const f4 x = *reinterpret_cast<const f4 *>(static_cast<const float *>(a.q) + at);
            const f4 y = *reinterpret_cast<const f4 *>(static_cast<const float *>(a.q) + at + 4);
            const float z[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t p[3];
                split2<3>(in ? z[2 * i] : 0.0f, in ? z[2 * i + 1] : 0.0f, p);
                q[0][s][i] = p[0];
                q[QP - 2 < 0 ? 0 : 1][s][i] = p[1];
                q[QP - 1][s][i] = p[2];
            }
        }
    }

    f4 o[NU][W];
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int j = 0; j < W; ++j) o[u][j] = f4{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;

    constexpr int EB = I8 ? 1 : 2;   // bytes of an element
    const int steps = (end - begin + kWaves * kTile - 1) / (kWaves * kTile);
    const int page_mask = (1 << a.c.page_log) - 1;

    // the pages of this wave's next 32 steps: lane 2 i + half
    int32_t page_of = -1;
    auto load_pages = [&](int step) {
        const int j = begin + ((step + (lane >> 1)) * kWaves + wave) * kTile + (lane & 1) * 16;
        const int idx = j >> a.c.page_log;
        page_of = j < end ? a.c.table[(int64_t)b * a.c.table_ld + idx] : -1;
    };
    // base row of half `hf` of a step; `there`: whether it has a page
    auto row_of = [&](int step, int hf, bool &there) -> int64_t {
        const int j = begin + (step * kWaves + wave) * kTile + hf * 16;
        const int32_t pg = __builtin_amdgcn_readlane(page_of, (step & 31) * 2 + hf);
        there = (uint32_t)pg < (uint32_t)a.c.pages;
        return (((int64_t)(there ? pg : 0) * a.c.heads + h) << a.c.page_log) + (j & page_mask);
    };

    u4 kreg[2][KS];
    u4 vreg[8][NU];       // bf16: W / 2 dwords used; int8: W / 4
    f4 ks[2], vs[2];
    bool there[2], v_there[2];

    auto load_k = [&](int step) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int64_t row = row_of(step, hf, there[hf]);
            const char *base = static_cast<const char *>(a.c.k) + row * (D * EB);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const int d = d_of(s);
                const char *p = base + col * (D * EB) + d * EB;
                if constexpr (!I8) {
                    if (EXACT || d < D) kreg[hf][s] = *reinterpret_cast<const u4 *>(p);
                    else kreg[hf][s] = u4{0, 0, 0, 0};
                } else if constexpr (EXACT) {
                    if (s % 2 == 0) kreg[hf][s / 2] = *reinterpret_cast<const u4 *>(p);
                } else {
                    u2 c = {0, 0};
                    if (d < D) c = *reinterpret_cast<const u2 *>(p);
                    kreg[hf][s][0] = c[0];
                    kreg[hf][s][1] = c[1];
                }
            }
            if constexpr (I8) ks[hf] = *reinterpret_cast<const f4 *>(a.c.k_scale + row + g4 * 4);
        }
    };
    auto load_v = [&](int step) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            const int64_t row = row_of(step, hf, v_there[hf]);
            const char *base = static_cast<const char *>(a.c.v) + row * (D * EB);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int u = 0; u < NU; ++u) {
                    int d = W * col + 16 * W * u;
                    if (!EXACT && d >= D) d = 0;   // (columns of the product that nobody reads)
                    const char *p = base + (g4 * 4 + i) * (D * EB) + d * EB;
                    u4 &r = vreg[hf * 4 + i][u];
                    if constexpr (W * EB == 16) r = *reinterpret_cast<const u4 *>(p);
                    else if constexpr (W * EB == 8) {
                        const u2 x = *reinterpret_cast<const u2 *>(p);
                        r[0] = x[0];
                        r[1] = x[1];
                    } else r[0] = *reinterpret_cast<const uint32_t *>(p);
                }
            if constexpr (I8) vs[hf] = *reinterpret_cast<const f4 *>(a.c.v_scale + row + g4 * 4);
        }
    };

    auto mine = [&](int step) { return begin + (step * kWaves + wave) * kTile < end; };   // wave-uniform
    if (mine(0)) {
        load_pages(0);
        load_k(0);
        load_v(0);
    }
    for (int step = 0; step < steps && mine(step); ++step) {
        const int j0 = begin + (step * kWaves + wave) * kTile;
        const bool more = step + 1 < steps && mine(step + 1);
        // scores: lane (head col, g4) gets tokens j0 + 16 hf + 4 g4 + i
        f4 s[2];
        bool ok[2] = {there[0], there[1]};
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
            s[hf] = f4{0, 0, 0, 0};
#pragma unroll
            for (int t = 0; t < KS; ++t) {
                u4 k;
                if constexpr (!I8) k = kreg[hf][t];
                else if constexpr (EXACT) k = widen8(t & 1 ? u2{kreg[hf][t / 2][2], kreg[hf][t / 2][3]} : u2{kreg[hf][t / 2][0], kreg[hf][t / 2][1]});
                else k = widen8(u2{kreg[hf][t][0], kreg[hf][t][1]});
#pragma unroll
                for (int p = 0; p < QP; ++p) s[hf] = mfma(k, q[p][t], s[hf]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[hf][i] *= a.scale2;
                if constexpr (I8) s[hf][i] *= ks[hf][i];
            }
        }
        const bool v_ok[2] = {v_there[0], v_there[1]};
        if (more) {
            if (((step + 1) & 31) == 0) load_pages(step + 1);
            load_k(step + 1);
        }
        // tokens that are left out
        bool whole = j0 + kTile <= end && ok[0] && ok[1] && !MASKED;
        bool use[2][4];
        if (!whole) {
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = j0 + hf * 16 + g4 * 4 + i;
                    use[hf][i] = ok[hf] && j < end;
                    if constexpr (MASKED) {
                        if (use[hf][i]) use[hf][i] = a.mask[(int64_t)b * a.mask_ld + j] != 0;
                    }
                    if (!use[hf][i]) s[hf][i] = -INFINITY;
                }
        }
        if constexpr (TRACK) {
            if (col < heads)
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                    *reinterpret_cast<f4 *>(a.scores + (head0 + col) * a.score_ld + j0 + hf * 16 + g4 * 4) = s[hf];
        }
        // The running maximum only moves when a score passes it by 2^8: weights
        // up to 256 are as exact, and most steps leave the sums as they are.
        float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                          fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
        if (__any(top > m + 8.0f)) {
            top = fmaxf(max_of_four(top), m);
            const float f = top == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - top);
            m = top;
            l *= f;
#pragma unroll
            for (int u = 0; u < NU; ++u)
#pragma unroll
                for (int j = 0; j < W; ++j) o[u][j] *= f;
        }
        const float base = m == -INFINITY ? 0.0f : m;
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            p[i] = __builtin_amdgcn_exp2f(s[i / 4][i % 4] - base);
            l += p[i];
            if constexpr (I8) p[i] *= vs[i / 4][i % 4];
        }
        if (!whole) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (!use[i / 4][i % 4]) {
                    p[i] = 0.0f;                       // (the scale may be anything)
#pragma unroll
                    for (int u = 0; u < NU; ++u) vreg[i][u] = u4{0, 0, 0, 0};
                }
        }
        u4 pp[PP];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t x[PP];
            split2<PP>(p[2 * i], p[2 * i + 1], x);
#pragma unroll
            for (int n = 0; n < PP; ++n) pp[n][i] = x[n];
        }
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            u4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if constexpr (!I8) v[i] = vreg[i][u];
                else if constexpr (W == 8) v[i] = widen8(u2{vreg[i][u][0], vreg[i][u][1]});
                else {
                    const u2 x = widen4(vreg[i][u][0]);
                    v[i] = u4{x[0], x[1], 0, 0};
                }
            }
#pragma unroll
            for (int j = 0; j < W; ++j) {
                u4 t;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    t[i] = __builtin_amdgcn_perm(v[2 * i + 1][j / 2], v[2 * i][j / 2], j & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
                for (int n = 0; n < PP; ++n) o[u][j] = mfma(t, pp[n], o[u][j]);
            }
        }
        (void)v_ok;
        if (more) load_v(step + 1);
    }

    // join the waves: o of lane (head col, g4) is d = W (4 g4 + i) + 16 W u + j
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (g4 == 0) {
        s_m[wave][col] = m;
        s_l[wave][col] = l;
    }
    __syncthreads();
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) M = fmaxf(M, s_m[w][col]);
    const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - M);
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) s_o[wave][col][W * (4 * g4 + i) + 16 * W * u + j] = o[u][j][i] * f;
    __syncthreads();
    for (int x = threadIdx.x; x < heads * (D / 4); x += kWaves * 64) {
        const int g = x / (D / 4), d = (x - g * (D / 4)) * 4;
        f4 r = {0, 0, 0, 0};
        float mm = -INFINITY, ll = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, s_m[w][g]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float *po = &s_o[w][g][d];
            r += f4{po[0], po[1], po[2], po[3]};
            if (s_m[w][g] != -INFINITY) ll += s_l[w][g] * __builtin_amdgcn_exp2f(s_m[w][g] - mm);
        }
        if (a.splits > 1) {
            *reinterpret_cast<f4 *>(a.part + ((head0 + g) * a.splits + sp) * D + d) = r;
            if (d == 0) {
                float *st = a.stat + ((head0 + g) * a.splits + sp) * 2;
                st[0] = mm;
                st[1] = ll;
            }
        } else {
            const float inv = mm == -INFINITY ? 0.0f : 1.0f / ll;
            const int64_t at = (int64_t)b * a.out_ld + (int64_t)(h * a.G + g0 + g) * D + d;
            if constexpr (BF16)
                *reinterpret_cast<u2 *>(static_cast<uint16_t *>(a.out) + at) = u2{pack2(r[0] * inv, r[1] * inv), pack2(r[2] * inv, r[3] * inv)};
            else
                *reinterpret_cast<f4 *>(static_cast<float *>(a.out) + at) = r * inv;
            if (d == 0) {
                if (a.lse) a.lse[head0 + g] = mm == -INFINITY ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994531f;
                if (TRACK) {
                    a.stat[(head0 + g) * 2] = mm;
                    a.stat[(head0 + g) * 2 + 1] = ll;
                }
            }
        }
    }
}

// Statistics of a head over its chunks, by one wave: all lanes get the maximum
// and the sum relative to it.
__device__ __forceinline__ void join_stats(const float *st, int n, int lane, float &M, float &L) {
    M = -INFINITY;
    for (int i = lane; i < n; i += 64) M = fmaxf(M, st[2 * i]);
    for (int o = 1; o < 64; o *= 2) M = fmaxf(M, __shfl_xor(M, o));
    L = 0.0f;
    for (int i = lane; i < n; i += 64)
        if (st[2 * i] != -INFINITY) L += st[2 * i + 1] * __builtin_amdgcn_exp2f(st[2 * i] - M);
    for (int o = 1; o < 64; o *= 2) L += __shfl_xor(L, o);
}

// Joins the chunks: block x < q heads writes the output of head x; the others
// add the weights of 1024 slots of one key-value head.
template <bool BF16>
__global__ void __launch_bounds__(256) join_kernel(Args a) {
    __shared__ float s_o[4][256];
    __shared__ float s_m[64], s_i[64];
    const int b = blockIdx.y, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, D = a.c.D;
    const int len = min(max(a.lens[b], 0), a.max_len);
    const int n = min(a.splits, (len + a.chunk - 1) / a.chunk);
    const int outs = a.splits > 1 ? a.hq : 0;
    if ((int)blockIdx.x < outs) {
        const int i = blockIdx.x;
        const int64_t head = (int64_t)b * a.hq + i;
        const float *st = a.stat + head * a.splits * 2;
        float M, L;
        join_stats(st, n, lane, M, L);
        f4 r = {0, 0, 0, 0};
        if (lane * 4 < D)
            for (int s = wave; s < n; s += 4) {
                const float m = st[2 * s];
                if (m == -INFINITY) continue;
                r += *reinterpret_cast<const f4 *>(a.part + (head * a.splits + s) * D + lane * 4) * __builtin_amdgcn_exp2f(m - M);
            }
        *reinterpret_cast<f4 *>(&s_o[wave][lane * 4]) = r;
        __syncthreads();
        if (wave == 0 && lane * 4 < D) {
            const float inv = M == -INFINITY ? 0.0f : 1.0f / L;
            for (int w = 1; w < 4; ++w) r += *reinterpret_cast<const f4 *>(&s_o[w][lane * 4]);
            const int64_t at = (int64_t)b * a.out_ld + (int64_t)i * D + lane * 4;
            if constexpr (BF16)
                *reinterpret_cast<u2 *>(static_cast<uint16_t *>(a.out) + at) = u2{pack2(r[0] * inv, r[1] * inv), pack2(r[2] * inv, r[3] * inv)};
            else
                *reinterpret_cast<f4 *>(static_cast<float *>(a.out) + at) = r * inv;
            if (lane == 0 && a.lse) a.lse[head] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
        }
        return;
    }
    const int blocks = (a.max_len + 1023) / 1024;
    const int x = blockIdx.x - outs, h = x / blocks, j = (x - h * blocks) * 1024 + threadIdx.x * 4;
    if ((x - h * blocks) * 1024 >= len) return;
    const int64_t head0 = (int64_t)b * a.hq + (int64_t)h * a.G;
    f4 w = {0, 0, 0, 0};
    for (int g0 = 0; g0 < a.G; g0 += 64) {
        const int gn = min(64, a.G - g0);
        __syncthreads();
        for (int g = wave; g < gn; g += 4) {
            float M, L;
            join_stats(a.stat + (head0 + g0 + g) * a.splits * 2, n, lane, M, L);
            if (lane == 0) {
                s_m[g] = M == -INFINITY ? 0.0f : M;
                s_i[g] = M == -INFINITY ? 0.0f : 1.0f / L;
            }
        }
        __syncthreads();
        if (j < len)
            for (int g = 0; g < gn; ++g) {
                const f4 s = *reinterpret_cast<const f4 *>(a.scores + (head0 + g0 + g) * a.score_ld + j);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] += __builtin_amdgcn_exp2f(s[e] - s_m[g]) * s_i[g];
            }
    }
    const int64_t at = ((int64_t)b * a.c.heads + h) * a.c.slots() + j;
    for (int e = 0; e < 4; ++e)
        if (j + e < len) a.weight_out[at + e] = a.weight[at + e] + w[e];
}

// Chunks of a call: enough workgroups for the device, but not shorter than one
// step of every wave.
struct Plan {
    int chunk, splits, score_ld;
    size_t part, stat, scores;   // bytes
};
Plan plan_of(const rq_kv_cache *c, int q_heads, int64_t max_len, int track) {
    Plan p;
    const int G = q_heads / c->heads;
    const int64_t rows = (int64_t)c->batch * c->heads * ((G + 15) / 16);
    const int64_t step = kWaves * kTile;
    const int64_t want = std::max<int64_t>(1, (4 * (int64_t)device_cus() + rows - 1) / std::max<int64_t>(rows, 1));
    int64_t chunk = (max_len + want - 1) / want;
    chunk = std::max(step, (chunk + step - 1) / step * step);
    p.chunk = (int)chunk;
    p.splits = (int)std::max<int64_t>(1, (max_len + chunk - 1) / chunk);
    p.score_ld = (int)((max_len + kTile - 1) / kTile * kTile);
    const size_t heads = (size_t)c->batch * q_heads;
    auto round = [](size_t n) { return (n + 15) / 16 * 16; };
    p.part = p.splits > 1 ? round(heads * p.splits * c->head_dim * 4) : 0;
    p.stat = p.splits > 1 || track ? round(heads * p.splits * 8) : 0;
    p.scores = track ? round(heads * p.score_ld * 4) : 0;
    return p;
}

}  // namespace

size_t attend_workspace_bytes(const rq_kv_cache *c, int q_heads, int64_t max_len, int track) {
    const Plan p = plan_of(c, q_heads, max_len, track);
    return p.part + p.stat + p.scores;
}

int launch_paged_attention(const rq_kv_cache *c, const void *q, int bf16, int64_t q_ld, int q_heads,
                           float scale, const int32_t *lens, int64_t max_len, const uint8_t *mask,
                           int64_t mask_ld, void *out, int64_t out_ld, float *lse, int track,
                           float *weight_out, void *workspace, void *stream) {
    const Plan p = plan_of(c, q_heads, max_len, track);
    Args a{};
    a.c = device_cache(c);
    a.q = q, a.out = out, a.lens = lens, a.mask = mask, a.lse = lse;
    a.weight = c->weight, a.weight_out = weight_out;
    char *ws = static_cast<char *>(workspace);
    a.part = reinterpret_cast<float *>(ws);
    a.stat = reinterpret_cast<float *>(ws + p.part);
    a.scores = reinterpret_cast<float *>(ws + p.part + p.stat);
    a.q_ld = q_ld, a.out_ld = out_ld, a.mask_ld = mask_ld;
    a.hq = q_heads, a.G = q_heads / c->heads, a.max_len = (int)max_len;
    a.chunk = p.chunk, a.splits = p.splits, a.score_ld = p.score_ld;
    a.scale2 = scale * 1.4426950408889634f;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const dim3 grid(p.splits, c->heads * ((a.G + 15) / 16), c->batch);
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(kWaves * 64), 0, s, a); };
    auto pick = [&](auto dp, auto exact, auto i8, auto io) {
        constexpr int DP = decltype(dp)::value;
        constexpr bool E = decltype(exact)::value, I = decltype(i8)::value, B = decltype(io)::value;
        if (mask) {
            if (track) go(attend_kernel<DP, E, I, B, true, true>);
            else go(attend_kernel<DP, E, I, B, true, false>);
        } else {
            if (track) go(attend_kernel<DP, E, I, B, false, true>);
            else go(attend_kernel<DP, E, I, B, false, false>);
        }
    };
    auto types = [&](auto dp, auto exact) {
        const bool i8 = c->dtype == RQ_I8;
        if (i8 && bf16) pick(dp, exact, std::true_type{}, std::true_type{});
        else if (i8) pick(dp, exact, std::true_type{}, std::false_type{});
        else if (bf16) pick(dp, exact, std::false_type{}, std::true_type{});
        else pick(dp, exact, std::false_type{}, std::false_type{});
    };
    auto dims = [&](auto dp) {
        if (c->head_dim == decltype(dp)::value) types(dp, std::true_type{});
        else types(dp, std::false_type{});
    };
    if (c->head_dim <= 64) dims(std::integral_constant<int, 64>{});
    else if (c->head_dim <= 128) dims(std::integral_constant<int, 128>{});
    else dims(std::integral_constant<int, 256>{});
    const int weights = track ? (int)((max_len + 1023) / 1024) * c->heads : 0;
    const int outs = p.splits > 1 ? q_heads : 0;
    if (outs + weights > 0) {
        const dim3 jg(outs + weights, c->batch);
        if (bf16) hipLaunchKernelGGL(join_kernel<true>, jg, dim3(256), 0, s, a);
        else hipLaunchKernelGGL(join_kernel<false>, jg, dim3(256), 0, s, a);
    }
    return (int)hipGetLastError();
}

}  // namespace rq
