// rq_rows.hip -- attention of many query rows over the same keys: the tokens of a
// block over an encoder's states (or over each other), and a batch of single
// tokens over a prefix that its sequences share.
//
//   s_j = scale q . k_j;  lse = log sum exp s_j;  out = sum exp(s_j - lse) v_j
//
// Query heads that share a key-value head, of all query tokens, are the rows of
// one problem: row r is token r / G, head r % G.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "rq_attn_util.h"
#include "rq_internal.h"

namespace rq {
namespace {

using namespace attn;

typedef float f16 __attribute__((ext_vector_type(16)));
typedef short s4 __attribute__((ext_vector_type(4)));

// where keys and values come from
enum Source { STATES, PAGES, PAGES_I8 };

struct Args {
    Cache c;                       // pages (heads, D: always)
    const void *k, *v;             // states
    int64_t k_ld, k_stride, v_ld, v_stride;
    const void *q;
    void *out;
    const int32_t *lens, *q_lens;
    const uint8_t *mask;
    float *lse;
    float *part;                   // [parts][rows of all][D], unnormalized outputs
    float *stat;                   // [parts][rows of all][2], their maxima (base 2) and sums
    const int32_t *prefix_table;
    int64_t q_ld, q_stride, out_ld, out_stride, mask_ld;
    int64_t rows;                  // rows of all problems: batch * heads * queries * G
    int32_t batch, queries, keys, hq, G;
    int32_t tiles, splits;         // row tiles and parts of a problem
    int32_t prefix, own_splits;    // shared prefix
    float scale2, q_factor;        // |scale| * log2(e); the queries' sign (0 with scale 0)
};

// One workgroup's share of one problem.
struct Job {
    int64_t q_at, out_at;          // elements before token 0's row
    const char *k, *v;             // states: the head's token 0
    const int32_t *table;          // pages
    const uint8_t *mask;
    int h, R, row0;                // head; rows of the problem; first row of the tile
    int begin, end;                // slots
    int64_t part, lse_at;          // part * rows of all + the problem's row 0; lse of token 0, head 0 of the group
};

__device__ __forceinline__ f16 mfma32(u4 a, u4 b, f16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
}
__device__ __forceinline__ u2 read_turned(const uint16_t *p) {
    return __builtin_bit_cast(u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4 *)p));
}
// eight int8 codes -> eight bf16 (exact)
__device__ __forceinline__ u4 widen(u2 c) {
    u4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = c[i / 2] >> (16 * (i % 2));
        r[i] = pack2((float)(int8_t)x, (float)(int8_t)(x >> 8));
    }
    return r;
}

// NB blocks of 32 rows a wave, RW waves along the rows, TW along the tokens of a step.
template <int DP_, bool BF16_, int NB_, int RW_, int TW_, Source SRC_>
struct Shape {
    static constexpr int DP = DP_, NB = NB_, RW = RW_, TW = TW_;
    static constexpr bool BF16 = BF16_;
    static constexpr Source SRC = SRC_;
    static constexpr int threads = RW * TW * 64;
    static constexpr int rows = RW * NB * 32;
    static constexpr int TB = TW == 1 ? 2 : 1;            // blocks of 32 tokens a wave takes in a step
    static constexpr int KT = TW * TB * 32;               // tokens of a step
    static constexpr int KP = DP + 8, VP = DP + 16;       // elements from token to token in LDS: no two of the
                                                          // eight rows that are read together share a bank
    static constexpr int stage = KT * (KP + VP);          // elements of one buffer
    static constexpr int scale_floats = SRC == PAGES_I8 ? 2 * KT : 0;
    static constexpr size_t buffers = 2 * (stage * 2 + scale_floats * 4);
    static constexpr int OP = DP + 4;                     // joining waves: floats from row to row
    static constexpr size_t join = TW == 1 ? 0 : (size_t)TW * NB * 32 * (OP + 2) * 4;
    static constexpr size_t lds = buffers > join ? buffers : join;
};

// A step of KT tokens goes through LDS (asked for a step ahead, in registers), and
// each wave computes with v_mfma_f32_32x32x16_bf16
//   S [token][row] = K Q^T: a lane gets, of row lane % 32, the tokens
//     8 (i / 4) + 4 (lane / 32) + i % 4, i = 0 .. 15, of a block;
//   O^T [d][row] = V^T P^T: the lane's weights are the operand as they lie, its k
//     slots 8 (lane / 32) + e standing for the tokens above, and V^T is read in that
//     order with the transposing LDS read.
//
// Rounding: K, V and bf16 queries enter exactly, fp32 queries as three bf16 parts
// (24 bits).  Weights enter as bf16 for bf16 outputs and as three bf16 parts for
// fp32 ones; sums and statistics are fp32.
template <class C>
__device__ __forceinline__ void attend_rows(const Args &a, const Job &job, char *lds) {
    constexpr int DP = C::DP, NB = C::NB, KT = C::KT, TB = C::TB;
    constexpr bool BF16 = C::BF16, I8 = C::SRC == PAGES_I8, PAGED = C::SRC != STATES;
    constexpr int QP = BF16 ? 1 : 3;                  // parts of queries and weights
    constexpr int KS = DP / 16, DB = DP / 32;
    constexpr int PIECES = DP / 8, N = KT * PIECES / C::threads;
    static_assert(KT * PIECES % C::threads == 0, "whole pieces a thread");
    constexpr int EB = I8 ? 1 : 2;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rw = wave / C::TW, tw = wave % C::TW;
    const int col = lane & 31, hf = lane >> 5;
    const int D = a.c.D, G = a.G;

    // rows and queries
    int row[NB];
    u4 q[NB][KS][QP];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        row[nb] = job.row0 + (rw * NB + nb) * 32 + col;
        const int r = min(row[nb], job.R - 1), t = r / G, g = r - t * G;
        const int64_t at = job.q_at + t * a.q_ld + (int64_t)(job.h * G + g) * D;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const int d = ks * 16 + hf * 8;
            const bool in = d < D;
            if constexpr (BF16) {
                const u4 x = *reinterpret_cast<const u4 *>(static_cast<const uint16_t *>(a.q) + at + (in ? d : 0));
                q[nb][ks][0] = in ? x : u4{0, 0, 0, 0};
            } else {
                const float *p = static_cast<const float *>(a.q) + at + (in ? d : 0);
                const f4 x = *reinterpret_cast<const f4 *>(p), y = *reinterpret_cast<const f4 *>(p + 4);
                const float z[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t p3[3];
                    split2<3>(in ? z[2 * i] : 0.0f, in ? z[2 * i + 1] : 0.0f, p3);
#pragma unroll
                    for (int n = 0; n < QP; ++n) q[nb][ks][n][i] = p3[n];
                }
            }
        }
        if (a.q_factor != 1.0f) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int n = 0; n < QP; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t x = q[nb][ks][n][i];
                        q[nb][ks][n][i] = pack2(lo_of(x) * a.q_factor, hi_of(x) * a.q_factor);
                    }
        }
    }

    f16 o[NB][DB];
    float m[NB], l[NB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        m[nb] = -INFINITY;
        l[nb] = 0.0f;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[nb][db][i] = 0.0f;
    }

    // ---- staging.  All loads leave under no condition (what lies outside reads some
    // place inside), what must not count is cleared on the way to LDS.
    constexpr int PG = (KT + 63) / 64;
    int32_t page_of[PG];               // of slot j0 + 64 i + lane, a step ahead of the loads
    u4 kreg[N], vreg[N];               // int8: the first two dwords
    float ksreg = 0, vsreg = 0;        // int8: scales of slot j0 + thread
    uint32_t use[PG];                  // slot j0 + 64 i + lane: whether it counts
    const int page_mask = (1 << a.c.page_log) - 1;
    auto load_pages = [&](int j0) {
#pragma unroll
        for (int i = 0; i < PG; ++i) page_of[i] = job.table[min(j0 + i * 64 + lane, job.end - 1) >> a.c.page_log];
    };
    auto load = [&](int j0) {
#pragma unroll
        for (int i = 0; i < PG; ++i) {
            const int j = j0 + i * 64 + lane, jj = min(j, job.end - 1);
            use[i] = job.mask ? job.mask[jj] : 1;
            if (j >= job.end) use[i] = 0;
            if constexpr (PAGED) {
                if ((uint32_t)page_of[i] >= (uint32_t)a.c.pages) use[i] = 0, page_of[i] = 0;
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = i * C::threads + (int)threadIdx.x, t = u / PIECES, p = u - t * PIECES;
            const int j = min(j0 + t, job.end - 1), d = p * 8 < D ? p * 8 : 0;
            if constexpr (!PAGED) {
                kreg[i] = *reinterpret_cast<const u4 *>(job.k + (j * a.k_ld + d) * 2);
                vreg[i] = *reinterpret_cast<const u4 *>(job.v + (j * a.v_ld + d) * 2);
            } else {
                int32_t pg = __shfl(page_of[0], t & 63);
                if constexpr (PG > 1) pg = t >= 64 ? __shfl(page_of[PG - 1], t & 63) : pg;
                const int64_t r = (((int64_t)pg * a.c.heads + job.h) << a.c.page_log) + (j & page_mask);
                const char *kp = static_cast<const char *>(a.c.k) + (r * D + d) * EB, *vp = static_cast<const char *>(a.c.v) + (r * D + d) * EB;
                if constexpr (!I8) {
                    kreg[i] = *reinterpret_cast<const u4 *>(kp);
                    vreg[i] = *reinterpret_cast<const u4 *>(vp);
                } else {
                    const u2 x = *reinterpret_cast<const u2 *>(kp), y = *reinterpret_cast<const u2 *>(vp);
                    kreg[i] = u4{x[0], x[1], 0, 0};
                    vreg[i] = u4{y[0], y[1], 0, 0};
                }
            }
        }
        if constexpr (I8) {
            const int t = threadIdx.x % KT, j = min(j0 + t, job.end - 1);
            int32_t pg = __shfl(page_of[0], t & 63);
            if constexpr (PG > 1) pg = t >= 64 ? __shfl(page_of[PG - 1], t & 63) : pg;
            const int64_t r = (((int64_t)pg * a.c.heads + job.h) << a.c.page_log) + (j & page_mask);
            ksreg = a.c.k_scale[r];
            vsreg = a.c.v_scale[r];
        }
    };
    uint64_t bits[PG];                 // which slots of a step count
    auto stage = [&](int buf) {
        uint16_t *kl = reinterpret_cast<uint16_t *>(lds) + buf * C::stage, *vl = kl + KT * C::KP;
#pragma unroll
        for (int i = 0; i < PG; ++i) bits[i] = __ballot(use[i] != 0);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int u = i * C::threads + (int)threadIdx.x, t = u / PIECES, p = u - t * PIECES;
            uint64_t b = bits[0];
            if constexpr (PG > 1) b = t >= 64 ? bits[PG - 1] : b;
            const bool ok = (b >> (t & 63) & 1) != 0 && p * 8 < D;
            u4 x = kreg[i], y = vreg[i];
            if constexpr (I8) {
                x = widen(u2{x[0], x[1]});
                y = widen(u2{y[0], y[1]});
            }
            *reinterpret_cast<u4 *>(kl + t * C::KP + p * 8) = ok ? x : u4{0, 0, 0, 0};
            *reinterpret_cast<u4 *>(vl + t * C::VP + p * 8) = ok ? y : u4{0, 0, 0, 0};
        }
        if constexpr (I8) {
            float *sc = reinterpret_cast<float *>(lds + 2 * C::stage * 2) + buf * 2 * KT;
            if (threadIdx.x < KT) {
                const int t = threadIdx.x;
                uint64_t b = bits[0];
                if constexpr (PG > 1) b = t >= 64 ? bits[PG - 1] : b;
                const bool ok = (b >> (t & 63) & 1) != 0;
                sc[t] = ok ? ksreg : 0.0f;
                sc[KT + t] = ok ? vsreg : 0.0f;
            }
        }
    };

    if (job.begin < job.end) {
        if constexpr (PAGED) load_pages(job.begin);
        load(job.begin);
        if constexpr (PAGED) load_pages(job.begin + KT);
    }
    int buf = 0;
    for (int j0 = job.begin; j0 < job.end; j0 += KT, buf ^= 1) {
        stage(buf);
        if (j0 + KT < job.end) {
            load(j0 + KT);
            if constexpr (PAGED) load_pages(j0 + 2 * KT);
        }
        // the next write to this buffer is two steps away, behind the next step's barrier
        __syncthreads();
        const uint16_t *kl = reinterpret_cast<const uint16_t *>(lds) + buf * C::stage, *vl = kl + KT * C::KP;
        const int first = C::TW == 1 ? 0 : tw * 32;
        f16 s[NB][TB];
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[nb][tb][i] = 0.0f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const u4 k = *reinterpret_cast<const u4 *>(kl + (first + tb * 32 + col) * C::KP + ks * 16 + hf * 8);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int n = 0; n < QP; ++n) s[nb][tb] = mfma32(k, q[nb][ks][n], s[nb][tb]);
            }
        }
        // int8: the scales of the lane's tokens
        float ksc[TB][16], vsc[TB][16];
        if constexpr (I8) {
            const float *sc = reinterpret_cast<const float *>(lds + 2 * C::stage * 2) + buf * 2 * KT + first + hf * 4;
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const f4 x = *reinterpret_cast<const f4 *>(sc + tb * 32 + i * 2), y = *reinterpret_cast<const f4 *>(sc + KT + tb * 32 + i * 2);
#pragma unroll
                    for (int e = 0; e < 4; ++e) ksc[tb][i + e] = x[e], vsc[tb][i + e] = y[e];
                }
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) s[nb][tb][i] *= ksc[tb][i];
        }
        // slots that do not count
        uint32_t mine[TB];
        bool whole = true;
#pragma unroll
        for (int tb = 0; tb < TB; ++tb) {
            uint64_t b = bits[0];
            if constexpr (PG > 1) b = first + tb * 32 >= 64 ? bits[PG - 1] : b;
            mine[tb] = (uint32_t)(b >> ((first + tb * 32) & 63));
            whole = whole && mine[tb] == 0xffffffffu;
        }
        if (!whole) {
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
                const uint32_t b = mine[tb] >> (4 * hf);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float x = s[nb][tb][i];
                        s[nb][tb][i] = (b >> (8 * (i / 4) + i % 4) & 1) ? x : -INFINITY;
                    }
            }
        }
        // The running maximum only moves when a score passes it by 2^8: weights up to
        // 256 are as exact, and most steps leave the sums as they are.
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            float top = -INFINITY;
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, s[nb][tb][i]);
            top *= a.scale2;
            if (__any(top > m[nb] + 8.0f)) {
                top = fmaxf(fmaxf(top, __shfl_xor(top, 32)), m[nb]);
                const float f = top == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m[nb] - top);
                m[nb] = top;
                l[nb] *= f;
#pragma unroll
                for (int db = 0; db < DB; ++db) o[nb][db] *= f;
            }
            const float base = m[nb] == -INFINITY ? 0.0f : -m[nb];
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float p = __builtin_amdgcn_exp2f(fmaf(s[nb][tb][i], a.scale2, base));
                    l[nb] += p;
                    s[nb][tb][i] = I8 ? p * vsc[tb][i] : p;
                }
        }
#pragma unroll
        for (int tb = 0; tb < TB; ++tb)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                u4 p[NB][QP];
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t x[QP];
                        split2<QP>(s[nb][tb][half * 8 + 2 * i], s[nb][tb][half * 8 + 2 * i + 1], x);
#pragma unroll
                        for (int n = 0; n < QP; ++n) p[nb][n][i] = x[n];
                    }
                // (a lane's address is its part of the 4 tokens x 16 columns that 16 lanes turn)
                const uint16_t *vb = vl + (first + tb * 32 + half * 16 + 4 * hf + (lane & 15) / 4) * C::VP + (lane & 16) + (lane & 3) * 4;
#pragma unroll
                for (int db = 0; db < DB; ++db) {
                    const u2 x = read_turned(vb + db * 32), y = read_turned(vb + 8 * C::VP + db * 32);
                    const u4 v = {x[0], x[1], y[0], y[1]};
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int n = 0; n < QP; ++n) o[nb][db] = mfma32(v, p[nb][n], o[nb][db]);
                }
            }
    }

    // ---- the end: o of lane (col, hf) is d = 32 db + 8 (i / 4) + 4 hf + i % 4 of its row
    const bool parts = a.part != nullptr;
    auto put = [&](int r, int d, f4 x, float M, float L) {
        if (parts) {
            const int64_t at = job.part + r;
            if (M != -INFINITY) *reinterpret_cast<f4 *>(a.part + at * D + d) = x;
            if (d == 0) *reinterpret_cast<f2 *>(a.stat + at * 2) = f2{M, L};
            return;
        }
        const int t = r / G, g = r - t * G;
        const float inv = M == -INFINITY ? 0.0f : 1.0f / L;
        store4<BF16>(a.out, job.out_at + t * a.out_ld + (int64_t)(job.h * G + g) * D + d, x * inv);
        if (d == 0 && a.lse) a.lse[job.lse_at + (int64_t)t * a.hq + g] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * kLn2;
    };
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
        l[nb] += __shfl_xor(l[nb], 32);
        // A NaN score is in l, but maxima drop it.  A maximum of infinity takes it
        // through every join: exp2(inf - inf) is NaN, other parts count 0 beside it.
        if (l[nb] != l[nb]) m[nb] = INFINITY;
    }
    if constexpr (C::TW == 1) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
            if (row[nb] < job.R)
#pragma unroll
                for (int db = 0; db < DB; ++db)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int d = db * 32 + i * 8 + hf * 4;
                        if (d < D) put(row[nb], d, f4{o[nb][db][4 * i], o[nb][db][4 * i + 1], o[nb][db][4 * i + 2], o[nb][db][4 * i + 3]}, m[nb], l[nb]);
                    }
    } else {
        static_assert(C::TW == 1 || (NB == 1 && C::RW == 1), "waves along the tokens have the same 32 rows");
        __syncthreads();   // (the last step's LDS is read no more)
        float *so = reinterpret_cast<float *>(lds), *st = so + C::TW * 32 * C::OP;
        if (hf == 0) {
            st[(tw * 32 + col) * 2] = m[0];
            st[(tw * 32 + col) * 2 + 1] = l[0];
        }
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<f4 *>(so + (tw * 32 + col) * C::OP + db * 32 + i * 8 + hf * 4) =
                    f4{o[0][db][4 * i], o[0][db][4 * i + 1], o[0][db][4 * i + 2], o[0][db][4 * i + 3]};
        __syncthreads();
        const int rows = min(32, job.R - job.row0), quads = D / 4;
        for (int x = threadIdx.x; x < rows * quads; x += C::threads) {
            const int r = x / quads, d = (x - r * quads) * 4;
            float M = -INFINITY, L = 0.0f;
#pragma unroll
            for (int w = 0; w < C::TW; ++w) M = fmaxf(M, st[(w * 32 + r) * 2]);
            f4 sum = {0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < C::TW; ++w) {
                const float mw = st[(w * 32 + r) * 2];
                if (mw == -INFINITY) continue;
                const float f = __builtin_amdgcn_exp2f(mw - M);
                L += st[(w * 32 + r) * 2 + 1] * f;
                sum += *reinterpret_cast<const f4 *>(so + (w * 32 + r) * C::OP + d) * f;
            }
            put(job.row0 + r, d, sum, M, L);
        }
    }
}

// Keys of part `split`: equal shares in whole steps.
__device__ __forceinline__ void share(int begin, int end, int splits, int split, int step, int &b, int &e) {
    const int per = ((end - begin + splits - 1) / splits + step - 1) / step * step;
    b = min(begin + split * per, end);
    e = min(b + per, end);
}

// Workgroups go round the 8 XCDs in turn; consecutive jobs, which share keys, are
// given to the same one.
__device__ __forceinline__ int64_t job_of_block() {
    const int64_t n = gridDim.x, id = blockIdx.x, each = n / 8, more = n % 8, x = id % 8;
    return x * each + min(x, more) + id / 8;
}

template <class C>
__global__ void __launch_bounds__(C::threads) cross_kernel(Args a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    int64_t id = job_of_block();
    const int tile = (int)(id % a.tiles);
    id /= a.tiles;
    const int split = (int)(id % a.splits);
    id /= a.splits;
    const int h = (int)(id % a.c.heads), b = (int)(id / a.c.heads);
    Job job;
    job.h = h;
    const int queries = a.q_lens ? min(max(a.q_lens[b], 0), a.queries) : a.queries;
    job.R = queries * a.G;
    job.row0 = tile * C::rows;
    if (job.row0 >= job.R) return;
    const int keys = a.lens ? min(max(a.lens[b], 0), a.keys) : a.keys;
    share(0, keys, a.splits, split, C::KT, job.begin, job.end);
    job.q_at = b * a.q_stride;
    job.out_at = b * a.out_stride;
    job.k = static_cast<const char *>(a.k) + (b * a.k_stride + (int64_t)h * a.c.D) * 2;
    job.v = static_cast<const char *>(a.v) + (b * a.v_stride + (int64_t)h * a.c.D) * 2;
    job.table = nullptr;
    job.mask = a.mask ? a.mask + b * a.mask_ld : nullptr;
    job.part = split * a.rows + ((int64_t)b * a.c.heads + h) * a.queries * a.G;
    job.lse_at = (int64_t)b * a.queries * a.hq + h * a.G;
    attend_rows<C>(a, job, lds);
}

// The prefix (a problem a head, of all sequences' rows) and what each sequence
// holds behind it (a problem a sequence and head).
template <class C>
__global__ void __launch_bounds__(C::threads) prefix_kernel(Args a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    int64_t id = job_of_block();
    Job job;
    const int tile = (int)(id % a.tiles);
    id /= a.tiles;
    const int split = (int)(id % a.splits);
    job.h = (int)(id / a.splits);
    job.R = a.batch * a.G;
    job.row0 = tile * C::rows;
    share(0, a.prefix, a.splits, split, C::KT, job.begin, job.end);
    job.q_at = job.out_at = job.lse_at = 0;
    job.k = job.v = nullptr;
    job.table = a.prefix_table;
    job.mask = nullptr;
    job.part = split * a.rows + (int64_t)job.h * job.R;
    attend_rows<C>(a, job, lds);
}
template <class C>
__global__ void __launch_bounds__(C::threads) own_kernel(Args a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    int64_t id = blockIdx.x;
    const int tiles = (a.G + C::rows - 1) / C::rows;
    const int tile = (int)(id % tiles);
    id /= tiles;
    const int split = (int)(id % a.own_splits);
    id /= a.own_splits;
    const int h = (int)(id % a.c.heads), b = (int)(id / a.c.heads);
    Job job;
    job.h = h;
    job.R = a.G;
    job.row0 = tile * C::rows;
    share(a.prefix, max(a.prefix, min(a.lens[b], a.keys)), a.own_splits, split, C::KT, job.begin, job.end);
    job.q_at = b * a.q_ld;
    job.out_at = job.lse_at = 0;
    job.k = job.v = nullptr;
    job.table = a.c.table + (int64_t)b * a.c.table_ld;
    job.mask = a.mask ? a.mask + b * a.mask_ld : nullptr;
    job.part = (a.splits + split) * a.rows + ((int64_t)h * a.batch + b) * a.G;
    attend_rows<C>(a, job, lds);
}

constexpr int kJoin = 256;

// Joins the parts of a row, a wave a row.
template <bool BF16, bool PREFIX>
__global__ void __launch_bounds__(kJoin) join_rows_kernel(Args a) {
    const int lane = threadIdx.x & 63, D = a.c.D;
    const int64_t row = (int64_t)blockIdx.x * (kJoin / 64) + (threadIdx.x >> 6);
    if (row >= a.rows) return;
    int n = a.splits + a.own_splits;
    int64_t out_at, lse_at;
    if constexpr (PREFIX) {
        const int64_t hb = row / a.G;
        const int g = (int)(row - hb * a.G), h = (int)(hb / a.batch), b = (int)(hb - (int64_t)h * a.batch);
        if (min(a.lens[b], a.keys) < a.prefix || a.lens[b] <= 0) n = 0;   // not in the batch
        out_at = b * a.out_ld + (int64_t)(h * a.G + g) * D;
        lse_at = (int64_t)b * a.hq + h * a.G + g;
    } else {
        const int64_t rows = (int64_t)a.queries * a.G, bh = row / rows;
        const int r = (int)(row - bh * rows), t = r / a.G, g = r - t * a.G;
        const int b = (int)(bh / a.c.heads), h = (int)(bh - (int64_t)b * a.c.heads);
        if (a.q_lens && t >= a.q_lens[b]) return;
        out_at = b * a.out_stride + t * a.out_ld + (int64_t)(h * a.G + g) * D;
        lse_at = ((int64_t)b * a.queries + t) * a.hq + h * a.G + g;
    }
    const f2 *st = reinterpret_cast<const f2 *>(a.stat) + row;
    float M = -INFINITY, L = 0.0f;
    for (int i = lane; i < n; i += 64) M = fmaxf(M, st[i * a.rows][0]);
    M = wave_max(M);
    f4 sum = {0, 0, 0, 0};
    for (int i = 0; i < n; ++i) {
        const f2 x = st[i * a.rows];
        if (x[0] == -INFINITY) continue;
        const float f = __builtin_amdgcn_exp2f(x[0] - M);
        L += x[1] * f;
        if (lane < D / 4) sum += *reinterpret_cast<const f4 *>(a.part + (i * a.rows + row) * D + lane * 4) * f;
    }
    const float inv = M == -INFINITY ? 0.0f : 1.0f / L;
    if (lane < D / 4) store4<BF16>(a.out, out_at + lane * 4, sum * inv);
    if (lane == 0 && a.lse) a.lse[lse_at] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * kLn2;
}

// The kernel's shape for a number of rows: many rows divide over the waves, few
// leave the waves the tokens.
constexpr int kNarrow = 32;
int wide_nb(int DP, bool bf16) { return bf16 && DP <= 128 ? 2 : 1; }
int narrow_waves(int DP) { return DP <= 128 ? 4 : 2; }
int padded(int D) { return D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : 256; }
int rows_of(int DP, bool bf16, int64_t R) { return R <= kNarrow ? 32 : 128 * wide_nb(DP, bf16); }
int step_of(int DP, int64_t R) { return R <= kNarrow ? narrow_waves(DP) * 32 : 64; }

// Parts of a problem of `keys` where `jobs` workgroups take one each.
int parts_of(int64_t jobs, int64_t keys, int step) {
    const int64_t steps = (keys + step - 1) / step, most = 2 * device_cus();
    if (jobs >= device_cus() || jobs < 1) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>({steps, most / jobs, 64}));
}

template <class F>
void by_dim(int DP, F f) {
    if (DP == 64) f(std::integral_constant<int, 64>{});
    else if (DP == 96) f(std::integral_constant<int, 96>{});
    else if (DP == 128) f(std::integral_constant<int, 128>{});
    else f(std::integral_constant<int, 256>{});
}
template <int DP, bool B, Source S>
using Narrow = Shape<DP, B, 1, 1, DP <= 128 ? 4 : 2, S>;
template <int DP, bool B, Source S>
using Wide = Shape<DP, B, B && DP <= 128 ? 2 : 1, 4, 1, S>;

template <class C>
int go(void (*kern)(Args), int64_t grid, const Args &a, hipStream_t s) {
    const int err = ensure_dyn_lds(reinterpret_cast<const void *>(kern), C::lds);
    if (err != (int)hipSuccess) return err;
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(C::threads), C::lds, s, a);
    return (int)hipSuccess;
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

struct CrossPlan {
    int DP, tiles, splits;
    int64_t rows, grid;
    size_t part, stat;
};
CrossPlan cross_plan(const rq_states *s, int64_t queries, int q_heads, bool bf16) {
    CrossPlan p{};
    const int G = q_heads / s->heads;
    const int64_t R = queries * G;
    p.DP = padded(s->head_dim);
    const int rows = rows_of(p.DP, bf16, R);
    p.tiles = (int)((R + rows - 1) / rows);
    const int64_t jobs = (int64_t)p.tiles * s->heads * s->batch;
    p.splits = parts_of(jobs, s->keys, step_of(p.DP, R));
    p.grid = jobs * p.splits;
    p.rows = R * s->heads * s->batch;
    if (p.splits > 1) {
        p.part = round16((size_t)p.splits * p.rows * s->head_dim * 4);
        p.stat = round16((size_t)p.splits * p.rows * 8);
    }
    return p;
}

struct PrefixPlan {
    int DP, tiles, splits, own_splits;
    int64_t rows, grid, own_grid;
    size_t part, stat;
};
PrefixPlan prefix_plan(const rq_kv_cache *c, int q_heads, bool bf16, int64_t prefix, int64_t max_len) {
    PrefixPlan p{};
    const int G = q_heads / c->heads;
    const int64_t R = (int64_t)c->batch * G;
    p.DP = padded(c->head_dim);
    const int rows = rows_of(p.DP, bf16, R);
    p.tiles = (int)((R + rows - 1) / rows);
    if (prefix > 0) p.splits = parts_of((int64_t)p.tiles * c->heads, prefix, step_of(p.DP, R));
    p.grid = (int64_t)p.tiles * c->heads * p.splits;
    const int own_tiles = (G + 31) / 32;
    if (max_len > prefix) p.own_splits = parts_of((int64_t)own_tiles * c->heads * c->batch, max_len - prefix, step_of(p.DP, 1));
    p.own_grid = (int64_t)own_tiles * c->heads * c->batch * p.own_splits;
    p.rows = R * c->heads;
    const int parts = p.splits + p.own_splits;
    p.part = round16((size_t)parts * p.rows * c->head_dim * 4);
    p.stat = round16((size_t)parts * p.rows * 8);
    return p;
}

void set_scale(Args &a, float scale) {
    a.scale2 = scale == 0.0f ? 1.0f : std::fabs(scale) * 1.4426950408889634f;
    a.q_factor = scale == 0.0f ? 0.0f : scale < 0.0f ? -1.0f : 1.0f;
}

}  // namespace

bool cross_fits(const rq_states *s, int64_t queries, int q_heads, int bf16) {
    const CrossPlan p = cross_plan(s, queries, q_heads, bf16);
    // (a launch holds 2^32 threads)
    return p.grid < (1 << 24) && p.rows < (int64_t(1) << 25);
}
size_t cross_workspace_bytes(const rq_states *s, int64_t queries, int q_heads, int bf16) {
    const CrossPlan p = cross_plan(s, queries, q_heads, bf16);
    return p.part + p.stat;
}

int launch_cross_attention(const rq_states *st, const void *q, int bf16, int64_t q_ld, int64_t q_stride, int64_t queries,
                           int q_heads, float scale, const int32_t *q_lens, void *out, int64_t out_ld,
                           int64_t out_stride, float *lse, void *workspace, void *stream) {
    const CrossPlan p = cross_plan(st, queries, q_heads, bf16);
    Args a{};
    a.c.heads = st->heads, a.c.D = st->head_dim;
    a.k = st->k, a.v = st->v, a.k_ld = st->k_ld, a.k_stride = st->k_stride, a.v_ld = st->v_ld, a.v_stride = st->v_stride;
    a.lens = st->lens, a.mask = st->mask, a.mask_ld = st->mask_ld, a.keys = (int)st->keys;
    a.q = q, a.q_ld = q_ld, a.q_stride = q_stride, a.q_lens = q_lens, a.queries = (int)queries;
    a.out = out, a.out_ld = out_ld, a.out_stride = out_stride, a.lse = lse;
    a.batch = st->batch, a.hq = q_heads, a.G = q_heads / st->heads;
    a.tiles = p.tiles, a.splits = p.splits, a.rows = p.rows;
    set_scale(a, scale);
    if (p.splits > 1) {
        a.part = static_cast<float *>(workspace);
        a.stat = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.part);
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    int err = 0;
    auto run = [&](auto dp, auto b) {
        constexpr int DP = decltype(dp)::value;
        constexpr bool B = decltype(b)::value;
        if (queries * a.G <= kNarrow) err = go<Narrow<DP, B, STATES>>(cross_kernel<Narrow<DP, B, STATES>>, p.grid, a, s);
        else err = go<Wide<DP, B, STATES>>(cross_kernel<Wide<DP, B, STATES>>, p.grid, a, s);
    };
    by_dim(p.DP, [&](auto dp) { bf16 ? run(dp, std::true_type{}) : run(dp, std::false_type{}); });
    if (err != 0) return err;
    if (p.splits > 1)
        hipLaunchKernelGGL((bf16 ? join_rows_kernel<true, false> : join_rows_kernel<false, false>),
                           dim3((unsigned)((p.rows + kJoin / 64 - 1) / (kJoin / 64))), dim3(kJoin), 0, s, a);
    return (int)hipGetLastError();
}

bool prefix_fits(const rq_kv_cache *c, int q_heads, int bf16, int64_t prefix, int64_t max_len) {
    const PrefixPlan p = prefix_plan(c, q_heads, bf16, prefix, max_len);
    return p.grid < (1 << 24) && p.own_grid < (1 << 24) && p.rows < (int64_t(1) << 25);
}
size_t prefix_workspace_bytes(const rq_kv_cache *c, int q_heads, int bf16, int64_t prefix, int64_t max_len) {
    const PrefixPlan p = prefix_plan(c, q_heads, bf16, prefix, max_len);
    return p.part + p.stat;
}

int launch_prefix_attention(const rq_kv_cache *c, const int32_t *prefix_table, int64_t prefix, const void *q, int bf16,
                            int64_t q_ld, int q_heads, float scale, const int32_t *lens, int64_t max_len,
                            const uint8_t *mask, int64_t mask_ld, void *out, int64_t out_ld, float *lse,
                            void *workspace, void *stream) {
    const PrefixPlan p = prefix_plan(c, q_heads, bf16, prefix, max_len);
    Args a{};
    a.c = device_cache(c);
    a.lens = lens, a.mask = mask, a.mask_ld = mask_ld, a.keys = (int)max_len;
    a.q = q, a.q_ld = q_ld, a.out = out, a.out_ld = out_ld, a.lse = lse;
    a.batch = c->batch, a.hq = q_heads, a.G = q_heads / c->heads;
    a.tiles = p.tiles, a.splits = p.splits, a.own_splits = p.own_splits, a.rows = p.rows;
    a.prefix = (int)prefix, a.prefix_table = prefix_table;
    set_scale(a, scale);
    a.part = static_cast<float *>(workspace);
    a.stat = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.part);
    hipStream_t s = static_cast<hipStream_t>(stream);
    int err = 0;
    auto run = [&](auto dp, auto b, auto src) {
        constexpr int DP = decltype(dp)::value;
        constexpr bool B = decltype(b)::value;
        constexpr Source S = decltype(src)::value;
        using N = Narrow<DP, B, S>;
        using W = Wide<DP, B, S>;
        if (p.grid > 0) {
            if ((int64_t)a.batch * a.G <= kNarrow) err = go<N>(prefix_kernel<N>, p.grid, a, s);
            else err = go<W>(prefix_kernel<W>, p.grid, a, s);
        }
        if (err == 0 && p.own_grid > 0) err = go<N>(own_kernel<N>, p.own_grid, a, s);
    };
    by_dim(p.DP, [&](auto dp) {
        auto typed = [&](auto b) {
            if (c->dtype == RQ_I8) run(dp, b, std::integral_constant<Source, PAGES_I8>{});
            else run(dp, b, std::integral_constant<Source, PAGES>{});
        };
        bf16 ? typed(std::true_type{}) : typed(std::false_type{});
    });
    if (err != 0) return err;
    hipLaunchKernelGGL((bf16 ? join_rows_kernel<true, true> : join_rows_kernel<false, true>),
                       dim3((unsigned)((p.rows + kJoin / 64 - 1) / (kJoin / 64))), dim3(kJoin), 0, s, a);
    return (int)hipGetLastError();
}

}  // namespace rq
