// rq_attend.hip -- attention of one new token per sequence over a paged cache.
//
//   s_j = scale q . k_j;  lse = log sum exp s_j;  out = sum exp(s_j - lse) v_j
//
// The cache is read once and nothing else is large, so HBM bounds it: 131071
// tokens of 8 heads x 128 in bf16 (537 MB) take 95 us, 5.7 TB/s, where a plain
// read of as much takes 87 us; 262143 tokens in int8 110 us with the joining, 5.0
// TB/s.  The matrix cores are 5% busy; they are there because 4 to 16 query heads a key
// would keep the vector units too busy to issue the loads.
//
// The tokens of all sequences are dealt out to the workgroups in equal shares, and
// a second kernel joins the parts of rows (7 us for 131071 tokens); short calls, and
// calls of many short rows, take one workgroup a row and no second kernel.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "rq_attn_util.h"
#include "rq_internal.h"

namespace rq {
namespace {

using namespace attn;

struct Args {
    Cache c;
    const void *q;
    void *out;
    const int32_t *lens;
    const uint8_t *mask;
    const float *weight;
    float *lse, *weight_out;
    float *scores;   // [rows][score_ld / 16][heads of a tile][16 slots], base-2 scores (tracked calls):
                     // what a wave's store writes lies together
    float *part;     // [workgroups + rows][heads of a tile][D], unnormalized outputs
    float *stat;     // [workgroups + rows][heads of a tile][2], their maxima and sums
    int32_t *ends;   // [rows][2]: the first and the last workgroup of a row with tokens
    int64_t q_ld, out_ld, mask_ld;
    int32_t hq, G, tiles, tile_heads, max_len, score_ld, step_log;
    float scale2;    // scale * log2(e)
};

// Waves of a workgroup: 4, and 8 in a direct call, which has one workgroup a row
// and wants it done soon (D > 128 needs the registers of 4).
constexpr int waves_of(int DP, bool direct) { return direct && DP <= 128 ? 8 : 4; }
// 16-token blocks of one wave's step: the 32 tokens of one value product.  (4 for
// int8, as many bytes as bf16, need the registers of a third wave: 48 uneven
// sequences of up to 8190 tokens took 100 us against 93, 200 of 1000 111 against 95,
// 96 of 8192 289 against 284; one of 262143 tokens 107 against 110.)
constexpr int kBlocks = 2, kTile = 16 * kBlocks;
// tokens of one workgroup's step
constexpr int step_of(int DP, bool direct) { return waves_of(DP, direct) * kTile; }
constexpr int kLeastStep = waves_of(128, false) * kTile;
constexpr int kMaxGroups = 1024;   // workgroups of a divided call, at most

// waves of a SIMD, by the registers they need
constexpr int resident(int DP, bool plain, bool bf16) {   // plain: D == DP and no mask
    return DP == 256 ? 1 : DP == 128 ? (plain && bf16 ? 3 : 2) : 3;
}

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
// an offset past any row of scores (2^30 bytes), whose end does not wrap either
constexpr int kNowhere = 0x7ffffff0;
// t[j] = the bytes j of a, b, c, d
__device__ __forceinline__ void turn4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&t)[4]) {
    const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x05010400u), AB = __builtin_amdgcn_perm(b, a, 0x07030602u);
    const uint32_t cd = __builtin_amdgcn_perm(d, c, 0x05010400u), CD = __builtin_amdgcn_perm(d, c, 0x07030602u);
    t[0] = __builtin_amdgcn_perm(cd, ab, 0x05040100u);
    t[1] = __builtin_amdgcn_perm(cd, ab, 0x07060302u);
    t[2] = __builtin_amdgcn_perm(CD, AB, 0x05040100u);
    t[3] = __builtin_amdgcn_perm(CD, AB, 0x07060302u);
}
__device__ __forceinline__ int length_of(const Args &a, int b) { return min(max(a.lens[b], 0), a.max_len); }
__device__ __forceinline__ int steps_of(const Args &a, int len) { return (int)((uint32_t)(len + (1 << a.step_log) - 1) >> a.step_log); }

// In a row whose sum is NaN every weight is, save those of slots that are left
// out: their scores are -infinity for all heads, and they receive nothing.
template <class Scores>
__device__ __forceinline__ void clear_left_out(f4 &add, int heads, Scores scores) {
    const float x[4] = {add[0], add[1], add[2], add[3]};
    if (x[0] == x[0] && x[1] == x[1] && x[2] == x[2] && x[3] == x[3]) return;
    float most[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};   // (NaN counts as a score)
    for (int g = 0; g < heads; ++g) {
        const f4 s = scores(g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float y = s[e];
            most[e] = y == -INFINITY ? most[e] : 0.0f;
        }
    }
    add = f4{x[0] == x[0] || most[0] == 0.0f ? x[0] : 0.0f, x[1] == x[1] || most[1] == 0.0f ? x[1] : 0.0f,
             x[2] == x[2] || most[2] == 0.0f ? x[2] : 0.0f, x[3] == x[3] || most[3] == 0.0f ? x[3] : 0.0f};
}

// A row is one (sequence, key-value head, tile of up to 16 query heads).
//
// DIRECT: one workgroup takes one row and writes its output.  Otherwise the
// steps of all rows, in order, are dealt out in equal contiguous
// shares: every workgroup is resident, starts once and ends with the others
// whatever the lengths are.  A share can end and begin inside rows; the parts of
// rows go to the workspace, part (workgroup + row), which no other pair shares
// because along the shares one of the two grows from pair to pair.
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
template <int DP, bool EXACT, bool I8, bool BF16, bool MASKED, bool TRACK, bool DIRECT>
__global__ void __launch_bounds__(waves_of(DP, DIRECT) * 64) __attribute__((amdgpu_waves_per_eu(DIRECT ? 1 : resident(DP, EXACT && !MASKED, BF16)))) attend_kernel(Args a) {
    constexpr int QP = BF16 ? 1 : 3, PP = BF16 ? 2 : 3;
    constexpr int KS = DP / 32;                  // products along d
    constexpr int W = DP == 64 ? 4 : 8;          // d of one value load
    constexpr int NU = DP / (16 * W);            // value loads of a token
    constexpr int H = kBlocks, TILE = kTile, STEP = step_of(DP, DIRECT);
    constexpr int kWaves = waves_of(DP, DIRECT), kThreads = kWaves * 64;
    __shared__ float s_m[kWaves][16], s_l[kWaves][16];
    __shared__ float s_o[kWaves][16][DP + 4];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g4 = lane >> 4;
    const int D = EXACT ? DP : a.c.D;
    const int rows_of_seq = a.c.heads * a.tiles;

    // this workgroup's steps [u, u_end), and the row that u lies in
    int b, r, len;            // sequence; row of the sequence; its length
    int64_t u = 0, u_end = 1;
    int step0 = 0;            // first step within the row
    if constexpr (DIRECT) {
        b = blockIdx.x / rows_of_seq;
        r = blockIdx.x - b * rows_of_seq;
        len = length_of(a, b);
    } else {
        __shared__ int64_t s_wave[kWaves];
        __shared__ int64_t s_at;
        __shared__ int s_b, s_len;
        const int each = (a.c.batch + kThreads - 1) / kThreads, lo = threadIdx.x * each, hi = min(lo + each, a.c.batch);
        const int len0 = lo < hi ? length_of(a, lo) : 0;
        int64_t mine = steps_of(a, len0);
        for (int i = lo + 1; i < hi; ++i) mine += steps_of(a, length_of(a, i));
        int64_t upto = mine;
        for (int o = 1; o < 64; o *= 2) {
            const int64_t y = __shfl_up(upto, o);
            if (lane >= o) upto += y;
        }
        if (lane == 63) s_wave[wave] = upto;
        __syncthreads();
        int64_t all = 0;
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) upto += s_wave[w];
            all += s_wave[w];
        }
        const int64_t per = max((int64_t)1, (all * rows_of_seq + gridDim.x - 1) / gridDim.x);
        u = blockIdx.x * per;
        u_end = min(all * rows_of_seq, u + per);
        if (u >= u_end) return;
        if ((upto - mine) * rows_of_seq <= u && u < upto * rows_of_seq) {   // one thread
            int64_t at = upto - mine;
            int i = lo, n = len0;
            while (u >= (at + steps_of(a, n)) * rows_of_seq) {
                at += steps_of(a, n);
                n = length_of(a, ++i);
            }
            s_b = i;
            s_len = n;
            s_at = at;
        }
        __syncthreads();
        b = __builtin_amdgcn_readfirstlane(s_b);
        const int64_t off = u - s_at * rows_of_seq;
        len = __builtin_amdgcn_readfirstlane(s_len);
        const int n = steps_of(a, len);
        r = __builtin_amdgcn_readfirstlane((int)(off / n));
        step0 = __builtin_amdgcn_readfirstlane((int)(off - (int64_t)r * n));
    }

    for (;;) {   // (rows of this workgroup's share)
    const int row_steps = steps_of(a, len);
    const int here = DIRECT ? row_steps : (int)min((int64_t)(row_steps - step0), u_end - u);
    const int begin = step0 * STEP, end = min(len, begin + here * STEP);
    const int h = r / a.tiles, g0 = (r - h * a.tiles) * 16;
    const int heads = min(16, a.G - g0);
    const int64_t head0 = (int64_t)b * a.hq + h * a.G + g0;

    // the pages of this wave's next 64 / H steps: lane H i + block
    int32_t page_of = -1;
    auto load_pages = [&](int step) {
        const int j = begin + ((step + lane / H) * kWaves + wave) * TILE + (lane % H) * 16;
        const int idx = j >> a.c.page_log;   // (asked for without waiting for the length)
        page_of = idx < a.c.table_ld ? a.c.table[(int64_t)b * a.c.table_ld + idx] : -1;
    };
    load_pages(0);

    // this row's scores, as a buffer
    const __amdgpu_buffer_rsrc_t score_row = __builtin_amdgcn_make_buffer_rsrc(
        TRACK ? a.scores + ((int64_t)b * rows_of_seq + r) * a.score_ld * a.tile_heads : nullptr, 0,
        TRACK ? a.score_ld * a.tile_heads * 4 : 0, 0x00020000);
    const int score_lane = col < heads ? (col * 16 + g4 * 4) * 4 : kNowhere;
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
    const int page_mask = (1 << a.c.page_log) - 1;

    // base row of block x of a step; `there`: whether it has a page
    auto row_of = [&](int step, int x, bool &there) -> int64_t {
        const int j = begin + (step * kWaves + wave) * TILE + x * 16;
        const int32_t pg = __builtin_amdgcn_readlane(page_of, (step & (64 / H - 1)) * H + x);
        there = (uint32_t)pg < (uint32_t)a.c.pages && j < end;
        return (((int64_t)(there ? pg : 0) * a.c.heads + h) << a.c.page_log) + (j & page_mask);
    };

    u4 kreg[H][KS];
    u4 vreg[H * 4][NU];   // bf16: W / 2 dwords used; int8: W / 4
    f4 ks[H], vs[H];
    bool there[H];
    uint32_t mreg[H];     // mask bytes of the lane's four tokens

    // Loads of a later step leave under no condition, so that the compiler's count
    // of what is in flight is exact and each use waits for its own operands only.
    // Past the end (live is false) all lanes read one place of page 0.
    const uint32_t k_lane = (col * D + (I8 && EXACT ? g4 * 16 : g4 * 8)) * EB;
    const uint32_t v_lane = (g4 * 4 * D + ((EXACT || W * col < D) ? W * col : 0)) * EB;
    auto load_k = [&](int step, int hf, bool live) {
        const int64_t row = row_of(step, hf, there[hf]);
        const char *base = static_cast<const char *>(a.c.k) + row * (D * EB);
        const uint32_t lane_at = live ? k_lane : 0;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            if constexpr (I8 && EXACT) {
                if (s % 2 == 0) kreg[hf][s / 2] = *reinterpret_cast<const u4 *>(base + lane_at + s * 32);
            } else {
                // (pieces past D: any place of the row; they are cleared where they are used)
                const char *p = base + ((EXACT || d_of(s) < D) ? lane_at + s * 32 * EB : 0);
                if constexpr (!I8) kreg[hf][s] = *reinterpret_cast<const u4 *>(p);
                else {
                    const u2 c = *reinterpret_cast<const u2 *>(p);
                    kreg[hf][s][0] = c[0];
                    kreg[hf][s][1] = c[1];
                }
            }
        }
        if constexpr (I8) ks[hf] = *reinterpret_cast<const f4 *>(a.c.k_scale + row + (live ? g4 * 4 : 0));
        if constexpr (MASKED) {
            const uint8_t *mask = a.mask + (int64_t)b * a.mask_ld;
            const int j = begin + (step * kWaves + wave) * TILE + hf * 16 + g4 * 4;
            mreg[hf] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) mreg[hf] |= (uint32_t)(mask[min(j + i, end - 1)] != 0) << i;
        }
    };
    auto load_v = [&](int step, int hf, bool live) {
        bool unused;
        const int64_t row = row_of(step, hf, unused);
        const char *base = static_cast<const char *>(a.c.v) + row * (D * EB);
        const uint32_t lane_at = live ? v_lane : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                // (d past D: columns of the product that nobody reads)
                const char *p = base + lane_at + ((EXACT || u == 0 || W * col + 16 * W * u < D) ? i * D + 16 * W * u : 0) * EB;
                u4 &r = vreg[hf * 4 + i][u];
                if constexpr (W * EB == 16) r = *reinterpret_cast<const u4 *>(p);
                else if constexpr (W * EB == 8) {
                    const u2 x = *reinterpret_cast<const u2 *>(p);
                    r[0] = x[0];
                    r[1] = x[1];
                } else r[0] = *reinterpret_cast<const uint32_t *>(p);
            }
        if constexpr (I8) vs[hf] = *reinterpret_cast<const f4 *>(a.c.v_scale + row + (live ? g4 * 4 : 0));
    };

    auto mine = [&](int step) { return begin + (step * kWaves + wave) * TILE < end; };   // wave-uniform
    if (mine(0)) {
#pragma unroll
        for (int hf = 0; hf < H; ++hf) load_k(0, hf, true);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int hf = 0; hf < H; ++hf) load_v(0, hf, true);
        __builtin_amdgcn_sched_barrier(0);
    }
    for (int step = 0; mine(step); ++step) {
        const int j0 = begin + (step * kWaves + wave) * TILE;
        const bool more = mine(step + 1);
        if (((step + 1) & (64 / H - 1)) == 0) {
            load_pages(step + 1);
            asm volatile("" : "+v"(page_of));   // waited for here and nowhere else
        }
        // scores: lane (head col, g4) gets tokens j0 + 16 hf + 4 g4 + i
        f4 s[H];
        bool ok[H];
        uint32_t masked_in[H];
#pragma unroll
        for (int hf = 0; hf < H; ++hf) {
            ok[hf] = there[hf];
            masked_in[hf] = MASKED ? mreg[hf] : 15;
            s[hf] = f4{0, 0, 0, 0};
#pragma unroll
            for (int t = 0; t < KS; ++t) {
                u4 k;
                if constexpr (!I8) k = kreg[hf][t];
                else if constexpr (EXACT) k = widen8(t & 1 ? u2{kreg[hf][t / 2][2], kreg[hf][t / 2][3]} : u2{kreg[hf][t / 2][0], kreg[hf][t / 2][1]});
                else k = widen8(u2{kreg[hf][t][0], kreg[hf][t][1]});
                if (!EXACT && d_of(t) >= D) k = u4{0, 0, 0, 0};
#pragma unroll
                for (int p = 0; p < QP; ++p) s[hf] = mfma(k, q[p][t], s[hf]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[hf][i] *= a.scale2;
                if constexpr (I8) s[hf][i] *= ks[hf][i];
            }
            load_k(step + 1, hf, more);
        }
        __builtin_amdgcn_sched_barrier(0);
        // tokens that are left out
        bool whole = j0 + TILE <= end && !MASKED;
#pragma unroll
        for (int hf = 0; hf < H; ++hf) whole = whole && ok[hf];
        bool use[H][4];
        if (!whole) {
#pragma unroll
            for (int hf = 0; hf < H; ++hf)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = j0 + hf * 16 + g4 * 4 + i;
                    // (one expression without branches: taken apart into nested ones by &&,
                    // the store into the vector's element was lost for masked tokens)
                    const bool in = (int)ok[hf] & (int)(j < end) & (int)(masked_in[hf] >> i & 1);
                    const float x = s[hf][i];
                    s[hf][i] = in ? x : -INFINITY;
                    use[hf][i] = in;
                }
        }
        if constexpr (TRACK) {
            // (a buffer store drops the lanes whose offset lies past the row; under a
            // branch the count of what is in flight would not be exact any more)
#pragma unroll
            for (int hf = 0; hf < H; ++hf)
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, s[hf]), score_row, score_lane,
                                                       (j0 + hf * 16) * a.tile_heads * 4, 0);
        }
        // The running maximum only moves when a score passes it by 2^8: weights
        // up to 256 are as exact, and most steps leave the sums as they are.
        float top = -INFINITY;
#pragma unroll
        for (int hf = 0; hf < H; ++hf) top = fmaxf(top, fmaxf(fmaxf(s[hf][0], s[hf][1]), fmaxf(s[hf][2], s[hf][3])));
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
        float p[H * 4];
#pragma unroll
        for (int i = 0; i < H * 4; ++i) {
            p[i] = __builtin_amdgcn_exp2f(s[i / 4][i % 4] - base);
            l += p[i];
            if constexpr (I8) p[i] *= vs[i / 4][i % 4];
        }
        if (!whole) {
#pragma unroll
            for (int i = 0; i < H * 4; ++i)
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
            if constexpr (!I8) {
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    u4 t;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        t[i] = __builtin_amdgcn_perm(vreg[2 * i + 1][u][j / 2], vreg[2 * i][u][j / 2], j & 1 ? 0x07060302u : 0x05040100u);
#pragma unroll
                    for (int n = 0; n < PP; ++n) o[u][j] = mfma(t, pp[n], o[u][j]);
                }
            } else {
                // four d at a time: the 4 x 4 bytes of four tokens turned, then
                // widened, are the operand's two dwords of those tokens
#pragma unroll
                for (int c = 0; c < W / 4; ++c) {
                    uint32_t t[2][4];
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int at = 4 * hf;
                        turn4(vreg[at][u][c], vreg[at + 1][u][c], vreg[at + 2][u][c], vreg[at + 3][u][c], t[hf]);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const u2 x = widen4(t[0][j]), y = widen4(t[1][j]);
#pragma unroll
                        for (int n = 0; n < PP; ++n) o[u][4 * c + j] = mfma(u4{x[0], x[1], y[0], y[1]}, pp[n], o[u][4 * c + j]);
                    }
                }
            }
        }
#pragma unroll
        for (int hf = 0; hf < H; ++hf) load_v(step + 1, hf, more);
        __builtin_amdgcn_sched_barrier(0);
    }

    // join the waves: o of lane (head col, g4) is d = W (4 g4 + i) + 16 W u + j
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    // A NaN score is in l, but maxima drop it.  A maximum of infinity takes it
    // through every join: exp2(inf - inf) is NaN, other parts count 0 beside it.
    if (l != l) m = INFINITY;
    if (g4 == 0) {
        s_m[wave][col] = m;
        s_l[wave][col] = l;
    }
    __syncthreads();
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) M = fmaxf(M, s_m[w][col]);
    const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - M);
    if (col < heads)
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < W; j += 4)
                    *reinterpret_cast<f4 *>(&s_o[wave][col][W * (4 * g4 + i) + 16 * W * u + j]) =
                        f4{o[u][j][i], o[u][j + 1][i], o[u][j + 2][i], o[u][j + 3][i]} * f;
    __syncthreads();
    for (int x = threadIdx.x; x < heads * (D / 4); x += kThreads) {
        const int g = x / (D / 4), d = (x - g * (D / 4)) * 4;
        f4 r4 = {0, 0, 0, 0};
        float mm = -INFINITY, ll = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, s_m[w][g]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            r4 += *reinterpret_cast<const f4 *>(&s_o[w][g][d]);
            if (s_m[w][g] != -INFINITY) ll += s_l[w][g] * __builtin_amdgcn_exp2f(s_m[w][g] - mm);
        }
        if constexpr (!DIRECT) {
            const int64_t part = (blockIdx.x + (int64_t)b * rows_of_seq + r) * a.tile_heads + g;
            *reinterpret_cast<f4 *>(a.part + part * D + d) = r4;
            if (d == 0) {
                a.stat[part * 2] = mm;
                a.stat[part * 2 + 1] = ll;
            }
        } else {
            const float inv = mm == -INFINITY ? 0.0f : 1.0f / ll;
            const int64_t at = (int64_t)b * a.out_ld + (int64_t)(h * a.G + g0 + g) * D + d;
            store4<BF16>(a.out, at, r4 * inv);
            if (d == 0 && a.lse) a.lse[head0 + g] = mm == -INFINITY ? -INFINITY : (mm + log2f(ll)) * kLn2;
        }
    }
    if constexpr (DIRECT && TRACK) {
        // this workgroup has all heads of its key-value head (one tile) and all their
        // scores: it adds the weights up itself
        __shared__ float s_fin[2][16];
        if ((int)threadIdx.x < heads) {
            float mm = -INFINITY, ll = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, s_m[w][threadIdx.x]);
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                if (s_m[w][threadIdx.x] != -INFINITY) ll += s_l[w][threadIdx.x] * __builtin_amdgcn_exp2f(s_m[w][threadIdx.x] - mm);
            s_fin[0][threadIdx.x] = mm == -INFINITY ? 0.0f : mm;
            s_fin[1][threadIdx.x] = mm == -INFINITY ? 0.0f : 1.0f / ll;
        }
        __threadfence_block();
        __syncthreads();
        const int64_t row = (int64_t)b * rows_of_seq + r;
        for (int j = threadIdx.x * 4; j < len; j += kThreads * 4) {
            const float *sc = a.scores + (row * a.score_ld + (j & ~15)) * a.tile_heads + (j & 15);
            const int64_t at = row * a.c.slots() + j;
            const f4 before = *reinterpret_cast<const f4 *>(a.weight + at);   // (slots come in whole pages)
            f4 add = {0, 0, 0, 0};
#pragma unroll 4
            for (int g = 0; g < heads; ++g) {
                const f4 x = *reinterpret_cast<const f4 *>(sc + g * 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) add[e] += __builtin_amdgcn_exp2f(x[e] - s_fin[0][g]) * s_fin[1][g];
            }
            clear_left_out(add, heads, [&](int g) { return *reinterpret_cast<const f4 *>(sc + g * 16); });
            for (int e = 0; e < 4; ++e)
                if (j + e < len) a.weight_out[at + e] = before[e] + add[e];
        }
    }
    if constexpr (DIRECT) return;
    if (threadIdx.x == 0) {
        int32_t *e = a.ends + ((int64_t)b * rows_of_seq + r) * 2;
        if (step0 == 0) e[0] = blockIdx.x;
        if (step0 + here == row_steps) e[1] = blockIdx.x;
    }
    u += here;
    if (u >= u_end) return;
    // the next row with tokens
    step0 = 0;
    if (++r == rows_of_seq) {
        r = 0;
        do len = length_of(a, ++b); while (len == 0);   // (u < u_end: there is one)
    }
    __syncthreads();
    }
}

constexpr int kJoin = 256;     // threads of a joining workgroup

// Joins the parts of rows (4 to 7 us; with the weights of 64 sequences of 4000
// tokens 18 us, 50 MB).  The first outs workgroups write outputs, a head by
// TPH threads each (all of a workgroup where heads are few, a wave where there
// are many); the others add the weights of kJoin * 4 slots of one key-value
// head.  All parts' factors come first, so that the loads of the partial outputs
// depend on nothing and are in flight together: everything comes from the
// caches, and latency is all there is.
template <bool BF16, int TPH>
__global__ void __launch_bounds__(kJoin) join_kernel(Args a, int outs) {
    constexpr int HEADS = kJoin / TPH;
    __shared__ float s_o[kJoin][4];
    __shared__ float s_f[HEADS][TPH == 64 ? 1 : kMaxGroups];
    __shared__ float s_m[64], s_i[64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, D = a.c.D;
    const int rows_of_seq = a.c.heads * a.tiles;
    // parts of head g of key-value head h of sequence b: their number, and the first
    auto parts = [&](int b, int len, int h, int g, int64_t &part) {
        const int64_t row = (int64_t)b * rows_of_seq + h * a.tiles + g / 16;
        const int32_t w0 = a.ends[row * 2], w1 = a.ends[row * 2 + 1];   // (garbage in an empty row)
        part = len > 0 ? (w0 + row) * a.tile_heads + g % 16 : 0;
        return len > 0 ? w1 - w0 + 1 : 0;
    };
    if ((int)blockIdx.x < outs) {
        const int64_t head = (int64_t)blockIdx.x * HEADS + threadIdx.x / TPH;
        if (head >= (int64_t)a.c.batch * a.hq) return;   // (whole waves; with TPH = kJoin none)
        const int b = (int)(head / a.hq), i = (int)(head - (int64_t)b * a.hq), t = threadIdx.x % TPH;
        int64_t part;
        const int n = parts(b, length_of(a, b), i / a.G, i % a.G, part);
        const f2 *st = reinterpret_cast<const f2 *>(a.stat) + part;
        const float *po = a.part + part * D;
        const int stride = a.tile_heads;
        float M, L;
        join_stats(st, n, stride, lane, M, L);
        auto factor = [&](int s) {
            const float m = st[(int64_t)s * stride][0];
            return m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - M);
        };
        f4 r = {0, 0, 0, 0};
        const int quads = D / 4;
        if constexpr (TPH == 64) {
            if (t < quads)
#pragma unroll 4
                for (int s = 0; s < n; ++s) r += *reinterpret_cast<const f4 *>(po + (int64_t)s * a.tile_heads * D + t * 4) * factor(s);
        } else {
            for (int s = t; s < n; s += TPH) s_f[0][s] = factor(s);
            __syncthreads();
            const int groups = TPH / quads, group = t / quads, d = (t - group * quads) * 4;
            if (group < groups)
#pragma unroll 8
                for (int s = group; s < n; s += groups) r += *reinterpret_cast<const f4 *>(po + (int64_t)s * a.tile_heads * D + d) * s_f[0][s];
            *reinterpret_cast<f4 *>(s_o[t]) = r;
            __syncthreads();
            if (t < quads)
                for (int g = 1; g < min(groups, n); ++g) r += *reinterpret_cast<const f4 *>(s_o[t + g * quads]);
        }
        if (t < quads) {
            const float inv = M == -INFINITY ? 0.0f : 1.0f / L;
            store4<BF16>(a.out, (int64_t)b * a.out_ld + (int64_t)i * D + t * 4, r * inv);
            if (t == 0 && a.lse) a.lse[head] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * kLn2;
        }
        return;
    }
    const int blocks = (a.max_len + kJoin * 4 - 1) / (kJoin * 4);
    const int64_t id = blockIdx.x - outs;
    const int row = (int)(id / blocks), b = row / a.c.heads, h = row - b * a.c.heads;
    const int j0 = (int)(id - (int64_t)row * blocks) * kJoin * 4, j = j0 + threadIdx.x * 4;
    const int len = length_of(a, b);
    if (j0 >= len) return;
    const int64_t at = (int64_t)row * a.c.slots() + j;
    auto scores = [&](int g) {
        return *reinterpret_cast<const f4 *>(a.scores + (((int64_t)row * a.tiles + g / 16) * a.score_ld + (j & ~15)) * a.tile_heads + (g % 16) * 16 + (j & 15));
    };
    // scores and weights are asked for before the statistics are waited for
    constexpr int AHEAD = 8;
    f4 ahead[AHEAD], w = {0, 0, 0, 0};
    if (j < len) {
#pragma unroll
        for (int g = 0; g < AHEAD; ++g)
            if (g < a.G) ahead[g] = scores(g);
        w = *reinterpret_cast<const f4 *>(a.weight + at);   // (slots come in whole pages)
    }
    f4 add = {0, 0, 0, 0};
    for (int g0 = 0; g0 < a.G; g0 += 64) {
        const int gn = min(64, a.G - g0);
        if (g0) __syncthreads();
        for (int g = wave; g < gn; g += kJoin / 64) {
            int64_t part;
            const int n = parts(b, len, h, g0 + g, part);
            float M, L;
            join_stats(reinterpret_cast<const f2 *>(a.stat) + part, n, a.tile_heads, lane, M, L);
            if (lane == 0) {
                s_m[g] = M == -INFINITY ? 0.0f : M;
                s_i[g] = M == -INFINITY ? 0.0f : 1.0f / L;
            }
        }
        __syncthreads();
        auto take = [&](const f4 &s, int g) {
#pragma unroll
            for (int e = 0; e < 4; ++e) add[e] += __builtin_amdgcn_exp2f(s[e] - s_m[g]) * s_i[g];
        };
        if (j < len) {
            if (g0 == 0) {
#pragma unroll
                for (int g = 0; g < AHEAD; ++g)
                    if (g < gn) take(ahead[g], g);
            }
            for (int g = g0 == 0 ? AHEAD : 0; g < gn; ++g)
                take(scores(g0 + g), g);
        }
    }
    if (j < len) clear_left_out(add, a.G, scores);
    w += add;
    if (j + 4 <= len) *reinterpret_cast<f4 *>(a.weight_out + at) = w;
    else
        for (int e = 0; e < 4; ++e)
            if (j + e < len) a.weight_out[at + e] = w[e];
}

// How a call is run.  Direct up to kDirect tokens: a workgroup walks them in
// fewer microseconds than the joining kernel costs (8 sequences of 300 tokens: 8.3
// us against 11.2; of 512 10.0 against 11.6; of 1024 14.6 against 15.2).  Direct too
// where the rows fill the device and are many for their length, so that uneven ones
// even out: 256 sequences of 2000 tokens, 8 heads 349 us (6.0 TB/s) against 371,
// uneven 188 against 215; 128 of 4000, uneven 201 against 204; but 64 of up to 8000,
// uneven 222 against 203.
constexpr int kDirect = 512;
// Shares per CU otherwise, at most: what is resident of the variant with the
// fewest registers.  With 3, 2, 1 of them 48 uneven int8 sequences take 96, 96, 107
// us, 64 uneven tracked ones 257, 258, 262; a sequence alone would like fewer (131071
// bf16 tokens 103, 98, 98, 262143 int8 ones 111, 108, 105).
constexpr int kGroupsPerCu = 3;
struct Plan {
    bool direct;
    bool many;                         // join: a wave a head instead of a workgroup
    int tiles, tile_heads, groups, score_ld;
    int64_t outs, weights;             // join: workgroups for outputs and for weights
    size_t part, stat, ends, scores;   // bytes
};
Plan plan_of(const rq_kv_cache *c, int q_heads, int64_t max_len, int track) {
    Plan p{};
    const int G = q_heads / c->heads;
    p.tiles = (G + 15) / 16;
    p.tile_heads = std::min(G, 16);
    const int64_t rows = (int64_t)c->batch * c->heads * p.tiles;
    // (tracked: where the workgroup has all of a key-value head's query heads)
    p.direct = (!track || p.tiles == 1) && rows <= (1 << 20) && (max_len <= kDirect || (rows >= device_cus() && max_len <= 4 * rows));
    p.score_ld = (int)((max_len + kTile - 1) / kTile * kTile);   // whole steps of a wave are written
    auto round = [](size_t n) { return (n + 15) / 16 * 16; };
    p.scores = track ? round((size_t)rows * p.tile_heads * p.score_ld * 4) : 0;
    if (p.direct) return p;
    // (the least step, whatever the head size)
    const int64_t steps = rows * ((max_len + kLeastStep - 1) / kLeastStep);
    p.groups = (int)std::max<int64_t>(1, std::min<int64_t>({steps, (int64_t)device_cus() * kGroupsPerCu, kMaxGroups}));
    const size_t parts = (size_t)(p.groups + rows) * p.tile_heads;
    p.part = round(parts * c->head_dim * 4);
    p.stat = round(parts * 8);
    p.ends = round((size_t)rows * 8);
    // A wave a head once that fills the device: 4096 heads of 6000 tokens 528 us
    // against 534 by a workgroup a head, 2048 of 4000 189 against 192, from 1280 down
    // to 256 alike; 32 heads of 131071 tokens 113 against 103.
    const int64_t heads = (int64_t)c->batch * q_heads;
    p.many = heads >= 4 * device_cus();
    p.outs = p.many ? (heads + kJoin / 64 - 1) / (kJoin / 64) : heads;
    p.weights = track ? (max_len + kJoin * 4 - 1) / (kJoin * 4) * c->batch * c->heads : 0;
    return p;
}

}  // namespace

bool attend_fits(const rq_kv_cache *c, int q_heads, int64_t max_len, int track) {
    const Plan p = plan_of(c, q_heads, max_len, track);
    return p.outs + p.weights < (1 << 24);   // (of kJoin threads: a launch holds 2^32)
}

size_t attend_workspace_bytes(const rq_kv_cache *c, int q_heads, int64_t max_len, int track) {
    const Plan p = plan_of(c, q_heads, max_len, track);
    return p.part + p.stat + p.ends + p.scores;
}

int launch_paged_attention(const rq_kv_cache *c, const void *q, int bf16, int64_t q_ld, int q_heads,
                           float scale, const int32_t *lens, int64_t max_len, const uint8_t *mask,
                           int64_t mask_ld, void *out, int64_t out_ld, float *lse, int track,
                           float *weight_out, void *workspace, void *stream) {
    const Plan p = plan_of(c, q_heads, max_len, track);
    // as many shares as are resident at once
    const int DP = c->head_dim > 128 ? 256 : c->head_dim > 64 ? 128 : 64;
    const int fit = device_cus() * std::min(kGroupsPerCu, resident(DP, c->head_dim == DP && !mask, bf16));
    const unsigned groups = p.direct ? (unsigned)c->batch * c->heads * p.tiles : (unsigned)std::min(p.groups, fit);
    Args a{};
    a.c = device_cache(c);
    a.q = q, a.out = out, a.lens = lens, a.mask = mask, a.lse = lse;
    a.weight = c->weight, a.weight_out = weight_out;
    char *ws = static_cast<char *>(workspace);
    a.part = reinterpret_cast<float *>(ws);
    a.stat = reinterpret_cast<float *>(ws + p.part);
    a.ends = reinterpret_cast<int32_t *>(ws + p.part + p.stat);
    a.scores = reinterpret_cast<float *>(ws + p.part + p.stat + p.ends);
    a.q_ld = q_ld, a.out_ld = out_ld, a.mask_ld = mask_ld;
    a.hq = q_heads, a.G = q_heads / c->heads, a.tiles = p.tiles, a.tile_heads = p.tile_heads;
    a.max_len = (int)max_len, a.score_ld = p.score_ld, a.step_log = ilog2(step_of(DP, p.direct));
    a.scale2 = scale * 1.4426950408889634f;
    hipStream_t s = static_cast<hipStream_t>(stream);
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(groups), dim3(waves_of(DP, p.direct) * 64), 0, s, a); };
    auto pick = [&](auto dp, auto exact, auto i8, auto io) {
        constexpr int DP = decltype(dp)::value;
        constexpr bool E = decltype(exact)::value, I = decltype(i8)::value, B = decltype(io)::value;
        auto run = [&](auto direct) {
            constexpr bool R = decltype(direct)::value;
            if (mask && track) go(attend_kernel<DP, E, I, B, true, true, R>);
            else if (mask) go(attend_kernel<DP, E, I, B, true, false, R>);
            else if (track) go(attend_kernel<DP, E, I, B, false, true, R>);
            else go(attend_kernel<DP, E, I, B, false, false, R>);
        };
        if (p.direct) run(std::true_type{});
        else run(std::false_type{});
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
    if (!p.direct) {
        auto join = [&](auto kern) { hipLaunchKernelGGL(kern, dim3((unsigned)(p.outs + p.weights)), dim3(kJoin), 0, s, a, (int)p.outs); };
        if (bf16) p.many ? join(join_kernel<true, 64>) : join(join_kernel<true, kJoin>);
        else p.many ? join(join_kernel<false, 64>) : join(join_kernel<false, kJoin>);
    }
    return (int)hipGetLastError();
}

}  // namespace rq
