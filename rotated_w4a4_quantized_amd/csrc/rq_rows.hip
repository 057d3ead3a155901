// rq_rows.hip -- attention of many query rows over the same keys: the tokens of a
// block over an encoder's states (or over each other), and a batch of single
// tokens over a prefix that its sequences share.
//
//   s_j = scale q . k_j;  lse = log sum exp s_j;  out = sum exp(s_j - lse) v_j
//
// Query heads that share a key-value head, of all query tokens, are the rows of
// one problem: row r is token r / G, head r % G.
//
// Many rows are bound by the matrix cores and by the vector units beside them: a block
// of 32 rows x 32 keys x 128 takes 24 products of 32 cycles and some 115 other
// instructions (half the maximum, exponent's argument, exponential at twice an
// instruction's time, sum, conversion and two for what the weight's first part leaves,
// for each of its 16 registers, and the step's own).  9216 x 9216 tokens, 12 heads of
// 128, take 720 us: 725 TFLOP/s, of products with the weights' second part 1090 (a large
// bf16 product of the library reaches 1220), where 864 row tiles on 512 places leave a
// sixth of the second round empty; 4 x 4096 x 1280 run at 730.  Short keys are bound by
// what every workgroup starts and ends with (5 us: arguments, keys and queries, results),
// of which as many as fit run side by side.  Few rows are bound by HBM: 77 queries on 201
// MB of keys and values 44 us (4.5 TB/s) and 7 us of joining.

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

// Division by a number that the host knows: n / d for n < 2^30, d <= 2^30.
// (With 2^shift <= d < 2^(shift + 1) and magic = ceil(2^(31 + shift) / d) the
// product is over by less than n d / 2^(31 + shift) < 1 parts of d.)
struct Over {
    uint32_t d, magic, shift;
    __device__ __forceinline__ int of(int n) const { return (int)(__umulhi(2u * (uint32_t)n, magic) >> shift); }
};
Over over(int64_t d) {
    Over x{(uint32_t)d, 0, 0};
    while ((int64_t(2) << x.shift) <= d) ++x.shift;
    x.magic = (uint32_t)(((uint64_t(1) << (31 + x.shift)) + d - 1) / d);
    return x;
}

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
    int32_t jobs;                  // of this launch
    int32_t longest_first;         // 1: by_share.d jobs of each sequence on an XCD, the longest sequence's first
    Over by_G, by_batch, by_tiles, by_splits, by_share, by_queries, by_heads, by_quads;
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
    int begin, end;                // slots; begin is a multiple of 16, and slots below first
    int first;                     // do not count
    int others;                    // parts of these rows that join (part: of the first of them)
    bool to_parts;
    int64_t part, lse_at;          // part * rows of all + the problem's row 0; lse of token 0, head 0 of the group
};

__device__ __forceinline__ f16 mfma32(u4 a, u4 b, f16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
}
__device__ __forceinline__ u2 read_turned(const char *p) {
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

// Pieces of 16 bytes (8 elements) of a token's row in LDS, as staged: without
// padding (what a direct-to-LDS load writes is contiguous), but in another order in
// each row, so that the lanes of one read fall on different banks.  K: 16 tokens'
// same piece; V: 4 tokens' 4 neighbouring pieces.
template <int PC>
__device__ __forceinline__ int k_place(int row, int piece) {
    return PC == 8 ? piece ^ (row >> 1 & 7) : PC == 12 ? piece ^ (row >> 2 & 3) : piece ^ (row & 15);
}
template <int PC>
__device__ __forceinline__ int v_place(int row, int piece) {
    return PC == 8 ? piece ^ ((row >> 1 & 1) * 4) : PC == 12 ? piece : piece ^ ((row & 3) * 4);
}

// A block of 16 tokens' keys and values to LDS, N loads of 16 bytes a lane each
// (buffer_load ... lds): load i of the keys takes base k + k_from[i], and lane l's
// bytes land at `at` + 1024 i + 16 l; the values `apart` behind.  Lanes with the
// offset kNowhere write zeros.  M0 holds the LDS address (saved and restored: the
// compiler reserves it; one wait state after writing it); completion is waited for
// by hand.  One piece of assembly: each load as a piece of its own took five scalar
// instructions more, and a wave spent a third of a step's time on them.
constexpr uint32_t kNowhere = 0xc0000000u, kReach = 0x80000000u;
#define RQ_LOAD(from, base) "buffer_load_dwordx4 %[" from "], %[" base "], 0 offen lds\n\t"
#define RQ_NEXT "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\t"
#define RQ_BEGIN "s_mov_b32 %[saved], m0\n\ts_mov_b32 m0, %[at]\n\ts_nop 0\n\t"
#define RQ_VALUES "s_add_u32 m0, %[at], %[apart]\n\ts_nop 0\n\t"
#define RQ_END "s_mov_b32 m0, %[saved]"
template <int N>
__device__ __forceinline__ void to_lds(const char *k, const char *v, const uint32_t (&k_from)[N], const uint32_t (&v_from)[N],
                                       uint32_t at, uint32_t apart) {
    const uint64_t pk = reinterpret_cast<uint64_t>(k), pv = reinterpret_cast<uint64_t>(v);
    const u4 rk = {(uint32_t)pk, (uint32_t)(pk >> 32), kReach, 0x00020000u}, rv = {(uint32_t)pv, (uint32_t)(pv >> 32), kReach, 0x00020000u};
    uint32_t saved;
    static_assert(N == 2 || N == 3 || N == 4 || N == 8, "loads of a block");
    if constexpr (N == 2)
        asm volatile(RQ_BEGIN RQ_LOAD("a", "rk") RQ_NEXT RQ_LOAD("b", "rk") RQ_VALUES RQ_LOAD("e", "rv") RQ_NEXT RQ_LOAD("f", "rv") RQ_END
                     : [saved] "=&s"(saved)
                     : [a] "v"(k_from[0]), [b] "v"(k_from[1]), [e] "v"(v_from[0]), [f] "v"(v_from[1]), [rk] "s"(rk), [rv] "s"(rv),
                       [at] "s"(at), [apart] "s"(apart)
                     : "memory", "scc");
    else if constexpr (N == 3)
        asm volatile(RQ_BEGIN RQ_LOAD("a", "rk") RQ_NEXT RQ_LOAD("b", "rk") RQ_NEXT RQ_LOAD("c", "rk")
                     RQ_VALUES RQ_LOAD("e", "rv") RQ_NEXT RQ_LOAD("f", "rv") RQ_NEXT RQ_LOAD("g", "rv") RQ_END
                     : [saved] "=&s"(saved)
                     : [a] "v"(k_from[0]), [b] "v"(k_from[1]), [c] "v"(k_from[2]), [e] "v"(v_from[0]), [f] "v"(v_from[1]), [g] "v"(v_from[2]),
                       [rk] "s"(rk), [rv] "s"(rv), [at] "s"(at), [apart] "s"(apart)
                     : "memory", "scc");
    else {
        asm volatile(RQ_BEGIN RQ_LOAD("a", "rk") RQ_NEXT RQ_LOAD("b", "rk") RQ_NEXT RQ_LOAD("c", "rk") RQ_NEXT RQ_LOAD("d", "rk")
                     RQ_VALUES RQ_LOAD("e", "rv") RQ_NEXT RQ_LOAD("f", "rv") RQ_NEXT RQ_LOAD("g", "rv") RQ_NEXT RQ_LOAD("h", "rv") RQ_END
                     : [saved] "=&s"(saved)
                     : [a] "v"(k_from[0]), [b] "v"(k_from[1]), [c] "v"(k_from[2]), [d] "v"(k_from[3]), [e] "v"(v_from[0]), [f] "v"(v_from[1]),
                       [g] "v"(v_from[2]), [h] "v"(v_from[3]), [rk] "s"(rk), [rv] "s"(rv), [at] "s"(at), [apart] "s"(apart)
                     : "memory", "scc");
        if constexpr (N == 8)
            asm volatile(RQ_BEGIN RQ_LOAD("a", "rk") RQ_NEXT RQ_LOAD("b", "rk") RQ_NEXT RQ_LOAD("c", "rk") RQ_NEXT RQ_LOAD("d", "rk")
                         RQ_VALUES RQ_LOAD("e", "rv") RQ_NEXT RQ_LOAD("f", "rv") RQ_NEXT RQ_LOAD("g", "rv") RQ_NEXT RQ_LOAD("h", "rv") RQ_END
                         : [saved] "=&s"(saved)
                         : [a] "v"(k_from[N - 4]), [b] "v"(k_from[N - 3]), [c] "v"(k_from[N - 2]), [d] "v"(k_from[N - 1]), [e] "v"(v_from[N - 4]),
                           [f] "v"(v_from[N - 3]), [g] "v"(v_from[N - 2]), [h] "v"(v_from[N - 1]), [rk] "s"(rk), [rv] "s"(rv),
                           [at] "s"(at + 4096), [apart] "s"(apart)
                         : "memory", "scc");
    }
}
// One of these loads, by the lanes in `lanes` (all or none).
__device__ __forceinline__ void one_to_lds(u4 base, uint32_t from, uint32_t at, uint64_t lanes) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %[saved], m0\n\ts_mov_b32 m0, %[at]\n\ts_mov_b64 exec, %[lanes]\n\t" RQ_LOAD("a", "base")
        "s_mov_b64 exec, -1\n\ts_mov_b32 m0, %[saved]"
        : [saved] "=&s"(saved)
        : [a] "v"(from), [base] "s"(base), [at] "s"(at), [lanes] "s"(lanes)
        : "memory");
}
#undef RQ_LOAD
#undef RQ_NEXT
#undef RQ_BEGIN
#undef RQ_VALUES
#undef RQ_END

constexpr int kOthers = 64;   // parts of a problem, at most

// 32 rows a wave; RW waves along the rows, or TW along the tokens.
template <int DP_, bool BF16_, int RW_, int TW_, Source SRC_>
struct Shape {
    static constexpr int DP = DP_, RW = RW_, TW = TW_;
    static constexpr bool BF16 = BF16_;
    static constexpr Source SRC = SRC_;
    static constexpr int waves = RW * TW, threads = waves * 64;
    static constexpr int rows = RW * 32;
    static constexpr int TB = TW == 1 ? 2 : 1;            // blocks of 32 tokens a wave takes in a step
    static constexpr int KT = TW * TB * 32;               // tokens of a step
    static constexpr int PC = DP / 8;                     // pieces of a row
    static constexpr int half = KT * PC * 16;             // bytes of a step's keys
    static constexpr int scales = SRC == PAGES_I8 ? 2 * KT * 4 : 0;
    static constexpr int stage = 2 * half + scales;
    static constexpr int bias = waves * 64 * 4;           // behind the two buffers: what each wave leaves out
    // at the end: rows of results, or of the waves' parts
    static constexpr int OP = DP + 4;                     // floats from row to row
    static constexpr int ends = waves * 32 * (OP * 4 + (TW > 1 ? 8 : 0)) + (TW > 1 ? kOthers * 128 + 256 + threads * 16 : 0);
    static constexpr size_t lds = 2 * stage + bias > ends ? 2 * stage + bias : ends;
};

// A step of KT tokens goes through LDS, one step ahead; each wave brings in its
// share, bf16 straight from memory, int8 through registers, where it is widened.
// A wave computes with v_mfma_f32_32x32x16_bf16
//   S [token][row] = K Q^T: a lane gets, of row lane % 32, the tokens
//     8 (i / 4) + 4 (lane / 32) + i % 4, i = 0 .. 15, of a block of 32;
//   O^T [d][row] = V^T P^T: the lane's weights are the operand as they lie, its k
//     slots 8 (lane / 32) + e standing for the tokens above, and V^T is read in that
//     order with the transposing LDS read.
// Where the waves divide the tokens, each reads only what it brought in itself and
// there is no barrier.
//
// Rounding: K, V and bf16 queries enter exactly, fp32 queries as three bf16 parts
// (24 bits).  Weights enter as two bf16 parts (16 bits) for bf16 outputs and as three
// for fp32 ones; sums and statistics are fp32.  One part for bf16 outputs would be off by
// as much as the output's own rounding (from 64 bits 0.0025 relative in all, with two
// 0.0017, as the rounding alone); the second costs a third where the products are the
// bound (9216 x 9216 tokens, 12 heads of 128: 541 -> 720 us; 4 x 4096 x 1280, 16 heads of 64:
// 100 -> 143), 8 to 18% on a caption's keys and at most 11% elsewhere.
template <class C>
__device__ __forceinline__ void attend_rows(const Args &a, const Job &job, char *lds) {
    constexpr int DP = C::DP, KT = C::KT, TB = C::TB, PC = C::PC;
    constexpr bool BF16 = C::BF16, I8 = C::SRC == PAGES_I8, PAGED = C::SRC != STATES, WIDE = C::TW == 1;
    constexpr int QP = BF16 ? 1 : 3, WP = BF16 ? 2 : 3;   // parts of queries, of weights
    constexpr int KS = DP / 16, DB = DP / 32;
    constexpr int BW = KT / 16 / C::waves;            // blocks of 16 tokens a wave brings in
    constexpr int NI = PC / 4;                        // its loads a block, of K and of V
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, hf = lane >> 5;
    const int D = a.c.D, G = a.G;
    const int own = WIDE ? 0 : wave * 32;             // first of the tokens of a step that the wave computes with

    // ---- bringing in
    // slot j0 + own + lane: whether it counts, and its page, asked for two steps ahead
    uint32_t use;
    int32_t page_of = 0;
    auto fetch = [&](int j0) {
        const int j = j0 + own + lane, jj = min(max(j, job.first), job.end - 1);
        use = job.mask ? job.mask[jj] : 1;
        if (j != jj) use = 0;
        if constexpr (PAGED) page_of = job.table[jj >> a.c.page_log];
    };
    auto settle = [&]() -> uint64_t {
        if constexpr (PAGED)
            if ((uint32_t)page_of >= (uint32_t)a.c.pages) use = 0, page_of = 0;
        const uint64_t b = __ballot(use != 0);
        return WIDE ? b : b & 0xffffffffull;
    };
    // the lane's pieces of a block: offsets of what lands at 16 lane of each load
    uint32_t k_from[NI], v_from[NI];
    const uint32_t k_row = PAGED ? D * 2 : (uint32_t)a.k_ld * 2, v_row = PAGED ? D * 2 : (uint32_t)a.v_ld * 2;
    if constexpr (!I8)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int s = i * 64 + lane, r = s / PC, kp = k_place<PC>(r, s % PC), vp = v_place<PC>(r, s % PC);
            k_from[i] = kp * 8 < D ? r * k_row + kp * 16 : kNowhere;
            v_from[i] = vp * 8 < D ? r * v_row + vp * 16 : kNowhere;
        }
    const uint32_t lds_at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)lds;
    const int page_mask = (1 << a.c.page_log) - 1;
    constexpr bool SPREAD = WIDE && !I8;   // the loads leave between the products of the scores
    u4 k_base{}, v_base{};
    uint32_t later_at = 0;
    uint64_t later = 0;
    auto bring = [&](int j0, uint64_t bits, int buf, bool now) {
#pragma unroll
        for (int b = 0; b < BW; ++b) {
            const int block = wave * BW + b, in_bits = block * 16 - own, j = j0 + block * 16;
            const char *kp, *vp;
            if constexpr (PAGED) {
                const int64_t pg = __builtin_amdgcn_readlane(page_of, in_bits);
                const int64_t at = (((pg * a.c.heads + job.h) << a.c.page_log) + (j & page_mask)) * D * 2;
                kp = static_cast<const char *>(a.c.k) + at;
                vp = static_cast<const char *>(a.c.v) + at;
            } else {
                kp = job.k + j * a.k_ld * 2;
                vp = job.v + j * a.v_ld * 2;
            }
            const uint32_t part = (uint32_t)(bits >> in_bits) & 0xffffu;
            const uint32_t at = __builtin_amdgcn_readfirstlane(lds_at + buf * C::stage + block * 16 * PC * 16);
            if (SPREAD && !now && part == 0xffffu) {
                const uint64_t pk = reinterpret_cast<uint64_t>(kp), pv = reinterpret_cast<uint64_t>(vp);
                k_base = u4{(uint32_t)pk, (uint32_t)(pk >> 32), kReach, 0x00020000u};
                v_base = u4{(uint32_t)pv, (uint32_t)(pv >> 32), kReach, 0x00020000u};
                later_at = at;
                later = ~0ull;
            } else if (part == 0xffffu) to_lds<NI>(kp, vp, k_from, v_from, at, C::half);
            else {
                uint32_t k_some[NI], v_some[NI];
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const bool in = (part >> ((i * 64 + lane) / PC) & 1) != 0;
                    k_some[i] = in ? k_from[i] : kNowhere;
                    v_some[i] = in ? v_from[i] : kNowhere;
                }
                to_lds<NI>(kp, vp, k_some, v_some, at, C::half);
            }
        }
    };
    // int8: the same through registers
    constexpr int N = I8 ? BW * NI : 1, NS = I8 ? BW : 1;
    u2 k_reg[N], v_reg[N];
    float k_sc[NS], v_sc[NS];          // scales of slot block + lane % 16
    auto load = [&](int j0) {
        if constexpr (I8) {
#pragma unroll
            for (int b = 0; b < BW; ++b) {
                const int block = wave * BW + b;
                const int64_t pg = __builtin_amdgcn_readlane(page_of, block * 16 - own);
                const int64_t at = ((pg * a.c.heads + job.h) << a.c.page_log) + ((j0 + block * 16) & page_mask);
                const char *kp = static_cast<const char *>(a.c.k) + at * D, *vp = static_cast<const char *>(a.c.v) + at * D;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int u = i * 64 + lane, t = u / PC, d = (u - t * PC) * 8;
                    const uint32_t from = t * D + (d < D ? d : 0);
                    k_reg[b * NI + i] = *reinterpret_cast<const u2 *>(kp + from);
                    v_reg[b * NI + i] = *reinterpret_cast<const u2 *>(vp + from);
                }
                k_sc[b] = a.c.k_scale[at + lane % 16];
                v_sc[b] = a.c.v_scale[at + lane % 16];
            }
        }
    };
    auto write = [&](uint64_t bits, int buf) {
        if constexpr (I8) {
            char *base = lds + buf * C::stage;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int u = i * 64 + lane, t = u / PC, p = u - t * PC, at = wave * BW * 16 + t;
                const bool in = (bits >> (at - own) & 1) != 0 && p * 8 < D;
                const u4 x = widen(k_reg[i]), y = widen(v_reg[i]);
                *reinterpret_cast<u4 *>(base + (at * PC + k_place<PC>(at, p)) * 16) = in ? x : u4{0, 0, 0, 0};
                *reinterpret_cast<u4 *>(base + C::half + (at * PC + v_place<PC>(at, p)) * 16) = in ? y : u4{0, 0, 0, 0};
            }
            if (lane < 16)
#pragma unroll
                for (int b = 0; b < BW; ++b) {
                    const int at = (wave * BW + b) * 16 + lane;
                    const bool in = (bits >> (at - own) & 1) != 0;
                    float *sc = reinterpret_cast<float *>(base + 2 * C::half);
                    sc[at] = in ? k_sc[b] : 1.0f;   // (times -infinity)
                    sc[KT + at] = in ? v_sc[b] : 0.0f;
                }
        }
    };

    uint64_t bits_next = 0;
    if (job.begin < job.end) {
        fetch(job.begin);
        bits_next = settle();
        if constexpr (I8) load(job.begin);
        else bring(job.begin, bits_next, 0, true);
        fetch(job.begin + KT);
    }

    // ---- rows and queries
    const int row = job.row0 + (WIDE ? wave * 32 : 0) + col;
    const int r0 = min(row, job.R - 1), t0 = a.by_G.of(r0);
    const int64_t q_at = job.q_at + t0 * a.q_ld + (int64_t)(job.h * G + r0 - t0 * G) * D;
    u4 q[KS][QP];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        // (past D: any of the row, K is zero there)
        const int d = ks * 16 + hf * 8 < D ? ks * 16 + hf * 8 : 0;
        if constexpr (BF16) {
            q[ks][0] = *reinterpret_cast<const u4 *>(static_cast<const uint16_t *>(a.q) + q_at + d);
        } else {
            const float *p = static_cast<const float *>(a.q) + q_at + d;
            const f4 x = *reinterpret_cast<const f4 *>(p), y = *reinterpret_cast<const f4 *>(p + 4);
            const float z[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t p3[3];
                split2<3>(z[2 * i], z[2 * i + 1], p3);
#pragma unroll
                for (int n = 0; n < QP; ++n) q[ks][n][i] = p3[n];
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
                    const uint32_t x = q[ks][n][i];
                    q[ks][n][i] = pack2(lo_of(x) * a.q_factor, hi_of(x) * a.q_factor);
                }
    }

    f16 o[DB];
    float m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[db][i] = 0.0f;

    // the lane's places in LDS, without the token block
    int k_at[KS], v_at[DB];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) k_at[ks] = ((own + col) * PC + k_place<PC>(col, 2 * ks + hf)) * 16;
    // (an address is the lane's part of the 4 tokens x 16 columns that 16 lanes turn)
    const int v_row0 = own + 4 * hf + (lane >> 2 & 3);
#pragma unroll
    for (int db = 0; db < DB; ++db)
        v_at[db] = C::half + (v_row0 * PC + v_place<PC>(v_row0, db * 4 + (lane >> 3 & 2) + (lane >> 1 & 1))) * 16 + (lane & 1) * 8;

    int buf = 0;
    uint64_t any = 0;
    for (int j0 = job.begin; j0 < job.end; j0 += KT, buf ^= 1) {
        const uint64_t bits = bits_next;
        any |= bits;
        const bool more = j0 + KT < job.end;
        if constexpr (I8) {
            // (the next write to this buffer is two steps away, behind the next step's barrier)
            write(bits, buf);
            if (more) {
                bits_next = settle();
                load(j0 + KT);
                fetch(j0 + 2 * KT);
            }
            if constexpr (WIDE) __syncthreads();
            else asm volatile("" ::: "memory");   // (a wave's LDS accesses keep their order)
        } else {
            // this step is here, and the other buffer is read no more
            // (vmcnt(0); by the builtin, so that the compiler knows that the queries are here,
            // too: in the loop it would wait for them behind the loads of the next step)
            __builtin_amdgcn_s_waitcnt(0xf70);
            if constexpr (WIDE) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            else asm volatile("" ::: "memory");
            later = 0;
            if (more) {
                bits_next = settle();
                bring(j0 + KT, bits_next, buf ^ 1, false);
                fetch(j0 + 2 * KT);
            }
        }
        const char *here = lds + buf * C::stage;
        f16 s[TB];
        // Reads leave a block of products ahead, into the places of what was just used (left
        // to itself, the compiler has each product wait for its own).
        auto scores = [&](auto from) {
            u4 k[KS];
            auto read_k = [&](int tb, int ks) { k[ks] = *reinterpret_cast<const u4 *>(here + k_at[ks] + tb * 32 * PC * 16); };
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) read_k(0, ks);
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
                from(tb);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
                    for (int n = 0; n < QP; ++n) s[tb] = mfma32(k[ks], q[ks][n], s[tb]);
                    if (tb + 1 < TB) read_k(tb + 1, ks);
                    // the next step's loads, spread: at once, a workgroup's would fill the way to LDS
                    // and its waves wait (32760 queries x 512 keys 173 -> 161 us, heads of 256 297 -> 266)
                    if constexpr (SPREAD) {
                        const int slot = tb * KS + ks;
#pragma unroll
                        for (int i = 0; i < 2 * NI; ++i)
                            if (slot == i * (TB * KS) / (2 * NI))
                                one_to_lds(i < NI ? k_base : v_base, i < NI ? k_from[i] : v_from[i - NI],
                                           later_at + (i < NI ? i * 1024 : C::half + (i - NI) * 1024), later);
                    }
                    // (at 96 the order costs registers that a third wave needs)
                    if (DP != 96) __builtin_amdgcn_sched_barrier(0);
                }
            }
        };
        if (bits == (WIDE ? ~0ull : 0xffffffffull)) {
            scores([&](int tb) {
#pragma unroll
                for (int i = 0; i < 16; ++i) s[tb][i] = 0.0f;
            });
        } else {
            // slots that do not count start from -infinity (their keys are zeros)
            float *bias = reinterpret_cast<float *>(lds + 2 * C::stage) + wave * 64;
            bias[lane] = (bits >> lane & 1) != 0 ? 0.0f : -INFINITY;
            scores([&](int tb) {
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const f4 x = *reinterpret_cast<const f4 *>(bias + tb * 32 + i * 2 + hf * 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[tb][i + e] = x[e];
                }
            });
        }
        // int8: the scales of the lane's tokens
        const float *scales = reinterpret_cast<const float *>(here + 2 * C::half) + own + hf * 4;
        if constexpr (I8)
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const f4 x = *reinterpret_cast<const f4 *>(scales + tb * 32 + i * 2);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[tb][i + e] *= x[e];
                }
        // The running maximum only moves when a score passes it by 2^8: weights up to
        // 256 are as exact, and most steps leave the sums as they are.
        float top = -INFINITY;
#pragma unroll
        for (int tb = 0; tb < TB; ++tb)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, s[tb][i]);
        top *= a.scale2;
        if (__any(top > m + 8.0f)) {
            top = fmaxf(fmaxf(top, __shfl_xor(top, 32)), m);
            const float f = top == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - top);
            m = top;
            if (j0 != job.begin) {   // (zeros so far)
                l *= f;
#pragma unroll
                for (int db = 0; db < DB; ++db) o[db] *= f;
            }
        }
        // Group g of 16 slots: its weights are computed between the products of the
        // group before, and its values read there.
        constexpr int GROUPS = TB * 2;
        const float base = m == -INFINITY ? 0.0f : -m;
        constexpr int VB = DB < 8 ? 2 : 1;   // (with 8 products a group, the next group's values take the places of those used)
        u4 v[VB][DB], p[2][WP];
        auto read_v = [&](int g, int db) {
            const char *at = here + v_at[db] + g * 16 * PC * 16;
            const u2 x = read_turned(at), y = read_turned(at + 8 * PC * 16);
            v[g % VB][db] = u4{x[0], x[1], y[0], y[1]};
        };
        auto weigh = [&](int g, int i) {   // two weights
            const int tb = g / 2, e = g % 2 * 8 + i * 2;
            float w0 = __builtin_amdgcn_exp2f(fmaf(s[tb][e], a.scale2, base));
            float w1 = __builtin_amdgcn_exp2f(fmaf(s[tb][e + 1], a.scale2, base));
            l += w0 + w1;
            if constexpr (I8) {
                const f2 x = *reinterpret_cast<const f2 *>(scales + KT + tb * 32 + (e / 4) * 8 + e % 4);
                w0 *= x[0], w1 *= x[1];
            }
            uint32_t x[WP];
            split2<WP>(w0, w1, x);
#pragma unroll
            for (int n = 0; n < WP; ++n) p[g & 1][n][i] = x[n];
        };
#pragma unroll
        for (int db = 0; db < DB; ++db) read_v(0, db);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 4; ++i) weigh(0, i);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)
#pragma unroll
            for (int db = 0; db < DB; ++db) {
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int n = 0; n < WP; ++n) o[db] = mfma32(v[g % VB][db], p[g & 1][n], o[db]);
                if (g + 1 < GROUPS) {
                    read_v(g + 1, db);
#pragma unroll
                    for (int i = db * 4 / DB; i < (db + 1) * 4 / DB; ++i) weigh(g + 1, i);
                }
            }
        __builtin_amdgcn_sched_barrier(0);
    }

    // ---- the end: o of lane (col, hf) is d = 32 db + 8 (i / 4) + 4 hf + i % 4 of its
    // row; rows go through LDS, so that they are written whole
    const bool parts = job.to_parts;
    auto place_of = [&](int r) {           // of row r of the problem in out, elements
        const int t = a.by_G.of(r), g = r - t * G;
        return job.out_at + t * a.out_ld + (int64_t)(job.h * G + g) * D;
    };
    auto put_stat = [&](int r, float M, float L) {
        if (parts) *reinterpret_cast<f2 *>(a.stat + (job.part + r) * 2) = f2{M, L};
        else if (a.lse) {
            const int t = a.by_G.of(r), g = r - t * G;
            a.lse[job.lse_at + (int64_t)t * a.hq + g] = M == -INFINITY ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * kLn2;
        }
    };
    l += __shfl_xor(l, 32);
    // A NaN score is in l, but maxima drop it.  A maximum of infinity takes it
    // through every join: exp2(inf - inf) is NaN, other parts count 0 beside it.
    if (l != l) m = INFINITY;
    // (slots that do not count give NaN, too, to a row whose queries are not finite)
    const bool none = any == 0;
    if (none) m = -INFINITY, l = 0.0f;
    __syncthreads();   // (the last step's LDS is read no more)
    if constexpr (WIDE) {
        constexpr bool H = BF16;               // rows of out in bf16, parts in fp32
        constexpr int OP = C::OP;
        char *mine = lds + wave * 32 * OP * 4;
        const float f = parts ? 1.0f : m == -INFINITY ? 0.0f : BF16 ? __builtin_amdgcn_rcpf(l) : 1.0f / l;
        if (hf == 0 && row < job.R) put_stat(row, m, l);
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = col * OP + db * 32 + i * 8 + hf * 4;
                const f4 x = none ? f4{0, 0, 0, 0} : f4{o[db][4 * i], o[db][4 * i + 1], o[db][4 * i + 2], o[db][4 * i + 3]} * f;
                if (H && !parts) store4<true>(mine, at, x);
                else store4<false>(mine, at, x);
            }
        const int first = job.row0 + wave * 32, n = min(32, job.R - first);   // (below 1: none)
        if (H && !parts) {
            for (int x = lane; x < n * PC; x += 64) {
                const int r = x / PC, d = (x - r * PC) * 8;
                if (d >= D) continue;
                // (rows lie 8-byte aligned)
                const u2 lo = *reinterpret_cast<const u2 *>(mine + (r * OP + d) * 2), hi = *reinterpret_cast<const u2 *>(mine + (r * OP + d) * 2 + 8);
                *reinterpret_cast<u4 *>(static_cast<uint16_t *>(a.out) + place_of(first + r) + d) = u4{lo[0], lo[1], hi[0], hi[1]};
            }
        } else {
            for (int x = lane; x < n * (DP / 4); x += 64) {
                const int r = x / (DP / 4), d = (x - r * (DP / 4)) * 4;
                if (d >= D) continue;
                const f4 v = *reinterpret_cast<const f4 *>(mine + (r * OP + d) * 4);
                if (parts) *reinterpret_cast<f4 *>(a.part + (job.part + first + r) * D + d) = v;
                else *reinterpret_cast<f4 *>(static_cast<float *>(a.out) + place_of(first + r) + d) = v;
            }
        }
    } else {
        static_assert(WIDE || C::RW == 1, "waves along the tokens have the same 32 rows");
        float *so = reinterpret_cast<float *>(lds), *st = so + C::TW * 32 * C::OP;
        if (hf == 0) {
            st[(wave * 32 + col) * 2] = m;
            st[(wave * 32 + col) * 2 + 1] = l;
        }
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<f4 *>(so + (wave * 32 + col) * C::OP + db * 32 + i * 8 + hf * 4) =
                    none ? f4{0, 0, 0, 0} : f4{o[db][4 * i], o[db][4 * i + 1], o[db][4 * i + 2], o[db][4 * i + 3]};
        __syncthreads();
        const int rows = min(32, job.R - job.row0);
        // Parts that another launch left for these rows join here.  A wave a row: lane
        // i has the other part i and, below TW, a wave's own; all factors come first.
        const int others = job.others;
        float *of = st + C::TW * 64, *fin = of + kOthers * 32;   // [kOthers][32]; [32][2]: maximum and sum of all
        for (int r = wave; r < rows; r += C::waves) {
            f2 other = {-INFINITY, 0.0f}, own = {-INFINITY, 0.0f};
            if (lane < others) other = reinterpret_cast<const f2 *>(a.stat)[lane * a.rows + job.part + job.row0 + r];
            if (lane < C::TW) own = *reinterpret_cast<const f2 *>(st + (lane * 32 + r) * 2);
            const float M = wave_max(fmaxf(other[0], own[0]));
            const float mo = other[0], mw = own[0];
            const float fo = mo == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mo - M), fw = mw == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mw - M);
            const float L = wave_sum((mo == -INFINITY ? 0.0f : other[1] * fo) + (mw == -INFINITY ? 0.0f : own[1] * fw));
            if (lane < others) of[lane * 32 + r] = fo;
            if (lane < C::TW) st[(lane * 32 + r) * 2] = fw;
            if (lane == 0) {
                fin[r * 2] = M;
                fin[r * 2 + 1] = L;
            }
        }
        __syncthreads();
        // the other parts, by as many threads as the rows leave
        const int quads = DP / 4, items = rows * quads;
        if (others) {
            const int groups = C::threads > items ? C::threads / items : 1, group = (int)threadIdx.x / items;
            for (int x = group < groups ? (int)threadIdx.x - group * items : items; x < items; x += C::threads) {
                const int r = x / quads, d = (x - r * quads) * 4;
                if (d >= D) continue;
                f4 sum = {0, 0, 0, 0};
                const float *other = a.part + (job.part + job.row0 + r) * D + d;
#pragma unroll 8
                for (int i = group; i < others; i += groups) sum += *reinterpret_cast<const f4 *>(other + i * a.rows * D) * of[i * 32 + r];
                // (the waves' own outputs of the row, scaled, make room for the groups')
                if (group == 0) {
#pragma unroll
                    for (int w = 0; w < C::TW; ++w) sum += *reinterpret_cast<const f4 *>(so + (w * 32 + r) * C::OP + d) * st[(w * 32 + r) * 2];
                }
                if (groups > 1) *reinterpret_cast<f4 *>(fin + 64 + (group * items + x) * 4) = sum;
                else *reinterpret_cast<f4 *>(so + r * C::OP + d) = sum;
            }
            __syncthreads();
            if (groups > 1 && (int)threadIdx.x < items) {
                const int r = threadIdx.x / quads, d = (threadIdx.x - r * quads) * 4;
                f4 sum = {0, 0, 0, 0};
                for (int g = 0; g < groups; ++g) sum += *reinterpret_cast<const f4 *>(fin + 64 + (g * items + threadIdx.x) * 4);
                *reinterpret_cast<f4 *>(so + r * C::OP + d) = sum;
            }
            if (groups > 1) __syncthreads();
        }
        for (int x = threadIdx.x; x < items; x += C::threads) {
            const int r = x / quads, d = (x - r * quads) * 4;
            if (d >= D) continue;
            const float M = fin[r * 2], L = fin[r * 2 + 1];
            f4 sum = {0, 0, 0, 0};
            if (others) sum = *reinterpret_cast<const f4 *>(so + r * C::OP + d);
            else
#pragma unroll
                for (int w = 0; w < C::TW; ++w) sum += *reinterpret_cast<const f4 *>(so + (w * 32 + r) * C::OP + d) * st[(w * 32 + r) * 2];
            if (d == 0) put_stat(job.row0 + r, M, L);
            if (parts) *reinterpret_cast<f4 *>(a.part + (job.part + job.row0 + r) * D + d) = sum;
            else store4<BF16>(a.out, place_of(job.row0 + r) + d, sum * (M == -INFINITY ? 0.0f : 1.0f / L));
        }
    }
}

// waves of a SIMD, by the registers they need (fp32 with heads up to 64 fits two either
// way; told so, the compiler leaves out moves to the accumulators' half of the file: 2 x
// 4096 fp32 queries, 1280 keys, 12 heads of 64 102.5 -> 97.1 us)
template <class C>
constexpr int resident() {
    if (C::SRC == PAGES_I8) return C::BF16 && C::DP <= 96 && C::TW == 1 ? 2 : 1;
    if (C::BF16) return C::DP == 96 ? 3 : C::DP <= 128 ? 2 : 1;
    return C::DP == 64 ? 2 : 1;
}

// Keys of part `split`: equal shares in whole steps.
__device__ __forceinline__ void share(int begin, int end, int splits, int split, int step, int &b, int &e) {
    const int per = ((end - begin + splits - 1) / splits + step - 1) / step * step;
    b = min(begin + split * per, end);
    e = min(b + per, end);
}

// The workgroup's number (a launch holds 2^32 threads along x, so that many
// workgroups go on along y; the last are more than there are jobs).
__device__ __forceinline__ int block_of_launch() { return (int)(blockIdx.y * gridDim.x + blockIdx.x); }

// Workgroups go round the 8 XCDs in turn; consecutive jobs, which share keys, are
// given to the same one.
__device__ __forceinline__ uint32_t job_of_block(uint32_t id, uint32_t n) {
    const uint32_t each = n / 8, more = n % 8, x = id % 8;
    return x * each + min(x, more) + id / 8;
}

template <class C>
__global__ void __launch_bounds__(C::threads) __attribute__((amdgpu_waves_per_eu(resident<C>()))) cross_kernel(Args a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    int b, id2;       // sequence; tile, part and head
    const int block = block_of_launch();
    if (block >= a.jobs) return;
    if (a.longest_first) {
        // Each XCD takes its share of the tiles of every sequence, the longest sequence's
        // first: the last workgroups to start are short (5 uneven sequences of 333 fp32
        // queries 45 -> 40 us; 4 of 4096 queries, 300 keys at most, 44.8 -> 44.4).
        const int x = (uint32_t)block % 8, l = (uint32_t)block / 8, rank = a.by_share.of(l), lane = threadIdx.x & 63;
        const int length = lane < a.batch ? min(max(a.lens[lane], 0), a.keys) : -1;
        int mine = 0;
        for (int i = 0; i < a.batch; ++i) {
            const int other = __builtin_amdgcn_readlane(length, i);
            mine += other > length || (other == length && i < lane);
        }
        b = __builtin_ctzll(__ballot(mine == rank));   // (ranks below the batch occur once)
        id2 = x * a.by_share.d + l - rank * a.by_share.d;
    } else {
        // Sequences innermost: their lengths differ, and each XCD gets some of all.  They
        // take turns in being first, or those of one length would meet on the same CUs.
        const int id = job_of_block(block, a.jobs);
        id2 = a.by_batch.of(id);
        const int turn = id - id2 * a.batch + id2 % a.batch;
        b = turn < a.batch ? turn : turn - a.batch;
    }
    const int id3 = a.by_tiles.of(id2), tile = id2 - id3 * a.tiles, h = a.by_splits.of(id3), split = id3 - h * a.splits;
    Job job;
    job.others = 0, job.to_parts = a.splits > 1;
    job.h = h;
    const int queries = a.q_lens ? min(max(a.q_lens[b], 0), a.queries) : a.queries;
    job.R = queries * a.G;
    job.row0 = tile * C::rows;
    if (job.row0 >= job.R) return;
    const int keys = a.lens ? min(max(a.lens[b], 0), a.keys) : a.keys;
    share(0, keys, a.splits, split, C::KT, job.begin, job.end);
    job.first = 0;
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
// holds behind it (a problem a sequence and head), which joins the prefix's parts
// unless it has several itself.
template <class C>
__global__ void __launch_bounds__(C::threads) __attribute__((amdgpu_waves_per_eu(resident<C>()))) prefix_kernel(Args a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int block = block_of_launch();
    if (block >= a.jobs) return;
    const int id = job_of_block(block, a.jobs), id2 = a.by_tiles.of(id), tile = id - id2 * a.tiles;
    Job job;
    job.h = a.by_splits.of(id2);
    job.others = 0, job.to_parts = true;
    const int split = id2 - job.h * a.splits;
    job.R = a.batch * a.G;
    job.row0 = tile * C::rows;
    share(0, a.prefix, a.splits, split, C::KT, job.begin, job.end);
    job.first = 0;
    job.q_at = job.out_at = job.lse_at = 0;
    job.k = job.v = nullptr;
    job.table = a.prefix_table;
    job.mask = nullptr;
    job.part = split * a.rows + (int64_t)job.h * job.R;
    attend_rows<C>(a, job, lds);
}
template <class C>
__global__ void __launch_bounds__(C::threads) __attribute__((amdgpu_waves_per_eu(resident<C>()))) own_kernel(Args a) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int tiles = (a.G + C::rows - 1) / C::rows;
    uint32_t id = block_of_launch();
    if ((int)id >= a.jobs) return;
    const int tile = id % tiles;
    id /= tiles;
    const int split = id % max(a.own_splits, 1);
    id /= max(a.own_splits, 1);
    const int h = id % a.c.heads, b = id / a.c.heads;
    Job job;
    job.h = h;
    job.R = a.G;
    job.row0 = tile * C::rows;
    const int len = min(a.lens[b], a.keys);
    const bool there = len >= a.prefix && len > 0;           // else it is not in the batch
    const int end = there ? len : a.prefix;                  // (its first 16 slots can begin below the prefix)
    share(end > a.prefix ? a.prefix & ~15 : end, end, max(a.own_splits, 1), split, C::KT, job.begin, job.end);
    job.first = a.prefix;
    job.q_at = b * a.q_ld;
    job.out_at = b * a.out_ld;
    job.lse_at = (int64_t)b * a.hq + h * a.G;
    job.k = job.v = nullptr;
    job.table = a.c.table + (int64_t)b * a.c.table_ld;
    job.mask = a.mask ? a.mask + b * a.mask_ld : nullptr;
    job.part = ((int64_t)h * a.batch + b) * a.G;
    job.to_parts = a.own_splits > 1;
    job.others = job.to_parts || !there ? 0 : a.splits;
    if (job.to_parts) job.part += (a.splits + split) * a.rows;
    attend_rows<C>(a, job, lds);
}

constexpr int kJoin = 256;

// Where row `row` of all goes, or that nothing does; parts: how many it has.
template <bool PREFIX>
__device__ __forceinline__ bool row_goes(const Args &a, int row, int64_t &out_at, int64_t &lse_at, int &parts) {
    if constexpr (PREFIX) {
        const int hb = a.by_G.of(row), g = row - hb * a.G, h = a.by_batch.of(hb), b = hb - h * a.batch;
        if (min(a.lens[b], a.keys) < a.prefix || a.lens[b] <= 0) parts = 0;   // not in the batch
        out_at = b * a.out_ld + (int64_t)(h * a.G + g) * a.c.D;
        lse_at = (int64_t)b * a.hq + h * a.G + g;
    } else {
        const int tg = a.by_G.of(row), g = row - tg * a.G, bh = a.by_queries.of(tg), t = tg - bh * a.queries;
        const int b = a.by_heads.of(bh), h = bh - b * a.c.heads;
        if (a.q_lens && t >= a.q_lens[b]) return false;
        out_at = b * a.out_stride + t * a.out_ld + (int64_t)(h * a.G + g) * a.c.D;
        lse_at = ((int64_t)b * a.queries + t) * a.hq + h * a.G + g;
    }
    return true;
}

// Joins the parts of rows, TPR threads a row: a wave where there are many rows, a
// workgroup where there are few.
template <bool BF16, bool PREFIX, int TPR>
__global__ void __launch_bounds__(kJoin) join_rows_kernel(Args a) {
    __shared__ float s_f[kJoin / TPR][2 * kOthers];
    __shared__ f4 s_o[TPR == 64 ? 1 : kJoin];
    const int lane = threadIdx.x & 63, D = a.c.D, quads = D / 4, t0 = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * (kJoin / TPR) + threadIdx.x / TPR;
    if (row >= a.rows) return;   // (whole waves; a workgroup a row: none)
    int n = a.splits + a.own_splits;
    int64_t out_at, lse_at;
    if (!row_goes<PREFIX>(a, (int)row, out_at, lse_at, n)) return;
    const f2 *st = reinterpret_cast<const f2 *>(a.stat) + row;
    float M, L;
    join_stats(st, n, a.rows, lane, M, L);
    float *f = s_f[threadIdx.x / TPR];
    for (int i = t0; i < n; i += TPR) {   // (a part without keys holds zeros)
        const float m = st[i * a.rows][0];
        f[i] = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - M);
    }
    if constexpr (TPR > 64) __syncthreads();
    // the threads of a row take its quads, several parts at a time
    const int groups = TPR / quads, group = t0 / quads, d = (t0 - group * quads) * 4;
    f4 sum = {0, 0, 0, 0};
    if (group < groups) {
        const float *part = a.part + row * D + d;
#pragma unroll 8
        for (int i = group; i < n; i += groups) sum += *reinterpret_cast<const f4 *>(part + i * a.rows * D) * f[i];
    }
    if constexpr (TPR > 64) {
        s_o[threadIdx.x] = sum;
        __syncthreads();
        if (t0 < quads)
            for (int g = 1; g < groups; ++g) sum += s_o[t0 + g * quads];
    } else {
        // (groups are runs of lanes)
        const f4 own = sum;
        for (int g = 1; g < groups; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = own[e];
                sum[e] += __shfl(x, (lane + g * quads) & 63);
            }
    }
    const float inv = M == -INFINITY ? 0.0f : 1.0f / L;
    if (t0 < quads) store4<BF16>(a.out, out_at + d, sum * inv);
    if (t0 == 0 && a.lse) a.lse[lse_at] = M == -INFINITY ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

// The same for rows of a few parts: a thread takes a quad of a row, all of its
// parts' statistics and outputs in flight at once (5 uneven sequences of 333 fp32
// queries, 26640 rows of 4 parts: the call 41.0 -> 40.1 us).
constexpr int kFew = 8;
template <bool BF16, bool PREFIX>
__global__ void __launch_bounds__(kJoin) join_few_kernel(Args a) {
    const int quads = a.c.D / 4, x = (int)(blockIdx.x * kJoin + threadIdx.x), row = a.by_quads.of(x), d = (x - row * quads) * 4;
    if (row >= a.rows) return;
    int64_t out_at, lse_at;
    int n = a.splits + a.own_splits;
    if (!row_goes<PREFIX>(a, row, out_at, lse_at, n)) return;
    f2 st[kFew];
    f4 part[kFew];
#pragma unroll
    for (int i = 0; i < kFew; ++i)
        if (i < n) {
            st[i] = reinterpret_cast<const f2 *>(a.stat)[i * a.rows + row];
            part[i] = *reinterpret_cast<const f4 *>(a.part + (i * a.rows + row) * a.c.D + d);
        }
    float M = -INFINITY, L = 0.0f;
#pragma unroll
    for (int i = 0; i < kFew; ++i)
        if (i < n) M = fmaxf(M, st[i][0]);
    f4 sum = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kFew; ++i)
        if (i < n) {   // (a part without keys holds zeros)
            const float m = st[i][0], f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - M);
            if (m != -INFINITY) L += st[i][1] * f;
            sum += part[i] * f;
        }
    store4<BF16>(a.out, out_at + d, sum * (M == -INFINITY ? 0.0f : 1.0f / L));
    if (d == 0 && a.lse) a.lse[lse_at] = M == -INFINITY ? -INFINITY : (M + __builtin_amdgcn_logf(L)) * kLn2;
}

template <bool BF16, bool PREFIX>
void join(const Args &a, hipStream_t s) {
    if (a.splits + a.own_splits <= kFew) {
        const int64_t threads = a.rows * (a.c.D / 4);
        hipLaunchKernelGGL((join_few_kernel<BF16, PREFIX>), dim3((unsigned)((threads + kJoin - 1) / kJoin)), dim3(kJoin), 0, s, a);
    } else if (a.rows >= 8 * device_cus())
        hipLaunchKernelGGL((join_rows_kernel<BF16, PREFIX, 64>), dim3((unsigned)((a.rows + 3) / 4)), dim3(kJoin), 0, s, a);
    else
        hipLaunchKernelGGL((join_rows_kernel<BF16, PREFIX, kJoin>), dim3((unsigned)a.rows), dim3(kJoin), 0, s, a);
}

// The kernel's shape: many rows divide over the waves, few leave the waves the
// tokens.  There, four waves a workgroup (heads of 65 to 128: one workgroup a CU) where a
// CU has no more than one step of them to do, two (two a CU, which overlap) beyond: 5
// sequences behind 1999 int8 tokens 21.0 us with four, 25.8 with two; 64 behind 16384
// 65.0 and 60.4; 256 of 500 keys 45.1 and 38.2; 1 x 32760 keys 49.9 and 46.4.
enum Kind { NARROW2 = 2, NARROW4 = 4, WIDE = 0 };
constexpr int kNarrow = 32;
Kind kind_of(int DP, int64_t R, int64_t problems, int64_t keys) {
    if (R > kNarrow) return WIDE;
    return DP == 64 || (DP <= 128 && problems * ((keys + 127) / 128) <= device_cus()) ? NARROW4 : NARROW2;
}
int padded(int D) { return D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : 256; }
int rows_of(Kind k) { return k == WIDE ? 128 : 32; }
int step_of(Kind k) { return k == WIDE ? 64 : k * 32; }

// Parts of a problem of `keys` where `jobs` workgroups take one each, of `least`
// steps at the least: as many as make two workgroups a CU; fp32 calls with heads up to
// 64, whose steps take longer, four, so that uneven ones even out (5 uneven sequences of
// 333 x 1999 47 -> 40 us; heads of 128, one workgroup a CU, lose: 4 of 1000 x 2000 80 -> 100;
// and bf16 pays more for the parts: 77 queries x 32760 56 -> 66).
int parts_of(int64_t jobs, int64_t keys, int step, int least, bool twice) {
    const int64_t steps = (keys + step - 1) / step, enough = (twice ? 2 : 1) * (int64_t)device_cus();
    if (jobs >= enough || jobs < 1) return 1;
    return (int)std::max<int64_t>(1, std::min<int64_t>({steps / least, 2 * enough / jobs, kOthers}));
}

template <class F>
void by_dim(int DP, F f) {
    if (DP == 64) f(std::integral_constant<int, 64>{});
    else if (DP == 96) f(std::integral_constant<int, 96>{});
    else if (DP == 128) f(std::integral_constant<int, 128>{});
    else f(std::integral_constant<int, 256>{});
}
template <int DP, bool B, Source S, int WAVES>
using Narrow = Shape<DP, B, 1, WAVES, S>;
// calls f with the shape of a narrow kind (those that kind_of() gives)
template <int DP, bool B, Source S, class F>
void narrow(Kind k, F f) {
    if constexpr (DP <= 128)
        if (k == NARROW4) return f(Narrow<DP, B, S, 4>{});
    if constexpr (DP > 64) f(Narrow<DP, B, S, 2>{});
}

template <class C>
int go(void (*kern)(Args), int64_t jobs, Args &a, hipStream_t s) {
    constexpr int64_t most = 1 << 23;   // workgroups along x
    a.jobs = (int)jobs;
    const dim3 grid((unsigned)std::min(jobs, most), (unsigned)((jobs + most - 1) / most));
    const int err = ensure_dyn_lds(reinterpret_cast<const void *>(kern), C::lds);
    if (err != (int)hipSuccess) return err;
    hipLaunchKernelGGL(kern, grid, dim3(C::threads), C::lds, s, a);
    return (int)hipSuccess;
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }

struct CrossPlan {
    Kind kind;
    int DP, tiles, splits;
    int64_t rows, grid;
    size_t part, stat;
};
CrossPlan cross_plan(const rq_states *s, int64_t queries, int q_heads, bool bf16) {
    CrossPlan p{};
    const int G = q_heads / s->heads;
    const int64_t R = queries * G;
    p.DP = padded(s->head_dim);
    p.kind = kind_of(p.DP, R, (int64_t)s->heads * s->batch, s->keys);
    const int rows = rows_of(p.kind);
    p.tiles = (int)((R + rows - 1) / rows);
    const int64_t jobs = (int64_t)p.tiles * s->heads * s->batch;
    p.splits = parts_of(jobs, s->keys, step_of(p.kind), 4, !bf16 && p.DP == 64);
    p.grid = jobs * p.splits;
    p.rows = R * s->heads * s->batch;
    if (p.splits > 1) {
        p.part = round16((size_t)p.splits * p.rows * s->head_dim * 4);
        p.stat = round16((size_t)p.splits * p.rows * 8);
    }
    return p;
}

struct PrefixPlan {
    Kind kind, own_kind;
    int DP, tiles, splits, own_splits;
    int64_t rows, grid, own_grid;
    size_t part, stat;
};
PrefixPlan prefix_plan(const rq_kv_cache *c, int q_heads, bool bf16, int64_t prefix, int64_t max_len) {
    PrefixPlan p{};
    const int G = q_heads / c->heads;
    const int64_t R = (int64_t)c->batch * G;
    p.DP = padded(c->head_dim);
    p.kind = kind_of(p.DP, R, c->heads, prefix);
    const int rows = rows_of(p.kind);
    p.tiles = (int)((R + rows - 1) / rows);
    if (prefix > 0) p.splits = parts_of((int64_t)p.tiles * c->heads, prefix, step_of(p.kind), 1, !bf16 && p.DP == 64);
    p.grid = (int64_t)p.tiles * c->heads * p.splits;
    const int own_tiles = (G + 31) / 32;
    p.own_kind = kind_of(p.DP, 1, (int64_t)own_tiles * c->heads * c->batch, max_len - prefix);
    p.own_splits = parts_of((int64_t)own_tiles * c->heads * c->batch, max_len - prefix, step_of(p.own_kind), 4, false);
    p.own_grid = (int64_t)own_tiles * c->heads * c->batch * p.own_splits;
    p.rows = R * c->heads;
    const int parts = p.splits + (p.own_splits > 1 ? p.own_splits : 0);
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
    return cross_plan(s, queries, q_heads, bf16).rows < (int64_t(1) << 25);
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
    a.by_G = over(a.G), a.by_batch = over(a.batch), a.by_tiles = over(a.tiles), a.by_splits = over(a.splits);
    // (ranking costs a few instructions a sequence; the share has to be the same for all XCDs)
    const int64_t each = p.grid / st->batch;
    a.longest_first = st->lens && st->batch > 1 && st->batch <= 16 && each % 8 == 0;
    a.by_share = over(std::max<int64_t>(each / 8, 1));
    a.by_queries = over(queries), a.by_heads = over(a.c.heads), a.by_quads = over(a.c.D / 4);
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
        using W = Shape<DP, B, 4, 1, STATES>;
        if (p.kind == WIDE) err = go<W>(cross_kernel<W>, p.grid, a, s);
        else narrow<DP, B, STATES>(p.kind, [&](auto n) { err = go<decltype(n)>(cross_kernel<decltype(n)>, p.grid, a, s); });
    };
    by_dim(p.DP, [&](auto dp) { bf16 ? run(dp, std::true_type{}) : run(dp, std::false_type{}); });
    if (err != 0) return err;
    if (p.splits > 1) bf16 ? join<true, false>(a, s) : join<false, false>(a, s);
    return (int)hipGetLastError();
}

bool prefix_fits(const rq_kv_cache *c, int q_heads, int bf16, int64_t prefix, int64_t max_len) {
    return prefix_plan(c, q_heads, bf16, prefix, max_len).rows < (int64_t(1) << 25);
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
    a.by_G = over(a.G), a.by_batch = over(a.batch), a.by_tiles = over(a.tiles), a.by_splits = over(std::max(a.splits, 1));
    a.by_quads = over(a.c.D / 4);
    set_scale(a, scale);
    a.part = static_cast<float *>(workspace);
    a.stat = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.part);
    hipStream_t s = static_cast<hipStream_t>(stream);
    int err = 0;
    auto run = [&](auto dp, auto b, auto src) {
        constexpr int DP = decltype(dp)::value;
        constexpr bool B = decltype(b)::value;
        constexpr Source S = decltype(src)::value;
        using W = Shape<DP, B, 4, 1, S>;
        if (p.grid > 0) {
            if (p.kind == WIDE) err = go<W>(prefix_kernel<W>, p.grid, a, s);
            else narrow<DP, B, S>(p.kind, [&](auto n) { err = go<decltype(n)>(prefix_kernel<decltype(n)>, p.grid, a, s); });
        }
        if (err == 0) narrow<DP, B, S>(p.own_kind, [&](auto n) { err = go<decltype(n)>(own_kernel<decltype(n)>, p.own_grid, a, s); });
    };
    by_dim(p.DP, [&](auto dp) {
        auto typed = [&](auto b) {
            if (c->dtype == RQ_I8) run(dp, b, std::integral_constant<Source, PAGES_I8>{});
            else run(dp, b, std::integral_constant<Source, PAGES>{});
        };
        bf16 ? typed(std::true_type{}) : typed(std::false_type{});
    });
    if (err != 0) return err;
    if (p.own_splits > 1) bf16 ? join<true, true>(a, s) : join<false, true>(a, s);
    return (int)hipGetLastError();
}

}  // namespace rq
