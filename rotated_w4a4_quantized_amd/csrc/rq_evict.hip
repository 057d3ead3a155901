// rq_evict.hip -- eviction from a cache by accumulated attention weight.
//
// Per (sequence, head) row of n slots: the keep first in the order (protected,
// weight descending, slot ascending) stay.  Survivors above `keep` move into
// the free slots below it: a move never reads what another one writes, and a
// cache a little over its budget moves a few tokens instead of closing ranks.
//
// Selection is one workgroup a row: short rows are bound by the chain of loads and
// barriers (2080 slots: 10 us with the moves, 2 of them to read, 1 a digit), long
// ones by the instructions over a row's slots on one CU (32749 slots: 36 us).  The
// moves are a copy, bound by HBM where they are many (193 MB moved in 88 us, 4.4
// TB/s read and written).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rq_attn_util.h"
#include "rq_internal.h"

namespace rq {
namespace {

using attn::Cache;

typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef int32_t i4 __attribute__((ext_vector_type(4)));

struct Args {
    Cache c;
    const int32_t *lens;
    int32_t *lens_out, *pos_out;
    float *weight_out;
    int32_t *count;      // [rows] moves of a row
    int32_t *moves;      // [rows][2][most] free slots, then survivors
    int64_t slots;
    int32_t max_len, keep, recent, sink, most, row_bytes;
};

// Order-preserving map of a weight to unsigned: NaN lowest, protected highest.
__device__ __forceinline__ uint32_t key_of(float w, bool held) {
    if (held) return 0xffffffffu;
    if (w != w) return 0u;
    const uint32_t b = __builtin_bit_cast(uint32_t, w);
    // (-0 and +0 are one weight)
    return b == 0x80000000u ? 0x80000000u : b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Moves of a row, at most, that the workgroup which found them copies too.  With
// limits of 128, 256 and 512, 32 int8 sequences of 8 heads take 21.1, 18.9, 18.8 us
// for 256 moves a row and 29.6, 29.0, 27.1 for 512, where 4 bf16 sequences take 15.9,
// 15.9, 17.8: few rows leave the device idle during long moves.
constexpr int kFused = 256;
constexpr int kBatch = 8;   // steps whose loads are in flight together, where keys are not held
constexpr int kThreads = 1024, kSelWaves = kThreads / 64;

// inclusive sum over the lanes up to this one: shifts within rows of 16, then
// the rows' last lanes passed on
__device__ __forceinline__ int wave_scan(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
    return x;
}
// the largest of the lanes, in lane 63
__device__ __forceinline__ int wave_max63(int x) {
    x = max(x, __builtin_amdgcn_update_dpp(x, x, 0x111, 0xf, 0xf, false));
    x = max(x, __builtin_amdgcn_update_dpp(x, x, 0x112, 0xf, 0xf, false));
    x = max(x, __builtin_amdgcn_update_dpp(x, x, 0x114, 0xf, 0xf, false));
    x = max(x, __builtin_amdgcn_update_dpp(x, x, 0x118, 0xf, 0xf, false));
    x = max(x, __builtin_amdgcn_update_dpp(x, x, 0x142, 0xa, 0xf, false));
    x = max(x, __builtin_amdgcn_update_dpp(x, x, 0x143, 0xc, 0xf, false));
    return x;
}
// sums of v[i] over the waves before this one and over all
__device__ __forceinline__ void over_waves(const int *v, int wave, int &before, int &all) {
    before = all = 0;
#pragma unroll
    for (int i = 0; i < kSelWaves; ++i) {
        const int x = v[i];
        before += i < wave ? x : 0;
        all += x;
    }
}
// Place of a digit's count: 32 digits and a gap of 4 words, so that lanes that
// each read 32 digits in a row meet different banks.
__device__ __forceinline__ int place_of(uint32_t d) { return (int)(d + (d >> 5) * 4); }

// Copies the moves [first, last) of a row by the whole workgroup (THREADS), VEC
// bytes a load: the rows of ROWS moves at a time through s_rows, then their keys
// and values as one run of vectors, U of a thread in flight.
template <int VEC, int THREADS, int ROWS, int U>
__device__ void copy_moves(const Args &a, int b, int h, const int32_t *free_list, const int32_t *up_list, int first, int last, int64_t (*s_rows)[ROWS]) {
    const int t = threadIdx.x;
    for (int at = first; at < last; at += ROWS) {
        const int n = min(ROWS, last - at);
        bool scaled = false;
        if (t < n) {
            const int64_t to = a.c.row(b, h, free_list[at + t]), from = a.c.row(b, h, up_list[at + t]);
            const bool both = to >= 0 && from >= 0;
            s_rows[0][t] = both ? to : -1;
            s_rows[1][t] = from;
            scaled = both && a.c.k_scale;
        }
        __syncthreads();
        float ks = 0.0f, vs = 0.0f;      // (asked for after the barrier, which would wait for them)
        if (scaled) {
            ks = a.c.k_scale[s_rows[1][t]];
            vs = a.c.v_scale[s_rows[1][t]];
        }
        const int vecs = a.row_bytes / VEC, all = n * vecs * 2;
        for (int i0 = t; i0 < all; i0 += THREADS * U) {
            u4 x[U];
            char *to[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * THREADS;
                to[u] = nullptr;
                if (i >= all) continue;
                const int m = i / (2 * vecs), v = i - m * 2 * vecs;
                if (s_rows[0][m] < 0) continue;
                char *base = static_cast<char *>(v < vecs ? a.c.k : a.c.v);
                const int off = (v < vecs ? v : v - vecs) * VEC;
                to[u] = base + s_rows[0][m] * a.row_bytes + off;
                const char *from = base + s_rows[1][m] * a.row_bytes + off;
                if constexpr (VEC == 16) x[u] = *reinterpret_cast<const u4 *>(from);
                else {
                    const u2 y = *reinterpret_cast<const u2 *>(from);
                    x[u][0] = y[0];
                    x[u][1] = y[1];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (to[u]) {
                    if constexpr (VEC == 16) *reinterpret_cast<u4 *>(to[u]) = x[u];
                    else *reinterpret_cast<u2 *>(to[u]) = u2{x[u][0], x[u][1]};
                }
        }
        if (scaled) {
            a.c.k_scale[s_rows[0][t]] = ks;
            a.c.v_scale[s_rows[0][t]] = vs;
        }
        __syncthreads();
    }
}

// One row.  Wave w owns the slots (w iters + i) 64 + lane, i < iters, so slots
// ascend along waves, steps and lanes: ranks within a wave are counts of ballot
// bits, and one exchange between the waves turns them into ranks in the row.
// K > 0: up to K steps, weights and positions held in registers and read once;
// K == 0: any length, read again in each pass (they come from the caches).
//
// The keep-th largest key is found by digits of 11, 11 and 10 bits, each with a
// histogram of the keys that share the digits before; it ends early when a
// digit's keys are all needed.
template <int K, bool FUSED>
__global__ void __launch_bounds__(kThreads) select_kernel(Args a) {
    __shared__ __align__(16) int s_hist[3][2048 + 64 * 4];
    __shared__ __align__(16) int s_wave[4][kSelWaves];
    __shared__ uint32_t s_digit;
    __shared__ int s_above, s_in;
    __shared__ int64_t s_rows[2][FUSED ? kFused : 1];
    const int row = blockIdx.x, b = row / a.c.heads, t = threadIdx.x, lane = t & 63;
    const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int n = min(max(a.lens[b], 0), a.max_len);
    const float *w_in = a.c.weight + row * a.slots;
    const int32_t *p_in = a.c.pos + row * a.slots;
    float *w_out = a.weight_out + row * a.slots;
    int32_t *p_out = a.pos_out + row * a.slots;
    if (FUSED && row == b * a.c.heads && t == 0) a.lens_out[b] = min(n, a.keep);
    if (n <= a.keep) {
        if (w_out != w_in || p_out != p_in)
            for (int j = t; j < n; j += kThreads) {
                w_out[j] = w_in[j];
                p_out[j] = p_in[j];
            }
        if (!FUSED && t == 0) a.count[row] = 0;
        return;
    }
    const int iters = (n + kThreads - 1) / kThreads;
    const int base = wave * iters * 64 + lane;
    constexpr int R = K ? K : 1;
    uint32_t kr[R];
    int32_t pr[R];           // (until the newest is known)
    int newest = -1;
    if constexpr (K > 0) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int j = base + i * 64;
            const bool in = i < iters && j < n;
            kr[i] = in ? __builtin_bit_cast(uint32_t, w_in[j]) : 0u;
            pr[i] = in ? p_in[j] : -1;
            newest = max(newest, pr[i]);
        }
    } else
        for (int i = 0; i < iters; ++i)
            if (base + i * 64 < n) newest = max(newest, p_in[base + i * 64]);
    for (int i = t; i < 3 * (2048 + 64 * 4); i += kThreads) (&s_hist[0][0])[i] = 0;
    newest = wave_max63(newest);
    if (lane == 63) s_wave[0][wave] = newest;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kSelWaves; ++i) newest = max(newest, s_wave[0][i]);
    newest = __builtin_amdgcn_readlane(newest, 63);
    const int from = newest - a.recent;
    auto protects = [&](int32_t p) { return p < a.sink || p > from; };
    if constexpr (K > 0) {
#pragma unroll
        for (int i = 0; i < K; ++i) kr[i] = key_of(__builtin_bit_cast(float, kr[i]), protects(pr[i]));
    }
    // f(j, the slot exists, its key) for this thread's slots; all lanes of a wave
    // take part in every step
    auto each = [&](auto f) {
        if constexpr (K > 0) {
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (i < iters) f(base + i * 64, base + i * 64 < n, kr[i]);
        } else
            for (int i0 = 0; i0 < iters; i0 += kBatch) {
                float w[kBatch];
                int32_t p[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int j = base + (i0 + u) * 64;
                    const bool in = i0 + u < iters && j < n;
                    w[u] = in ? w_in[j] : 0.0f;
                    p[u] = in ? p_in[j] : 0;
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
                    if (i0 + u < iters) f(base + (i0 + u) * 64, base + (i0 + u) * 64 < n, key_of(w[u], protects(p[u])));
            }
    };

    // the threshold: keys above it stay, and the first `ties` keys equal to it
    uint32_t thr = 0;
    int need = a.keep;       // of the keys that share the digits found so far
    bool all_in = false;
    for (int pass = 0; pass < 3 && !all_in; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t digits = pass == 2 ? 1024 : 2048;
        const uint32_t seen = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
        each([&](int, bool in, uint32_t k) {
            if (in && (k & seen) == thr) atomicAdd(&s_hist[pass][place_of((k >> shift) & (digits - 1))], 1);
        });
        __syncthreads();
        // the first wave finds the digit: the 32 that it is among (lane l has
        // digits 2047 - 32 l downwards), then which of them (a lane each)
        if (wave == 0) {
            int sum = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const i4 v = *reinterpret_cast<const i4 *>(&s_hist[pass][place_of(2016 - 32 * lane) + 4 * i]);
                sum += v[0] + v[1] + v[2] + v[3];
            }
            int upto = wave_scan(sum);
            const int group = __ffsll((long long)__ballot(upto >= need)) - 1;   // (the last sum is all keys)
            const int above = __builtin_amdgcn_readlane(upto - sum, group);
            const int top = 2047 - 32 * group;
            const int one = lane < 32 ? s_hist[pass][place_of(top - lane)] : 0;
            upto = above + wave_scan(one);
            const int x = __ffsll((long long)__ballot(upto >= need)) - 1;
            if (lane == x) {
                s_digit = top - x;
                s_above = upto - one;
                s_in = one;
            }
        }
        __syncthreads();
        thr |= s_digit << shift;
        need -= s_above;
        all_in = need == s_in;
    }
    // (ended early: every key with these digits stays, and thr is their lower bound)
    const int ties = all_in ? 0x7fffffff : need;
    // Ended early, keys from thr up stay; otherwise those above it and some ties.
    int tie_at = 0;
    if (!all_in) {
        int tied = 0, all;
        each([&](int, bool in, uint32_t k) { tied += __popcll(__ballot(in && k == thr)); });
        if (lane == 0) s_wave[2][wave] = tied;
        __syncthreads();
        over_waves(s_wave[2], wave, tie_at, all);
    }
    const uint64_t below = (1ull << lane) - 1;
    uint32_t stay_bits = 0;   // K > 0: of this thread's slots, so that they are found once
    auto walk = [&](auto f) {   // f(i, the slot stays, is a free place, is a survivor from above)
        int at = tie_at, i = 0;
        each([&](int j, bool in, uint32_t k) {
            bool stays;
            if (all_in) stays = in && k >= thr;
            else {
                const bool tie = in && k == thr;
                const uint64_t m = __ballot(tie);
                stays = in && (k > thr || (tie && at + __popcll(m & below) < ties));
                at += __popcll(m);
            }
            f(i++, j, stays, in && !stays && j < a.keep, stays && j >= a.keep);
        });
    };
    int frees = 0, ups = 0;
    walk([&](int i, int, bool stays, bool is_free, bool is_up) {
        if (K > 0) stay_bits |= (uint32_t)stays << i;
        frees += __popcll(__ballot(is_free));
        ups += __popcll(__ballot(is_up));
    });
    if (lane == 0) {
        s_wave[1][wave] = frees;
        s_wave[3][wave] = ups;
    }
    __syncthreads();
    int free_at, up_at, total, all_free;
    over_waves(s_wave[1], wave, free_at, all_free);
    over_waves(s_wave[3], wave, up_at, total);
    // the lists: here if this workgroup alone reads them
    __shared__ int32_t s_list[2][FUSED ? kFused : 1];
    int32_t *free_list = FUSED ? s_list[0] : a.moves + (int64_t)row * 2 * a.most;
    int32_t *up_list = FUSED ? s_list[1] : free_list + a.most;
    auto list = [&](int j, bool is_free, bool is_up) {
        const uint64_t mf = __ballot(is_free), mu = __ballot(is_up);
        if (is_free) free_list[free_at + __popcll(mf & below)] = j;
        if (is_up) up_list[up_at + __popcll(mu & below)] = j;
        free_at += __popcll(mf);
        up_at += __popcll(mu);
    };
    if constexpr (K > 0) {
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (i < iters) {
                const int j = base + i * 64;
                const bool stays = stay_bits >> i & 1;
                list(j, j < n && !stays && j < a.keep, stays && j >= a.keep);
            }
    } else
        walk([&](int, int j, bool, bool is_free, bool is_up) { list(j, is_free, is_up); });
    if (!FUSED && t == 0) a.count[row] = total;
    __threadfence_block();
    __syncthreads();
    // Weights and positions last, for the places written may be the ones read
    // above: apart from the inputs, first what lies below keep; then the moves,
    // which fill every place there that did not stay.
    if (w_out != w_in || p_out != p_in) {
        for (int j = t * 4; j < a.keep; j += kThreads * 4) {
            if (j + 4 <= a.keep) {
                *reinterpret_cast<u4 *>(w_out + j) = *reinterpret_cast<const u4 *>(w_in + j);
                *reinterpret_cast<u4 *>(p_out + j) = *reinterpret_cast<const u4 *>(p_in + j);
            } else
                for (int e = j; e < a.keep; ++e) {
                    w_out[e] = w_in[e];
                    p_out[e] = p_in[e];
                }
        }
        __threadfence_block();
        __syncthreads();
    }
    for (int i0 = t; i0 < total; i0 += kThreads * 4) {   // (four moves of a thread in flight)
        int to[4];
        float w[4];
        int32_t p[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kThreads;
            const bool in = i < total;
            to[u] = in ? free_list[i] : -1;
            const int up = in ? up_list[i] : 0;
            w[u] = w_in[up];
            p[u] = p_in[up];
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (to[u] >= 0) {
                w_out[to[u]] = w[u];
                p_out[to[u]] = p[u];
            }
    }
    if constexpr (FUSED) {
        const int h = row - b * a.c.heads;
        if (a.row_bytes % 16 == 0) copy_moves<16, kThreads, kFused, 4>(a, b, h, free_list, up_list, 0, total, s_rows);
        else copy_moves<8, kThreads, kFused, 4>(a, b, h, free_list, up_list, 0, total, s_rows);
    }
}

constexpr int kChunk = 64;   // moves of a workgroup (32 to 128 measured alike)

// Keys and values of the moves, and the lengths: nothing reads those any more, so
// lens_out may be lens.
template <int VEC>
__global__ void __launch_bounds__(256) move_kernel(Args a, int chunks, int lens_groups) {
    __shared__ int64_t s_rows[2][kChunk];
    if ((int)blockIdx.x < lens_groups) {
        const int b = blockIdx.x * 256 + threadIdx.x;
        if (b < a.c.batch) a.lens_out[b] = min(min(max(a.lens[b], 0), a.max_len), a.keep);
        return;
    }
    const int id = blockIdx.x - lens_groups, row = id / chunks, first = (id - row * chunks) * kChunk;
    const int count = a.count[row];
    if (first >= count) return;
    const int b = row / a.c.heads, h = row - b * a.c.heads;
    const int32_t *free_list = a.moves + (int64_t)row * 2 * a.most, *up_list = free_list + a.most;
    copy_moves<VEC, 256, kChunk, 4>(a, b, h, free_list, up_list, first, min(count, first + kChunk), s_rows);
}

int most_moves(int keep, int64_t max_len) {
    return (int)std::max<int64_t>(0, std::min<int64_t>(keep, max_len - keep));
}

// workgroups of move_kernel: for a row's moves, and for the lengths
int64_t move_chunks(int keep, int64_t max_len) { return (most_moves(keep, max_len) + kChunk - 1) / kChunk; }
int64_t lens_groups_of(const rq_kv_cache *c) { return (c->batch + 255) / 256; }

}  // namespace

// (a launch holds 2^32 threads: 1024 a row for the selection, 256 a workgroup of the moves)
bool evict_fits(const rq_kv_cache *c, int keep, int64_t max_len) {
    const int64_t rows = (int64_t)c->batch * c->heads;
    return rows < (1 << 22) && move_chunks(keep, max_len) * rows + lens_groups_of(c) < (1 << 24);
}

size_t evict_workspace_bytes(const rq_kv_cache *c, int keep, int64_t max_len) {
    const size_t rows = (size_t)c->batch * c->heads;
    return (rows + rows * 2 * most_moves(keep, max_len)) * 4;
}

int launch_cache_evict(const rq_kv_cache *c, const int32_t *lens, int64_t max_len, int keep,
                       int recent, int sink, int32_t *lens_out, float *weight_out,
                       int32_t *pos_out, void *workspace, void *stream) {
    Args a{};
    a.c = device_cache(c);
    a.lens = lens, a.lens_out = lens_out, a.weight_out = weight_out, a.pos_out = pos_out;
    const int rows = c->batch * c->heads;
    a.count = static_cast<int32_t *>(workspace);
    a.moves = a.count + rows;
    a.slots = (int64_t)c->table_ld * c->page;
    a.max_len = (int)max_len, a.keep = keep, a.recent = recent, a.sink = sink;
    a.most = most_moves(keep, max_len);
    a.row_bytes = c->head_dim * (c->dtype == RQ_I8 ? 1 : 2);
    hipStream_t s = static_cast<hipStream_t>(stream);
    // Few moves are done by the workgroup that found them.  (Not with lens_out in
    // place: another row of the sequence may still have to read its length.  Two
    // launches take 9.3 + 4.2 us where one takes 10.0, 2080 slots to 2048, and 10.9 +
    // 11.0 where one takes 18.3, 32 int8 sequences of 4352 to 4096.)
    const bool fused = a.most <= kFused && lens_out != lens;
    const int64_t chunks = move_chunks(keep, max_len), lens_groups = lens_groups_of(c);
    auto select = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(rows), dim3(kThreads), 0, s, a); };
    auto pick = [&](auto f) {
        constexpr bool F = decltype(f)::value;
        // (steps held in registers, as few as will do, or none: 2048 slots take 8.9 us
        // with 2, 10.0 with 8, 14.2 with none; 8192 16.4 with 8, 22.9 with 32, 25.7 with
        // none; 32768 41.4 with 32, 70.9 with none)
        const int64_t iters = (max_len + kThreads - 1) / kThreads;
        if (iters <= 2) select(select_kernel<2, F>);
        else if (iters <= 8) select(select_kernel<8, F>);
        else if (iters <= 32) select(select_kernel<32, F>);
        else select(select_kernel<0, F>);
    };
    if (fused) pick(std::true_type{});
    else {
        pick(std::false_type{});
        const dim3 grid((unsigned)(chunks * rows + lens_groups));
        if (a.row_bytes % 16 == 0) hipLaunchKernelGGL(move_kernel<16>, grid, dim3(256), 0, s, a, (int)chunks, (int)lens_groups);
        else hipLaunchKernelGGL(move_kernel<8>, grid, dim3(256), 0, s, a, (int)chunks, (int)lens_groups);
    }
    return (int)hipGetLastError();
}

}  // namespace rq
