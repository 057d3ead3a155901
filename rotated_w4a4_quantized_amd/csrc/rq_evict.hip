// rq_evict.hip -- eviction from a cache by accumulated attention weight.
//
// Per (sequence, head) row of n slots: the keep first in the order (protected,
// weight descending, slot ascending) stay.  Survivors above `keep` move into
// the free slots below it, so a move never reads what another one writes.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rq_attn_util.h"
#include "rq_internal.h"

namespace rq {
namespace {

using attn::Cache;

struct Args {
    Cache c;
    const int32_t *lens;
    int32_t *lens_out, *pos_out;
    float *weight_out;
    int32_t *count;      // [rows] moves of a row
    int32_t *moves;      // [rows][2][most] free slots, then survivors
    int64_t slots;
    int32_t max_len, keep, recent, sink, most;
};

// Order-preserving map of a weight to unsigned: NaN lowest, protected highest.
__device__ __forceinline__ uint32_t key_of(float w, bool held) {
    if (held) return 0xffffffffu;
    if (w != w) return 0u;
    const uint32_t b = __builtin_bit_cast(uint32_t, w);
    // (-0 and +0 are one weight)
    return b == 0x80000000u ? 0x80000000u : b & 0x80000000u ? ~b : b | 0x80000000u;
}

constexpr int kThreads = 1024;

__device__ int block_sum(int v, int *part) {
    for (int o = 1; o < 64; o *= 2) v += __shfl_xor(v, o);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    int s = 0;
    for (int i = 0; i < kThreads / 64; ++i) s += part[i];
    __syncthreads();
    return s;
}
// exclusive prefix over the threads
__device__ int block_scan(int v, int *part, int &total) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int x = v;
    for (int o = 1; o < 64; o *= 2) {
        const int y = __shfl_up(x, o);
        if (lane >= o) x += y;
    }
    if (lane == 63) part[w] = x;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int i = 0; i < kThreads / 64; ++i) {
        if (i < w) before += part[i];
        total += part[i];
    }
    __syncthreads();
    return before + x - v;
}

__global__ void __launch_bounds__(kThreads) select_kernel(Args a) {
    __shared__ int part[kThreads / 64];
    const int row = blockIdx.x, b = row / a.c.heads, t = threadIdx.x;
    const int n = min(max(a.lens[b], 0), a.max_len);
    const float *w = a.c.weight + row * a.slots;
    const int32_t *pos = a.c.pos + row * a.slots;
    float *wo = a.weight_out + row * a.slots;
    int32_t *po = a.pos_out + row * a.slots;
    if (n <= a.keep) {
        for (int j = t; j < n; j += kThreads) {
            wo[j] = w[j];
            po[j] = pos[j];
        }
        if (t == 0) a.count[row] = 0;
        return;
    }
    int newest = -1;
    for (int j = t; j < n; j += kThreads) newest = max(newest, pos[j]);
    for (int o = 1; o < 64; o *= 2) newest = max(newest, __shfl_xor(newest, o));
    if ((t & 63) == 0) part[t >> 6] = newest;
    __syncthreads();
    for (int i = 0; i < kThreads / 64; ++i) newest = max(newest, part[i]);
    __syncthreads();
    const int from = newest - a.recent;
    auto key = [&](int j) { return key_of(w[j], pos[j] < a.sink || pos[j] > from); };
    // the largest key that at least `keep` keys reach
    uint32_t thr = 0;
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t c = thr | (1u << bit);
        int mine = 0;
        for (int j = t; j < n; j += kThreads) mine += key(j) >= c;
        if (block_sum(mine, part) >= a.keep) thr = c;
    }
    int above = 0;
    for (int j = t; j < n; j += kThreads) above += key(j) > thr;
    int ties = a.keep - block_sum(above, part);   // of the keys at the threshold, the lowest slots
    // (weights and positions of the places below keep are written by the move: they may be the inputs)
    int free_at = 0, up_at = 0;
    int32_t *free_list = a.moves + (int64_t)row * 2 * a.most, *up_list = free_list + a.most;
    for (int base = 0; base < n; base += kThreads) {
        const int j = base + t;
        const uint32_t k = j < n ? key(j) : 0;
        int total;
        const int tied = j < n && k == thr;
        const int rank = block_scan(tied, part, total);
        const bool kept = j < n && (k > thr || (tied && rank < ties));
        ties -= min(total, ties);
        const int is_free = j < a.keep && !kept, is_up = j >= a.keep && j < n && kept;
        const int f = block_scan(is_free, part, total) + free_at;
        free_at += total;
        const int u = block_scan(is_up, part, total) + up_at;
        up_at += total;
        if (is_free) free_list[f] = j;
        if (is_up) up_list[u] = j;
    }
    if (t == 0) a.count[row] = up_at;
    __threadfence_block();
    __syncthreads();
    if (wo != w || po != pos)
        for (int j = t; j < a.keep; j += kThreads) {
            wo[j] = w[j];
            po[j] = pos[j];
        }
    __threadfence_block();
    __syncthreads();
    for (int i = t; i < up_at; i += kThreads) {
        wo[free_list[i]] = w[up_list[i]];
        po[free_list[i]] = pos[up_list[i]];
    }
}

// Keys and values of one row's moves: a wave per move.
__global__ void __launch_bounds__(256) move_kernel(Args a, int bytes) {
    const int row = blockIdx.y, b = row / a.c.heads, h = row % a.c.heads, lane = threadIdx.x & 63;
    const int count = a.count[row];
    const int32_t *free_list = a.moves + (int64_t)row * 2 * a.most, *up_list = free_list + a.most;
    for (int i = blockIdx.x * 4 + (threadIdx.x >> 6); i < count; i += gridDim.x * 4) {
        const int64_t to = a.c.row(b, h, free_list[i]), from = a.c.row(b, h, up_list[i]);
        if (to < 0 || from < 0) continue;
        for (int d = lane * 8; d < a.c.D * bytes; d += 512) {
            *reinterpret_cast<uint2 *>(static_cast<char *>(a.c.k) + to * a.c.D * bytes + d) =
                *reinterpret_cast<const uint2 *>(static_cast<const char *>(a.c.k) + from * a.c.D * bytes + d);
            *reinterpret_cast<uint2 *>(static_cast<char *>(a.c.v) + to * a.c.D * bytes + d) =
                *reinterpret_cast<const uint2 *>(static_cast<const char *>(a.c.v) + from * a.c.D * bytes + d);
        }
        if (bytes == 1 && lane == 0) {
            a.c.k_scale[to] = a.c.k_scale[from];
            a.c.v_scale[to] = a.c.v_scale[from];
        }
    }
}

// Last: nothing reads lens after it, so lens_out may be lens.
__global__ void __launch_bounds__(256) lens_kernel(Args a) {
    const int b = blockIdx.x * 256 + threadIdx.x;
    if (b < a.c.batch) a.lens_out[b] = min(min(max(a.lens[b], 0), a.max_len), a.keep);
}

int most_moves(int keep, int64_t max_len) {
    return (int)std::max<int64_t>(0, std::min<int64_t>(keep, max_len - keep));
}

}  // namespace

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
    hipStream_t s = static_cast<hipStream_t>(stream);
    hipLaunchKernelGGL(select_kernel, dim3(rows), dim3(kThreads), 0, s, a);
    if (a.most > 0)
        hipLaunchKernelGGL(move_kernel, dim3((unsigned)std::min((a.most + 3) / 4, 256), rows), dim3(256), 0, s, a,
                           c->dtype == RQ_I8 ? 1 : 2);
    hipLaunchKernelGGL(lens_kernel, dim3((c->batch + 255) / 256), dim3(256), 0, s, a);
    return (int)hipGetLastError();
}

}  // namespace rq
