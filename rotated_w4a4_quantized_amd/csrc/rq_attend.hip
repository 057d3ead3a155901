// rq_attend.hip -- attention of one new token per sequence over a paged cache.
//
//   s_j = scale q . k_j;  lse = log sum exp s_j;  out = sum exp(s_j - lse) v_j

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "rq_attn_util.h"
#include "rq_internal.h"

namespace rq {
namespace {

using attn::Cache;

struct Args {
    Cache c;
    const void *q;
    void *out;
    const int32_t *lens;
    const uint8_t *mask;
    float *lse, *weight_out, *scores;
    int64_t q_ld, out_ld, mask_ld;
    int32_t hq, max_len;
    float scale;
};

template <bool I8>
__device__ __forceinline__ float cache1(const void *p, int64_t i) {
    if constexpr (I8) return (float)static_cast<const int8_t *>(p)[i];
    else return attn::bf16_f32(static_cast<const uint16_t *>(p)[i]);
}

// Scores of one (sequence, query head): a wave per slot, lanes along d.
template <bool BF16, bool I8>
__global__ void __launch_bounds__(256) scores_kernel(Args a) {
    const int b = blockIdx.y, i = blockIdx.z, lane = threadIdx.x & 63, h = i / (a.hq / a.c.heads);
    const int len = min(max(a.lens[b], 0), a.max_len);
    const int64_t slots = a.max_len;
    for (int j = blockIdx.x * 4 + (threadIdx.x >> 6); j < len; j += gridDim.x * 4) {
        const int64_t row = a.mask && !a.mask[b * a.mask_ld + j] ? -1 : a.c.row(b, h, j);
        float s = 0.0f;
        if (row >= 0)
            for (int d = lane; d < a.c.D; d += 64)
                s += attn::load1<BF16>(a.q, b * a.q_ld + (int64_t)i * a.c.D + d) * cache1<I8>(a.c.k, row * a.c.D + d);
        for (int o = 1; o < 64; o *= 2) s += __shfl_xor(s, o);
        s *= a.scale;
        if (row >= 0 && I8) s *= a.c.k_scale[row];
        if (lane == 0) a.scores[((int64_t)b * a.hq + i) * slots + j] = row >= 0 ? s : -INFINITY;
    }
}

// Softmax and output of one (sequence, query head) by one workgroup.
template <bool BF16, bool I8>
__global__ void __launch_bounds__(256) output_kernel(Args a) {
    __shared__ float part[256];
    const int b = blockIdx.x, i = blockIdx.y, t = threadIdx.x, h = i / (a.hq / a.c.heads);
    const int len = min(max(a.lens[b], 0), a.max_len);
    const int64_t slots = a.max_len;
    float *s = a.scores + ((int64_t)b * a.hq + i) * slots;
    auto reduce = [&](float v, bool is_max) {
        part[t] = v;
        __syncthreads();
        for (int o = 128; o > 0; o /= 2) {
            if (t < o) part[t] = is_max ? fmaxf(part[t], part[t + o]) : part[t] + part[t + o];
            __syncthreads();
        }
        v = part[0];
        __syncthreads();
        return v;
    };
    float m = -INFINITY, l = 0.0f;
    for (int j = t; j < len; j += 256) m = fmaxf(m, s[j]);
    m = reduce(m, true);
    for (int j = t; j < len; j += 256)
        if (s[j] != -INFINITY) l += expf(s[j] - m);
    l = reduce(l, false);
    for (int j = t; j < len; j += 256) s[j] = s[j] != -INFINITY ? expf(s[j] - m) / l : 0.0f;
    __threadfence_block();
    __syncthreads();
    if (t < a.c.D) {
        float o = 0.0f;
        for (int j = 0; j < len; ++j) {
            const int64_t row = a.mask && !a.mask[b * a.mask_ld + j] ? -1 : a.c.row(b, h, j);
            if (row < 0) continue;
            float v = cache1<I8>(a.c.v, row * a.c.D + t);
            if (I8) v *= a.c.v_scale[row];
            o += s[j] * v;
        }
        attn::store1<BF16>(a.out, b * a.out_ld + (int64_t)i * a.c.D + t, o);
    }
    if (t == 0 && a.lse) a.lse[(int64_t)b * a.hq + i] = m + logf(l);
}

__global__ void __launch_bounds__(256) weights_kernel(Args a) {
    const int b = blockIdx.y, h = blockIdx.z, G = a.hq / a.c.heads;
    const int len = min(max(a.lens[b], 0), a.max_len);
    const int j = blockIdx.x * 256 + threadIdx.x;
    if (j >= len) return;
    const int64_t at = ((int64_t)b * a.c.heads + h) * a.c.slots() + j;
    float w = 0.0f;
    for (int g = 0; g < G; ++g) w += a.scores[((int64_t)b * a.hq + h * G + g) * a.max_len + j];
    a.weight_out[at] = a.c.weight[at] + w;
}

}  // namespace

size_t attend_workspace_bytes(const rq_kv_cache *c, int q_heads, int64_t max_len, int track) {
    return (size_t)c->batch * q_heads * max_len * 4;
}

int launch_paged_attention(const rq_kv_cache *c, const void *q, int bf16, int64_t q_ld, int q_heads,
                           float scale, const int32_t *lens, int64_t max_len, const uint8_t *mask,
                           int64_t mask_ld, void *out, int64_t out_ld, float *lse, int track,
                           float *weight_out, void *workspace, void *stream) {
    Args a{};
    a.c = device_cache(c);
    a.q = q, a.out = out, a.lens = lens, a.mask = mask, a.lse = lse, a.weight_out = weight_out;
    a.scores = static_cast<float *>(workspace);
    a.q_ld = q_ld, a.out_ld = out_ld, a.mask_ld = mask_ld, a.hq = q_heads, a.max_len = (int)max_len;
    a.scale = scale;
    hipStream_t s = static_cast<hipStream_t>(stream);
    const unsigned B = c->batch, H = q_heads;
    auto go = [&](auto k1, auto k2) {
        if (max_len > 0)
            hipLaunchKernelGGL(k1, dim3((unsigned)std::min<int64_t>((max_len + 3) / 4, 1024), B, H), dim3(256), 0, s, a);
        hipLaunchKernelGGL(k2, dim3(B, H), dim3(256), 0, s, a);
    };
    const bool i8 = c->dtype == RQ_I8;
    if (bf16) {
        if (i8) go(scores_kernel<true, true>, output_kernel<true, true>);
        else go(scores_kernel<true, false>, output_kernel<true, false>);
    } else {
        if (i8) go(scores_kernel<false, true>, output_kernel<false, true>);
        else go(scores_kernel<false, false>, output_kernel<false, false>);
    }
    if (track && max_len > 0)
        hipLaunchKernelGGL(weights_kernel, dim3((unsigned)((max_len + 255) / 256), B, c->heads), dim3(256), 0, s, a);
    return (int)hipGetLastError();
}

}  // namespace rq
