// Distillation of tile scores from a teacher's top logits, loss and gradient in one pass.
//
// For a row of student scores s over n columns and the teacher's listed logits t:
//     p = softmax(t / tau) over the row's list,   q = softmax(s / tau) over all columns,
//     L = sum_list p (log p - log q),   loss = w L,   d loss / d s_j = (w / tau) (q_j - p_j).
// With ms, mt the maxima of s / tau and t / tau, Zs and Zt the sums of exp(. - max):
//     L = sum_list p ((t / tau - mt) - (s / tau - ms)) - log Zt + log Zs,
// differences of numbers near zero, where log p - log q would cancel two long logarithms.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

namespace veda {

constexpr int kErrDistillList = 2;  // the latched bit of a malformed list, as the attend's

struct DistillArgs {
    const float* scores;      // [n_heads * n, n]
    const int32_t* t_idx;     // [n_heads * n, width]
    const float* t_val;       // [n_heads * n, width], or [n_heads * n, n] with by_column
    const int32_t* t_cnt;     // [n_heads * n]
    const float* row_weight;  // [n_heads * n] or null (1)
    float* loss;              // [n_heads * n]
    float* d_scores;          // [n_heads * n, n] or null
    int64_t rows;
    int n, width, n_tiles, by_column;
    float inv_tau;
    int* err;
};

template <class Op>
__device__ __forceinline__ float block_reduce_128(float v, float* scratch, Op op) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    return op(op(scratch[0], scratch[1]), op(scratch[2], scratch[3]));
}

// One CTA per row.
__global__ void __launch_bounds__(128) distill_kernel(const DistillArgs a) {
    __shared__ float scratch[4];
    __shared__ int s_cnt;
    const int64_t r = blockIdx.x;
    const float* s = a.scores + r * a.n;
    const int32_t* idx = a.t_idx + r * a.width;
    const float* val = a.t_val + r * (a.by_column ? a.n : a.width);
    const auto maxf = [](float x, float y) { return fmaxf(x, y); };
    const auto add = [](float x, float y) { return x + y; };
    // the list: its entries are ascending tile ids; it is cut at the first bad one, and ids from n on
    // (global tiles, which no score column stands for) end the part that counts
    if (threadIdx.x == 0) s_cnt = max(0, min(a.t_cnt[r], a.width));
    __syncthreads();
    const int given = s_cnt;
    bool bad = a.t_cnt[r] < 0 || a.t_cnt[r] > a.width;
    __syncthreads();
    for (int e = threadIdx.x; e < given; e += 128) {
        const int id = idx[e];
        const bool wrong = id < 0 || id >= a.n_tiles || (e > 0 && id <= idx[e - 1]);
        if (wrong) bad = true;
        if (wrong || id >= a.n) atomicMin(&s_cnt, e);
    }
    if (bad) atomicOr(a.err, kErrDistillList);
    __syncthreads();
    const int cnt = s_cnt;

    float ms = -INFINITY;
    for (int j = threadIdx.x; j < a.n; j += 128) ms = fmaxf(ms, s[j] * a.inv_tau);
    ms = block_reduce_128(ms, scratch, maxf);
    float mt = -INFINITY;
    for (int e = threadIdx.x; e < cnt; e += 128) mt = fmaxf(mt, val[a.by_column ? idx[e] : e] * a.inv_tau);
    mt = block_reduce_128(mt, scratch, maxf);
    float zs = 0.f, zt = 0.f, gap = 0.f;
    for (int j = threadIdx.x; j < a.n; j += 128) {
        const float x = s[j] * a.inv_tau;
        zs += x == -INFINITY ? 0.f : expf(x - ms);
    }
    zs = block_reduce_128(zs, scratch, add);
    for (int e = threadIdx.x; e < cnt; e += 128) {
        const float t = val[a.by_column ? idx[e] : e] * a.inv_tau;
        if (t == -INFINITY) continue;
        const float p = expf(t - mt);
        zt += p;
        if (p > 0.f) gap += p * ((t - mt) - (s[idx[e]] * a.inv_tau - ms));
    }
    zt = block_reduce_128(zt, scratch, add);
    gap = block_reduce_128(gap, scratch, add);
    // no target (an empty list, or only -inf in it) or no student column above -inf: the row is left out
    const bool out = zt == 0.f || zs == 0.f;
    const float w = a.row_weight ? a.row_weight[r] : 1.f;
    if (threadIdx.x == 0) a.loss[r] = out ? 0.f : w * (gap / zt - logf(zt) + logf(zs));
    if (!a.d_scores) return;
    float* d = a.d_scores + r * a.n;
    const float c = w * a.inv_tau, iz = 1.f / zs, izt = 1.f / zt;
    for (int j = threadIdx.x; j < a.n; j += 128) d[j] = out ? 0.f : c * (expf(s[j] * a.inv_tau - ms) * iz);
    __syncthreads();
    if (out) return;
    for (int e = threadIdx.x; e < cnt; e += 128) {
        const float t = val[a.by_column ? idx[e] : e] * a.inv_tau;
        const float q = expf(s[idx[e]] * a.inv_tau - ms) * iz;
        d[idx[e]] = c * (q - (t == -INFINITY ? 0.f : expf(t - mt) * izt));
    }
}

}  // namespace veda
