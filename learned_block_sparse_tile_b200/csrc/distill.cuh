// Distillation of tile scores from a teacher's top logits, loss and gradient in one pass.
//
// For a row of student scores s over n columns and the teacher's listed logits t:
//     p = softmax(t / tau) over the row's list,   q = softmax(s / tau) over all columns,
//     L = sum_list p (log p - log q),   loss = w L,   d loss / d s_j = (w / tau) (q_j - p_j).
// With ms, mt the maxima of s / tau and t / tau, Zs and Zt the sums of exp(. - max):
//     L = sum_list p ((t / tau - mt) - (s / tau - ms)) - log Zt + log Zs,
// differences of numbers near zero, where log p - log q would cancel two long logarithms.
//
// The floor is one read of the scores and one write of their gradient (8 n bytes a row), so a row stays in registers
// between them: up to 32 columns a thread, one warp for a row of up to 1024 columns and 2 to 16 warps beyond. Its
// exponentials are taken once (2^x of (s - max) log2(e) / tau), serve both the sum and the gradient, and only the
// listed columns, a tenth of the row or less, are visited again: they are written as q, and after a barrier as q - p.
// What bounds it beside the bytes is the chain of latencies of a row (count, list, listed scores, two rounds of
// reductions), so the count, the first kListed entries of the list and the row are loaded together, entries behind the
// count among them, which nothing uses; longer lists read the rest again where they need it.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ptx.cuh"
#include "warp.cuh"

namespace veda {

constexpr int kErrDistillList = 2;  // the latched bit of a malformed list, as the attend's
constexpr int kListed = 4;          // list entries a thread keeps in registers

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

// One value for the row's kWarps warps, from one per warp. `scratch` holds kWarps floats, free again for the next reduction
// but one.
template <int kWarps, class Op>
__device__ __forceinline__ float across_warps(float v, float* scratch, Op op) {
    if constexpr (kWarps > 1) {
        if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
        __syncthreads();
        v = scratch[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v = op(v, scratch[w]);
    }
    return v;
}
template <int kWarps>
__device__ __forceinline__ float row_max(float v, float* scratch) {
    return across_warps<kWarps>(warp_max(v), scratch, [](float x, float y) { return fmaxf(x, y); });
}
template <int kWarps>
__device__ __forceinline__ float row_sum(float v, float* scratch) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return across_warps<kWarps>(v, scratch, [](float x, float y) { return x + y; });
}

// Rows of up to 32 * kPer * kWarps columns. One warp per row: four rows in a CTA; else one row in a CTA. The registers are
// held to 72 a thread, 28 warps an SM: 220k rows, 24 heads take 111 us with 28 warps, 132 with 20 and 165 with 32 (spills);
// 121 in repeated calls from the host.
template <int kPer, int kWarps>
__global__ void __launch_bounds__(kWarps == 1 ? 128 : 32 * kWarps, kWarps == 1 ? 7 : kWarps == 2 ? 14 : 1) distill_kernel(const DistillArgs a) {
    constexpr int kLanes = 32 * kWarps;
    __shared__ float scratch[2][kWarps];
    __shared__ int s_cnt;
    const int64_t r = kWarps == 1 ? int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5) : int64_t(blockIdx.x);
    if (kWarps == 1 && r >= a.rows) return;
    const int lane = kWarps == 1 ? threadIdx.x & 31 : threadIdx.x;
    const float* s = a.scores + r * a.n;
    const int32_t* idx = a.t_idx + r * a.width;
    const float* val = a.t_val + r * (a.by_column ? a.n : a.width);

    const int given = a.t_cnt[r];
    float v[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int j = lane + kLanes * k;
        v[k] = j < a.n ? __ldg(s + j) : -INFINITY;
    }
    int id[kListed], before[kListed];
    float t[kListed], x[kListed];
#pragma unroll
    for (int u = 0; u < kListed; ++u) {
        const int e = lane + kLanes * u;
        id[u] = e < a.width ? __ldg(idx + e) : -1;
        before[u] = e < a.width && e > 0 ? __ldg(idx + e - 1) : -1;
        t[u] = e < a.width && !a.by_column ? __ldg(val + e) : 0.f;
    }
    // the list: its entries are ascending tile ids; it is cut at the first bad one, and ids from n on (global tiles,
    // which no score column stands for) end the part that counts
    bool bad = given < 0 || given > a.width;
    int cnt = max(0, min(given, a.width));
    {
        int end = cnt;
        const auto check = [&](int e, int mine, int previous) {
            const bool wrong = mine < 0 || mine >= a.n_tiles || mine <= previous;
            bad |= wrong;
            if (wrong || mine >= a.n) end = min(end, e);
        };
#pragma unroll
        for (int u = 0; u < kListed; ++u)
            if (lane + kLanes * u < end) check(lane + kLanes * u, id[u], before[u]);
        for (int e = lane + kLanes * kListed; e < end; e += kLanes) check(e, idx[e], idx[e - 1]);
        if constexpr (kWarps == 1) {
            cnt = __reduce_min_sync(0xffffffffu, end);
        } else {
            if (threadIdx.x == 0) s_cnt = cnt;
            __syncthreads();
            if (end < cnt) atomicMin(&s_cnt, end);
            __syncthreads();
            cnt = s_cnt;
        }
        if (bad) atomicOr(a.err, kErrDistillList);
    }
    float mt = -INFINITY;
#pragma unroll
    for (int u = 0; u < kListed; ++u) {
        const bool on = lane + kLanes * u < cnt;
        x[u] = on ? __ldg(s + id[u]) : 0.f;
        if (a.by_column && on) t[u] = __ldg(val + id[u]);
        if (!on) t[u] = -INFINITY;
        mt = fmaxf(mt, t[u]);
    }
    for (int e = lane + kLanes * kListed; e < cnt; e += kLanes) mt = fmaxf(mt, val[a.by_column ? idx[e] : e]);
    float ms = -INFINITY;
#pragma unroll
    for (int k = 0; k < kPer; ++k) ms = fmaxf(ms, v[k]);
    ms = row_max<kWarps>(ms, scratch[0]);
    mt = row_max<kWarps>(mt, scratch[1]);

    const float c2 = a.inv_tau * 1.4426950408889634f;
    float zs = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        // (a column of -inf, or one past the row, has no mass, whatever the maximum is)
        v[k] = v[k] == -INFINITY ? 0.f : ptx::ex2((v[k] - ms) * c2);
        zs += v[k];
    }
    float zt = 0.f, gap = 0.f;
    // a listed logit becomes its exponential; -inf has no mass
    const auto entry = [&](float logit, float score) {
        if (logit == -INFINITY) return 0.f;
        const float p = ptx::ex2((logit - mt) * c2);
        zt += p;
        if (!(p == 0.f)) gap += p * (((logit - mt) - (score - ms)) * a.inv_tau);
        return p;
    };
#pragma unroll
    for (int u = 0; u < kListed; ++u) t[u] = entry(t[u], x[u]);
    for (int e = lane + kLanes * kListed; e < cnt; e += kLanes) entry(val[a.by_column ? idx[e] : e], __ldg(s + idx[e]));
    zs = row_sum<kWarps>(zs, scratch[0]);
    zt = row_sum<kWarps>(zt, scratch[1]);
    if constexpr (kWarps > 1) __syncthreads();
    gap = row_sum<kWarps>(gap, scratch[0]);
    // no target (an empty list, or only -inf in it) or no student column above -inf: the row is left out
    const bool out = zt == 0.f || zs == 0.f;
    const float w = a.row_weight ? a.row_weight[r] : 1.f;
    if (lane == 0) a.loss[r] = out ? 0.f : w * (gap / zt - logf(zt) + logf(zs));
    if (!a.d_scores) return;
    float* d = a.d_scores + r * a.n;
    const float c = w * a.inv_tau, iz = 1.f / zs;
    if (out) {  // zeros, whatever the row's scores are (a product with zero would keep a NaN)
        for (int j = lane; j < a.n; j += kLanes) d[j] = 0.f;
        return;
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int j = lane + kLanes * k;
        if (j < a.n) d[j] = c * (v[k] * iz);
    }
    if constexpr (kWarps == 1) __syncwarp();
    else __syncthreads();
    const float izt = 1.f / zt;
    const auto mass = [&](float score) { return score == -INFINITY ? 0.f : ptx::ex2((score - ms) * c2) * iz; };
#pragma unroll
    for (int u = 0; u < kListed; ++u)
        if (lane + kLanes * u < cnt) d[id[u]] = c * (mass(x[u]) - t[u] * izt);
    for (int e = lane + kLanes * kListed; e < cnt; e += kLanes) {
        const float logit = val[a.by_column ? idx[e] : e];
        d[idx[e]] = c * (mass(__ldg(s + idx[e])) - (logit == -INFINITY ? 0.f : ptx::ex2((logit - mt) * c2) * izt));
    }
}

}  // namespace veda
