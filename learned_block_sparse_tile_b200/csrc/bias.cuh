// Learned relative position bias of the tile scores, by buckets of the two tiles' offset.
//
// A video tile has a place (t, h, w) in its span's array of tiles. Two tiles of one span have the offset
// r = key place - query place, and per axis the distance |r| falls into one of `reach` classes: the first
// e = (reach + 1) / 2 hold one distance each, the others widen geometrically up to `far` tiles (class
// e + m starts at the smallest a with a^k >= e^(k - m) far^m, k = reach - e; whole numbers, so nothing
// rounds at a border). With the sign of r an axis has 2 reach - 1 indices, and the pair's bucket is the
// three axes' mixed-radix number. Pairs of tiles of different spans share two more buckets: the key's
// span before, and behind, the query's.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

namespace veda {

constexpr int kBiasMaxReach = 16;
constexpr int kBiasMaxBuckets = 4096;
constexpr float kBiasLargest = 0x1p120f;  // finite biases are taken no larger than this

// starts[a][c] = the smallest distance of class c (c >= 1) on axis a
struct BiasClasses {
    int reach[3];
    int starts[3][kBiasMaxReach];
    int buckets;  // all of them, the two of other spans last
};

// index of a signed offset on one axis: 0 .. 2 reach - 2
__host__ __device__ __forceinline__ int bias_axis_index(const int* starts, int reach, int r) {
    const int a = r < 0 ? -r : r;
    int c = 0;
    for (int k = 1; k < reach; ++k) c += a >= starts[k];
    return r > 0 ? reach - 1 + c : c;
}

__host__ __device__ __forceinline__ int bias_bucket(const BiasClasses& b, int dt, int dh, int dw) {
    const int it = bias_axis_index(b.starts[0], b.reach[0], dt);
    const int ih = bias_axis_index(b.starts[1], b.reach[1], dh);
    const int iw = bias_axis_index(b.starts[2], b.reach[2], dw);
    return (it * (2 * b.reach[1] - 1) + ih) * (2 * b.reach[2] - 1) + iw;
}

// Offsets as one number. In a span of T x H x W tiles a place's number is (h (2W - 1) + w) (2T - 1) + t, and an
// offset's number is the difference of two places' numbers, so the bias of a pair is one load of a table per
// head that holds the bias of every offset: the spans' offsets one span after the other ((2T - 1)(2H - 1)(2W - 1)
// each, fewer than 8 per tile), then the two buckets of other spans. The layout keeps each tile's part of the
// index as a key (its number) and as a query (where the table's part of its span is centred, less its number). Tiles are
// in (h, w, t) order, t fastest, and so are the numbers: neighbouring keys read neighbouring entries.

// The table, written by otherwise idle warps of the launch that computes the projected features (train_gemm.cuh):
// table[head][o] = factor bias[head][bucket(o)]; the sums that start from it are scaled by 1 / factor at their end.
struct BiasExpand {
    const float* bias;  // [heads, buckets], or null: no table
    float* table;       // [heads, count + 2]
    float factor;
    const int4* span_grid;
    int n_spans, count, heads;
    BiasClasses b;
};

// entry i of every head's table
__device__ __forceinline__ void bias_expand(const BiasExpand& x, int i) {
    int bucket = x.b.buckets - 2 + (i - x.count);
    if (i < x.count) {
        int o = i;
        int4 g = x.span_grid[0];
        for (int s = 0; s < x.n_spans; ++s) {
            g = x.span_grid[s];
            const int offsets = (2 * g.y - 1) * (2 * g.z - 1) * (2 * g.w - 1);
            if (o < offsets) break;
            o -= offsets;
        }
        const int rt = 2 * g.y - 1, rw = 2 * g.w - 1;
        bucket = bias_bucket(x.b, o % rt - (g.y - 1), o / (rt * rw) - (g.z - 1), (o / rt) % rw - (g.w - 1));
    }
    for (int h = 0; h < x.heads; ++h) {
        float v = x.bias[int64_t(h) * x.b.buckets + bucket];
        // a mask of the type's lowest value stays finite under the factor
        if (fabsf(v) > kBiasLargest && fabsf(v) < INFINITY) v = copysignf(kBiasLargest, v);
        x.table[int64_t(h) * (x.count + 2) + i] = x.factor * v;
    }
}

struct BiasBackwardArgs {
    const float* d_scores;     // [n_heads, n, n]
    const int4* tile_pos;      // [n] {span, t, h, w}
    const int4* tile_num;      // [n] {span, number as key, number as query, 0}
    const int4* span_grid;     // [n_spans] {first tile, tiles along t, h, w}
    float* partial;            // [n_heads, chunks, buckets]
    int n, n_spans, offsets, rows_per_chunk;
    BiasClasses b;
};

// places [lo, hi) of an axis of `count` places whose offset from `at` has index `idx`
__device__ __forceinline__ void bias_interval(const int* starts, int reach, int idx, int at, int count, int& lo, int& hi) {
    if (reach == 1) {
        lo = 0;
        hi = count;
        return;
    }
    const int c = idx < reach ? idx : idx - reach + 1;
    const int a0 = c == 0 ? 0 : starts[c], a1 = c + 1 < reach ? starts[c + 1] - 1 : 1 << 28;
    if (idx < reach && c > 0) {  // r = -a1 .. -a0
        lo = at - a1;
        hi = at - a0 + 1;
    } else if (idx < reach) {    // r = 0
        lo = at - a1;
        hi = at + 1;
    } else {                     // r = a0 .. a1
        lo = at + a0;
        hi = at + a1 + 1;
    }
    lo = max(lo, 0);
    hi = min(hi, count);
}

// Sums of one chunk of query rows, by offset first. Within a row no two keys of the query's span have the same offset, so
// a row adds to as many different sums as it has columns: the CTA keeps one sum per offset in shared memory (fewer than 8
// per tile), its threads add a row's columns without collisions, and a barrier parts the rows. Nothing is atomic, and
// every sum is added up in row order. The loads run kDepth rows ahead in registers, because the rows' own work is short:
// an addition in shared memory and a barrier; a warp waits for its newer loads with its older ones, so they cover the
// latency of L2 and not of memory, and one thread asks for the chunk's next rows, a run of memory, in L2 further ahead
// (104k rows, 24 heads, from HBM: 44 -> 32 us). At the end each bucket is the sum of a box of offsets, taken axis by axis:
// a box may hold nearly all offsets, and one chain of them would lose what a few long ones do not. Bound by the chain
// of shared-memory addition and barrier, with up to three CTAs on an SM taking turns (104k, 24 heads: 28 us from HBM, 23
// from L2, 31 in repeated calls from the host; two CTAs: 32 and 24; two sets of sums and a barrier for each two rows gain
// nothing: 29 and 23); the floor is reading d_scores once. With two values a thread the registers are held to three CTAs of
// any size (960 tiles, 24 heads: 36 us, two CTAs 40; 868 tiles 32, and 49 where the third waits for the others' end).
template <int kPer, bool kOneSpan>
__global__ void __launch_bounds__(512, kPer == 2 ? 3 : kPer <= 4 ? 2 : 1) bias_backward_kernel(const BiasBackwardArgs a) {
    constexpr int kDepth = kPer <= 2 ? 8 : kPer <= 4 ? 4 : 2;
    constexpr int kAhead = kDepth;  // rows asked for in L2 ahead of the loads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    extern __shared__ float sums[];  // [offsets], 2 x 16 cross-span sums of the warps, then the rows' queries
    const int head = blockIdx.y, pairs = a.b.buckets - 2, nt = blockDim.x;
    const int i0 = blockIdx.x * a.rows_per_chunk, i1 = min(a.n, i0 + a.rows_per_chunk);
    int2* query = reinterpret_cast<int2*>(sums + (a.offsets + 32 + 1) / 2 * 2);      // {span, number}
    const float* next = a.d_scores + (int64_t(head) * a.n + i0) * a.n + threadIdx.x;  // of the next row to load
    // rows [i, i + count) of the chunk into L2, in whole 16-byte parts
    const auto prefetch = [&](int i, int count) {
        const int rows = min(count, i1 - i);
        if (threadIdx.x != 0 || rows <= 0) return;
        const float* p = a.d_scores + (int64_t(head) * a.n + i) * a.n;
        const uintptr_t begin = (reinterpret_cast<uintptr_t>(p) + 15) & ~uintptr_t(15);
        const uintptr_t end = reinterpret_cast<uintptr_t>(p + int64_t(rows) * a.n) & ~uintptr_t(15);
        if (end > begin)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(begin), "r"(uint32_t(end - begin)) : "memory");
    };
    prefetch(i0 + kDepth, kAhead);
    float v[kDepth][kPer];
    int span[kPer], num[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int j = threadIdx.x + nt * k;
        const int4 key = a.tile_num[min(j, a.n - 1)];
        span[k] = j < a.n ? key.x : -1;
        num[k] = key.y;
    }
    const auto load = [&](float (&x)[kPer]) {
#pragma unroll
        for (int k = 0; k < kPer; ++k) x[k] = span[k] >= 0 ? __ldg(next + nt * k) : 0.f;
        next += a.n;
    };
#pragma unroll
    for (int r = 0; r < kDepth; ++r)
        if (i0 + r < i1) load(v[r]);
    for (int i = i0 + threadIdx.x; i < i1; i += nt) {
        const int4 q = a.tile_num[i];
        query[i - i0] = make_int2(q.x, q.z);
    }
    for (int o = threadIdx.x; o < a.offsets; o += nt) sums[o] = 0.f;
    __syncthreads();
    float before = 0.f, behind = 0.f;
    for (int i = i0; i < i1; i += kDepth) {
        prefetch(i + kDepth + kAhead, kDepth);
#pragma unroll
        for (int r = 0; r < kDepth; ++r) {
            if (i + r < i1) {
                const int2 q = query[i - i0 + r];
                float* at = sums + q.y;
#pragma unroll
                for (int k = 0; k < kPer; ++k) {
                    if (kOneSpan ? span[k] >= 0 : span[k] == q.x) {
                        at[num[k]] += v[r][k];
                    } else if (!kOneSpan) {  // (threads past the row hold zeros)
                        before += span[k] < q.x ? v[r][k] : 0.f;
                        behind += span[k] > q.x ? v[r][k] : 0.f;
                    }
                }
                if (i + r + kDepth < i1) load(v[r]);
            }
            __syncthreads();
        }
    }
    float* cross = sums + a.offsets;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        behind += __shfl_xor_sync(0xffffffffu, behind, o);
    }
    if ((threadIdx.x & 31) == 0) {
        cross[threadIdx.x >> 5] = before;
        cross[16 + (threadIdx.x >> 5)] = behind;
    }
    __syncthreads();
    float* out = a.partial + (int64_t(head) * gridDim.x + blockIdx.x) * a.b.buckets;
    const int ih = 2 * a.b.reach[1] - 1, iw = 2 * a.b.reach[2] - 1;
    for (int b = threadIdx.x; b < a.b.buckets; b += nt) {
        float sum = 0.f;
        if (b >= pairs) {
            for (int w = 0; w < nt / 32; ++w) sum += cross[16 * (b - pairs) + w];
        } else {
            const float* at = sums;
            for (int s = 0; s < a.n_spans; ++s) {
                const int4 g = a.span_grid[s];
                const int rt = 2 * g.y - 1, rh = 2 * g.z - 1, rw = 2 * g.w - 1;
                int t0, t1, h0, h1, w0, w1;
                bias_interval(a.b.starts[0], a.b.reach[0], b / (iw * ih), g.y - 1, rt, t0, t1);
                bias_interval(a.b.starts[1], a.b.reach[1], (b / iw) % ih, g.z - 1, rh, h0, h1);
                bias_interval(a.b.starts[2], a.b.reach[2], b % iw, g.w - 1, rw, w0, w1);
                for (int h = h0; h < h1; ++h) {
                    float plane = 0.f;
                    for (int w = w0; w < w1; ++w) {
                        float run = 0.f;
#pragma unroll 4
                        for (int t = t0; t < t1; ++t) run += at[(h * rw + w) * rt + t];
                        plane += run;
                    }
                    sum += plane;
                }
                at += rt * rh * rw;
            }
        }
        out[b] = sum;
    }
}

// The same for layouts of so many tiles that their offsets do not fit a CTA's shared memory (over 7000 tiles): each
// bucket of a row is a box of its span's tile array (the classes are intervals of the offset), and a thread adds
// its buckets' boxes in a fixed order.
__global__ void __launch_bounds__(256) bias_backward_wide_kernel(const BiasBackwardArgs a) {
    extern __shared__ float row[];
    const int head = blockIdx.y, pairs = a.b.buckets - 2;
    const int i0 = blockIdx.x * a.rows_per_chunk, i1 = min(a.n, i0 + a.rows_per_chunk);
    const int nh = 2 * a.b.reach[1] - 1, nw = 2 * a.b.reach[2] - 1;
    float* out = a.partial + (int64_t(head) * gridDim.x + blockIdx.x) * a.b.buckets;
    float acc[kBiasMaxBuckets / 256] = {};
    for (int i = i0; i < i1; ++i) {
        const float* src = a.d_scores + (int64_t(head) * a.n + i) * a.n;
        __syncthreads();
        for (int j = threadIdx.x; j < a.n; j += 256) row[j] = src[j];
        __syncthreads();
        const int4 p = a.tile_pos[i];
        const int4 g = a.span_grid[p.x];
        const int end = g.x + g.y * g.z * g.w;
#pragma unroll
        for (int u = 0; u < kBiasMaxBuckets / 256; ++u) {
            const int b = threadIdx.x + 256 * u;
            if (b >= a.b.buckets) break;
            float sum = 0.f;
            if (b >= pairs) {
                const int lo = b == pairs ? 0 : end, hi = b == pairs ? g.x : a.n;
                for (int j = lo; j < hi; ++j) sum += row[j];
            } else {
                int t0, t1, h0, h1, w0, w1;
                bias_interval(a.b.starts[0], a.b.reach[0], b / (nw * nh), p.y, g.y, t0, t1);
                bias_interval(a.b.starts[1], a.b.reach[1], (b / nw) % nh, p.z, g.z, h0, h1);
                bias_interval(a.b.starts[2], a.b.reach[2], b % nw, p.w, g.w, w0, w1);
                for (int h = h0; h < h1; ++h) {
                    float plane = 0.f;
                    for (int w = w0; w < w1; ++w) {
                        float run = 0.f;
                        for (int t = t0; t < t1; ++t) run += row[g.x + (h * g.w + w) * g.y + t];
                        plane += run;
                    }
                    sum += plane;
                }
            }
            acc[u] += sum;
        }
    }
#pragma unroll
    for (int u = 0; u < kBiasMaxBuckets / 256; ++u) {
        const int b = threadIdx.x + 256 * u;
        if (b < a.b.buckets) out[b] = acc[u];
    }
}

// d_bias[head][b] = the chunks' sums, eight loads at a time, added as pairs and eight by eight (a programmatic dependent launch)
__global__ void __launch_bounds__(128) bias_reduce_kernel(const float* partial, float* d_bias, int chunks, int buckets) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.x * 128 + threadIdx.x;
    if (b >= buckets) return;
    const float* p = partial + int64_t(blockIdx.y) * chunks * buckets + b;
    float sum = 0.f;
    for (int c = 0; c < chunks; c += 8) {
        float v[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) v[x] = c + x < chunks ? p[int64_t(c + x) * buckets] : 0.f;
        sum += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
    d_bias[int64_t(blockIdx.y) * buckets + b] = sum;
}

}  // namespace veda
