// The teacher's tile logits: full attention's logits, max-pooled over every pair of 128-row tiles.
//     teacher[h, i, j] = max_{r in tile i, s in tile j} ( c q_r . k_s - lse_r ),   c = D^-1/2
// c > 0 and lse_r does not depend on s, so a row's part is c max_s(q_r . k_s) - lse_r: the pooling needs one
// maximum per logit, and scale and lse touch one number per row and tile.
//
// The product is the whole cost (2 S^2 D operations per head against 4 n^2 bytes written, n = S / 128), so the
// kernel is built to keep the tensor core fed: a work unit is two query tiles of a head against a run of key
// tiles. Q stays in shared memory; K streams through a ring two tiles at a time, so each MMA is 128 x 256 x 16
// and each K pair is used by both query tiles. Their two accumulators are all of TMEM (2 x 256 columns): while
// one is reduced by its four epilogue warps the other is being written. A row of the accumulator is a thread's;
// it takes the maximum of 128 columns per key tile two at a time (three-operand max), the warp's 32 rows meet in
// one redux, and a combiner warp joins the four warps' values of 32 key tiles and stores them as one row.
//   warp 0      TMA producer (Q once per unit, K pairs through the ring)
//   warp 1      MMA issuer
//   warps 2, 3  combiners of the two query tiles; warp 2 owns the TMEM allocation
//   warps 4-7, 8-11  epilogue of query tile 0 and 1
// Units are numbered head by head, key run by key run, so that the CTAs in flight read the same K run from L2.
// Every wait is bounded; a CTA that gives up lets its copies and MMAs finish, frees its TMEM and returns.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "wait.cuh"
#include "warp.cuh"

namespace veda {
namespace teacher {

constexpr int kThreads = 384;
constexpr int kStages = 2;
constexpr int kBatch = 16;                 // K pairs whose partial maxima a combiner takes at once
constexpr int kErrTimeoutBit = 1;
constexpr uint64_t kDrainNs = 200000000ull;

struct Bars {
    uint64_t q_full, q_empty;
    uint64_t k_full[kStages], k_empty[kStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t part_full[2][2], part_empty[2][2];
    uint64_t drain;
};

template <int D>
struct Cfg {
    static constexpr int kBoxes = D / 64;                  // 64-column (128-byte) boxes per tile
    static constexpr int kBox = 128 * 128;                 // bytes of one box
    static constexpr int kQBytes = 2 * kBoxes * kBox;      // both query tiles
    static constexpr int kStageBytes = 2 * kBoxes * kBox;  // a K pair: per box column, 256 rows
    static constexpr int kOffK = kQBytes;
    static constexpr int kOffPart = kOffK + kStages * kStageBytes;
    static constexpr int kPartBytes = 2 * 2 * 2 * kBatch * 4 * 4;  // [tile][buffer][key tile][warp]
    static constexpr int kOffBar = kOffPart + kPartBytes;
    static constexpr size_t kSmem = 1024 + size_t(kOffBar) + sizeof(Bars) + 16;
};

struct Maps {
    CUtensorMap q, k;  // [n_heads * N, D] bf16, boxes of 128 rows x 64 columns, 128-byte swizzle
};

struct Args {
    const int32_t* valid_count;  // [n_tiles]
    const int32_t* perm;         // [n_slots]
    const float* lse;            // [n_heads, seq_len] or null
    float* out;                  // [n_heads, n, n]
    int64_t seq_len;
    int n, n_tiles, groups, runs, pairs, units;  // groups of two query tiles; runs of key pairs
    float scale;
    uint64_t timeout_ns;
    int* err;
};

struct Unit {
    int head, q0, p0, p1;
    __device__ __forceinline__ Unit(const Args& a, int u) {
        const int per_head = a.groups * a.runs;
        head = u / per_head;
        const int r = u - head * per_head;
        const int run = r / a.groups;
        q0 = 2 * (r - run * a.groups);
        p0 = int(int64_t(a.pairs) * run / a.runs);
        p1 = int(int64_t(a.pairs) * (run + 1) / a.runs);
    }
};

// best = max(best, the first `cols` of 32 columns)
__device__ __forceinline__ float take(float best, const uint32_t (&v)[32], int cols) {
    if (cols >= 32) {
        float a = best, b = -INFINITY;
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            a = ptx::max3(a, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
            b = ptx::max3(b, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
        }
        return fmaxf(a, b);
    }
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (e < cols) best = fmaxf(best, __uint_as_float(v[e]));
    return best;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) teacher_kernel(const __grid_constant__ Maps maps, const Args a) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* part = reinterpret_cast<float*>(smem + C::kOffPart);
    Bars& B = *reinterpret_cast<Bars*>(smem + C::kOffBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(&B + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint64_t tmo = a.timeout_ns;

    if (threadIdx.x == 0) {
        ptx::mbar_init(&B.q_full, 1);
        ptx::mbar_init(&B.q_empty, 1);
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&B.k_full[s], 1);
            ptx::mbar_init(&B.k_empty[s], 1);
        }
        for (int g = 0; g < 2; ++g) {
            ptx::mbar_init(&B.acc_full[g], 1);
            ptx::mbar_init(&B.acc_empty[g], 128);
            for (int b = 0; b < 2; ++b) {
                ptx::mbar_init(&B.part_full[g][b], 4);
                ptx::mbar_init(&B.part_empty[g][b], 1);
            }
        }
        ptx::mbar_init(&B.drain, 1);
        *abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 0 && lane == 0) {
        ptx::tma_prefetch_desc(&maps.q);
        ptx::tma_prefetch_desc(&maps.k);
    }
    if (warp == 2) ptx::tmem_alloc(tmem_slot, 512);
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ---------------------------------------------------------------------------- TMA producer
        const uint64_t keep = ptx::policy_evict_last();  // every tile is read by many units
        int g = 0, lu = 0;   // K pairs and units issued (warp-uniform)
        bool stop = false;
        for (int u = blockIdx.x; u < a.units && !stop; u += gridDim.x, ++lu) {
            const Unit w(a, u);
            const int row0 = w.head * a.n_tiles * 128;
            if (!warp_wait(&B.q_empty, (lu & 1) ^ 1, abort_flag, tmo)) break;
            if (ptx::elect_one()) {
                ptx::mbar_arrive_expect_tx(&B.q_full, C::kQBytes);
                for (int t = 0; t < 2; ++t)  // the last group of an odd count takes its tile twice
                    for (int b = 0; b < C::kBoxes; ++b)
                        ptx::tma_load_2d_hint(smem + (t * C::kBoxes + b) * C::kBox, &maps.q, 64 * b,
                                              row0 + min(w.q0 + t, a.n - 1) * 128, &B.q_full, keep);
            }
            __syncwarp();
            for (int p = w.p0; p < w.p1; ++p, ++g) {
                const int s = g % kStages, ph = g / kStages;
                if (!warp_wait(&B.k_empty[s], (ph & 1) ^ 1, abort_flag, tmo)) {
                    stop = true;
                    break;
                }
                if (ptx::elect_one()) {
                    const int tiles = min(2, a.n - 2 * p);
                    uint8_t* st = smem + C::kOffK + s * C::kStageBytes;
                    ptx::mbar_arrive_expect_tx(&B.k_full[s], tiles * C::kBoxes * C::kBox);
                    for (int t = 0; t < tiles; ++t)
                        for (int b = 0; b < C::kBoxes; ++b)
                            ptx::tma_load_2d_hint(st + (2 * b + t) * C::kBox, &maps.k, 64 * b, row0 + (2 * p + t) * 128,
                                                  &B.k_full[s], keep);
                }
                __syncwarp();
            }
        }
        if (*abort_flag && lane == 0) {
            // every copy already issued must land before the CTA releases its shared memory
            volatile int never = 0;
            for (int k = (g > kStages ? g - kStages : 0); k < g; ++k)
                ptx::mbar_wait(&B.k_full[k % kStages], (k / kStages) & 1, &never, kDrainNs);
            if (lu > 0) ptx::mbar_wait(&B.q_full, (lu - 1) & 1, &never, kDrainNs);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------------------- MMA issuer
        constexpr uint32_t kPair = ptx::idesc_bf16_f32(128, 256, false, false);
        constexpr uint32_t kSingle = ptx::idesc_bf16_f32(128, 128, false, false);
        int g = 0, lu = 0;
        bool stop = false;
        for (int u = blockIdx.x; u < a.units && !stop; u += gridDim.x, ++lu) {
            const Unit w(a, u);
            if (!warp_wait(&B.q_full, lu & 1, abort_flag, tmo)) break;
            for (int p = w.p0; p < w.p1; ++p, ++g) {
                const int s = g % kStages, ph = g / kStages;
                if (!warp_wait(&B.k_full[s], ph & 1, abort_flag, tmo)) {
                    stop = true;
                    break;
                }
                const uint32_t id = 2 * p + 1 < a.n ? kPair : kSingle;
                const uint32_t kb = ptx::smem_addr(smem + C::kOffK + s * C::kStageBytes);
                for (int t = 0; t < 2; ++t) {
                    if (!warp_wait(&B.acc_empty[t], (g & 1) ^ 1, abort_flag, tmo)) {
                        stop = true;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t qb = ptx::smem_addr(smem + t * C::kBoxes * C::kBox);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint64_t qa = ptx::smem_desc_sw128(qb + (k / 4) * C::kBox, 16, 1024) + uint64_t((k % 4) * 2);
                        const uint64_t ka = ptx::smem_desc_sw128(kb + (k / 4) * 2 * C::kBox, 16, 1024) + uint64_t((k % 4) * 2);
                        ptx::mma_bf16_ss_w(tmem + 256u * t, qa, ka, id, k > 0 ? 1u : 0u);
                    }
                    ptx::mma_commit_w(&B.acc_full[t]);
                }
                if (stop) break;
                ptx::mma_commit_w(&B.k_empty[s]);
            }
            if (!stop) ptx::mma_commit_w(&B.q_empty);
        }
        // every product issued must be complete before the TMEM is released
        volatile int never = 0;
        ptx::mma_commit_w(&B.drain);
        ptx::mbar_wait(&B.drain, 0, &never, kDrainNs);
    } else if (warp < 4) {
        // ---------------------------------------------------------------------------- combiner
        const int t = warp - 2;
        int batch = 0;
        bool stop = false;
        for (int u = blockIdx.x; u < a.units && !stop; u += gridDim.x) {
            const Unit w(a, u);
            float* out = a.out + (int64_t(w.head) * a.n + w.q0 + t) * a.n;
            for (int p = w.p0; p < w.p1; p += kBatch, ++batch) {
                const int b = batch & 1;
                if (!warp_wait(&B.part_full[t][b], (batch >> 1) & 1, abort_flag, tmo)) {
                    stop = true;
                    break;
                }
                const float4 v = *reinterpret_cast<const float4*>(part + ((t * 2 + b) * 2 * kBatch + lane) * 4);
                const int j = 2 * p + lane;
                if (w.q0 + t < a.n && j < min(2 * w.p1, a.n)) out[j] = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&B.part_empty[t][b]);
            }
        }
    } else {
        // ---------------------------------------------------------------------------- epilogue
        const int t = (warp - 4) >> 2, q = warp & 3;  // query tile; TMEM lane quarter (rows 32 q ..)
        const uint32_t acc = tmem + 256u * t + (uint32_t(32 * q) << 16);
        int g = 0, batch = 0;
        bool stop = false;
        for (int u = blockIdx.x; u < a.units && !stop; u += gridDim.x) {
            const Unit w(a, u);
            const int tile = min(w.q0 + t, a.n - 1), r = 32 * q + lane;
            float off = INFINITY;  // a padding row: passed over
            if (r < a.valid_count[tile]) off = a.lse ? a.lse[w.head * a.seq_len + a.perm[tile * 128 + r]] : 0.f;
            const bool out = !isfinite(off);
            for (int p = w.p0; p < w.p1; ++p, ++g) {
                const int at = (p - w.p0) % kBatch, b = batch & 1;
                if (at == 0 &&
                    !warp_wait(&B.part_empty[t][b], ((batch >> 1) & 1) ^ 1, abort_flag, tmo)) {
                    stop = true;
                    break;
                }
                const int j0 = 2 * p, vj0 = a.valid_count[j0], vj1 = j0 + 1 < a.n ? a.valid_count[j0 + 1] : 0;
                if (!warp_wait(&B.acc_full[t], g & 1, abort_flag, tmo)) {
                    stop = true;
                    break;
                }
                ptx::tc_fence_after();
                float best[2] = {-INFINITY, -INFINITY};
                uint32_t x[32], y[32];
                ptx::tmem_ld32(acc, x);
#pragma unroll
                for (int c = 0; c < 8; c += 2) {
                    ptx::tmem_wait_ld();
                    ptx::tmem_ld32(acc + 32 * (c + 1), y);
                    best[c / 4] = take(best[c / 4], x, (c < 4 ? vj0 : vj1) - 32 * (c % 4));
                    ptx::tmem_wait_ld();
                    if (c < 6) ptx::tmem_ld32(acc + 32 * (c + 2), x);
                    if (c == 6) {
                        ptx::tc_fence_before();
                        ptx::mbar_arrive(&B.acc_empty[t]);  // the accumulator is in registers
                    }
                    best[c / 4] = take(best[c / 4], y, (c < 4 ? vj0 : vj1) - 32 * (c % 4 + 1));
                }
                const float m0 = warp_max(out ? -INFINITY : best[0] * a.scale - off);
                const float m1 = warp_max(out ? -INFINITY : best[1] * a.scale - off);
                const bool last = at == kBatch - 1 || p + 1 == w.p1;
                if (lane == 0) {
                    float* dst = part + ((t * 2 + b) * 2 * kBatch + 2 * at) * 4 + q;
                    dst[0] = m0;
                    dst[4] = m1;
                    if (last) ptx::mbar_arrive(&B.part_full[t][b]);
                }
                batch += last;
            }
        }
    }

    __syncthreads();
    if (warp == 2) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && *abort_flag) atomicOr(a.err, kErrTimeoutBit);
}

}  // namespace teacher
}  // namespace veda
