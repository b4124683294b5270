// fp32 products of the predictor's scores and of their gradients on the tensor cores:
//     C[batch] = scale A[batch] B[batch]^T (+ a residual, or + the relative position bias),
// A [M][K] and B [N][K] in any of three layouts in memory, read where they are (no transposed copies).
//
// Each fp32 operand is split into two tf32 parts, x = hi + lo, and a b is taken as hi_a hi_b + hi_a lo_b +
// lo_a hi_b (what is left out is under 1.25 x 2^-20 |a b|; score.cuh has the bound). Two things keep the sums at
// the level of fp32 rounding as well. The tensor core truncates when it adds into its accumulator, so errors of a
// long sum all have one sign and add up (one accumulator over K = 384 and three products loses 1.4e-6, measured;
// rounded fp32 sums lose 2e-7). So the small products (hi lo and lo hi) have an accumulator of their own, where a
// truncation is 2^-11 as large, and the sums are cut every kChunk values of K: the epilogue warps add each
// chunk's two accumulators into registers in rounded fp32.
//
// Persistent CTAs walk 128 x 128 output tiles; K runs in slices of 32 (one 128-byte swizzled row per operand row)
// through a ring of kStages stages, each the hi and lo parts of an A and a B slice:
//   warp 0       MMA issuer, 12 MMAs per slice; warp 1 owns the TMEM (two buffers of main + correction, 512 columns)
//   warps 4-11   epilogue, two warps per TMEM lane quarter with half of the columns each: TMEM -> sums in registers ->
//                global memory, 32 x 32 blocks transposed through shared memory
//   warps 12-19  producers, two groups that take the slices in turn: global -> registers -> hi and lo in the
//                swizzled layout, so one group's loads are in flight while the other one splits. A thread's piece
//                is 16 bytes of one operand row (4 values of K); with K innermost 8 lanes read one row's 128
//                bytes, with the rows innermost a warp reads 32 neighbouring rows, and either way 8 lanes store
//                to 8 different 16-byte banks.
// What bounds it: shared memory. A slice writes 64 KB and its MMAs read 96 KB, about 1250 cycles at 128 bytes per
// cycle against 768 cycles of tensor time.
// Every wait is bounded; a CTA that gives up lets its MMAs finish, frees its TMEM and returns.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "tf32.cuh"
#include "wait.cuh"

namespace veda {
namespace train {

constexpr int kBM = 128, kBN = 128, kBK = 32, kChunk = 128;
constexpr int kPart = 128 * kBK * 4;    // 16 KB: one 128-row slice of one operand part
constexpr int kStages = 2;
constexpr int kStageBytes = 4 * kPart;  // A hi, A lo, B hi, B lo
constexpr int kOffEpi = kStages * kStageBytes;
constexpr int kEpiBytes = 8 * 16 * 33 * 4;  // a 16 x 33 transpose block per epilogue warp
constexpr int kOffBar = kOffEpi + kEpiBytes;
constexpr int kThreads = 640;
constexpr int kEpilogue = 256;   // threads
constexpr int kGroup = 128;      // threads of one producer group
constexpr int kTimeoutBit = 1;
constexpr uint64_t kDrainNs = 200000000ull;

struct Bars {
    uint64_t full[kStages];   // producers (one arrival per warp) -> MMA
    uint64_t empty[kStages];  // MMA commit -> producers
    uint64_t acc_full[2];     // MMA commit -> epilogue
    uint64_t acc_empty[2];    // epilogue (one arrival per thread) -> MMA
    uint64_t drain;
};
constexpr size_t kSmem = 1024 + size_t(kOffBar) + sizeof(Bars) + 16;

enum Layout : int {
    kRowsVec = 0,  // element (r, k) at r * stride + k, rows of whole 16-byte pieces
    kRows = 1,     // the same without the alignment
    kCols = 2,     // element (r, k) at k * stride + r
};

struct Operand {
    const float* base;
    int64_t batch;   // elements between two batches
    int64_t stride;
    int rows;
    int layout;
};

struct Set {
    Operand a, b;
    float* C;                // [batch][M][N]
    const float* residual;   // element (m, n) at batch * residual_batch + m * residual_stride + n, or null
    int64_t residual_batch, residual_stride;
};

struct Args {
    Set set[2];
    int n_sets, nb;          // operand sets (1 or 2) of one shape, batches in each
    int M, N, K;
    int tiles_m, tiles_n, n_tiles;
    float scale;
    // the bias of score tiles (table null: none): table[batch][key number + query number], bias.cuh
    const float* table;
    const int4* tile_num;
    int64_t table_stride;
    int offsets;
    uint64_t timeout_ns;
    int* err;
};

struct Tile {
    int set, batch, m0, n0;
    __device__ __forceinline__ Tile(const Args& a, int t) {
        const int per_batch = a.tiles_m * a.tiles_n;
        const int bt = t / per_batch, r = t - bt * per_batch;
        set = bt / a.nb;
        batch = bt - set * a.nb;
        m0 = (r / a.tiles_n) * kBM;
        n0 = (r % a.tiles_n) * kBN;
    }
};

// Loads that stay where they are written: the compiler may otherwise move them behind the wait for a free stage, and
// then nothing hides their latency.
__device__ __forceinline__ float load1(const float* p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}
__device__ __forceinline__ float4 load4(const float* p) {
    float4 v;
    asm volatile("ld.global.nc.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}

// One operand as a producer thread (i of 128) reads it: eight 16-byte pieces of each slice. With kCols piece u is row i,
// values of K from 4 u; else it is row i / 8 + 16 u, values of K from 4 (i % 8).
struct Reader {
    const float* p;    // this thread's first value of slice 0
    uint32_t stride;
    int rows;          // rows of the tile from this thread's first one on
    int layout;
    bool inside;       // the whole tile's rows exist
    __device__ __forceinline__ Reader(const Operand& o, int batch, int r0, int i) {
        layout = o.layout;
        stride = uint32_t(o.stride);
        const int r = r0 + (layout == kCols ? i : i >> 3);
        rows = o.rows - r;
        inside = r0 + 128 <= o.rows;
        p = o.base + batch * o.batch + (layout == kCols ? int64_t(r) : int64_t(r) * o.stride + 4 * (i & 7));
    }
    __device__ __forceinline__ void load(float (&v)[32], int k0, int K, int i) const {
        const bool full = inside && k0 + kBK <= K;
        if (layout == kCols) {
            const float* q = p + int64_t(k0) * stride;
            if (full) {
#pragma unroll
                for (int x = 0; x < 32; ++x) v[x] = load1(q + uint32_t(x) * stride);
            } else {
                const int ks = rows > 0 ? K - k0 : 0;
#pragma unroll
                for (int x = 0; x < 32; ++x) v[x] = x < ks ? load1(q + uint32_t(x) * stride) : 0.f;
            }
        } else if (layout == kRowsVec) {
            const float* q = p + k0;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (full || (16 * u < rows && k0 + 4 * (i & 7) < K)) f = load4(q + 16 * u * stride);
                v[4 * u] = f.x;
                v[4 * u + 1] = f.y;
                v[4 * u + 2] = f.z;
                v[4 * u + 3] = f.w;
            }
        } else {
            const float* q = p + k0;
            const int ks = K - k0 - 4 * (i & 7);
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    v[4 * u + x] = full || (16 * u < rows && x < ks) ? load1(q + 16 * u * stride + x) : 0.f;
        }
    }
};

// x rounded to the nearest tf32 value, ties away from zero; infinities stay, a NaN's remainder stays NaN
__device__ __forceinline__ float hi_part(float x) { return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u); }

// the pieces as hi and lo parts in the 128-byte swizzle (16-byte piece c of row r at piece c ^ (r % 8))
__device__ __forceinline__ void store_slice(const float (&v)[32], uint8_t* part, int layout, int i) {
    const bool cols = layout == kCols;
    // piece u of a row's eight lies at c ^ (r % 8): r is fixed with kCols, c with the others, and r % 8 = (i / 8) % 8 there
    uint8_t* row = part + (cols ? i * 128 : (i >> 3) * 128 + (((i & 7) ^ ((i >> 3) & 7)) << 4));
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        uint8_t* dst = cols ? row + ((u ^ (i & 7)) << 4) : row + u * 2048;
        float4 h, l;
        h.x = hi_part(v[4 * u]);
        h.y = hi_part(v[4 * u + 1]);
        h.z = hi_part(v[4 * u + 2]);
        h.w = hi_part(v[4 * u + 3]);
        l.x = v[4 * u] - h.x;
        l.y = v[4 * u + 1] - h.y;
        l.z = v[4 * u + 2] - h.z;
        l.w = v[4 * u + 3] - h.w;
        *reinterpret_cast<float4*>(dst) = h;
        *reinterpret_cast<float4*>(dst + kPart) = l;
    }
}

__global__ void __launch_bounds__(kThreads, 1) gemm_kernel(const __grid_constant__ Args a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars& B = *reinterpret_cast<Bars*>(smem + kOffBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(&B + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nk = (a.K + kBK - 1) / kBK, nc = (a.K + kChunk - 1) / kChunk;
    const uint64_t tmo = a.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&B.full[s], kGroup / 32);
            ptx::mbar_init(&B.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&B.acc_full[b], 1);
            ptx::mbar_init(&B.acc_empty[b], kEpilogue);
        }
        ptx::mbar_init(&B.drain, 1);
        *abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 1) ptx::tmem_alloc(tmem_slot, 512);
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp < 4) {
        ptx::regs_dec<40>();
        if (warp == 0) {
            // ------------------------------------------------------------------------ MMA issuer
            constexpr uint32_t kId = tf32x3::idesc(kBM, kBN);
            int g = 0, gc = 0;  // slices and chunks consumed
            bool stop = false;
            for (int t = blockIdx.x; t < a.n_tiles && !stop; t += gridDim.x) {
                for (int kk = 0; kk < nk; ++kk, ++g) {
                    const int s = g % kStages, ph = g / kStages, b = gc & 1;
                    const bool first = kk % (kChunk / kBK) == 0;
                    if (first && !warp_wait(&B.acc_empty[b], ((gc >> 1) & 1) ^ 1, abort_flag, tmo)) {
                        stop = true;
                        break;
                    }
                    if (!warp_wait(&B.full[s], ph & 1, abort_flag, tmo)) {
                        stop = true;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t d = tmem + uint32_t(b * 256);
                    const uint32_t base = ptx::smem_addr(smem + s * kStageBytes);
                    const uint64_t ah = ptx::smem_desc_sw128(base, 16, 1024);
                    const uint64_t al = ptx::smem_desc_sw128(base + kPart, 16, 1024);
                    const uint64_t bh = ptx::smem_desc_sw128(base + 2 * kPart, 16, 1024);
                    const uint64_t bl = ptx::smem_desc_sw128(base + 3 * kPart, 16, 1024);
#pragma unroll
                    for (int k8 = 0; k8 < kBK / 8; ++k8) {
                        const uint64_t o = uint64_t(k8 * 2);  // 8 tf32 = 32 bytes per k-step, in 16-byte units
                        const uint32_t add = first && k8 == 0 ? 0u : 1u;
                        tf32x3::mma_ss_w(d, ah + o, bh + o, kId, add);
                        tf32x3::mma_ss_w(d + 128, al + o, bh + o, kId, add);
                        tf32x3::mma_ss_w(d + 128, ah + o, bl + o, kId, 1u);
                    }
                    ptx::mma_commit_w(&B.empty[s]);
                    if (kk % (kChunk / kBK) == kChunk / kBK - 1 || kk == nk - 1) {
                        ptx::mma_commit_w(&B.acc_full[b]);
                        ++gc;
                    }
                }
            }
            // every product issued must be complete before the TMEM is released
            volatile int never = 0;
            ptx::mma_commit_w(&B.drain);
            ptx::mbar_wait(&B.drain, 0, &never, kDrainNs);
        }
    } else if (warp < 12) {
        // ---------------------------------------------------------------------------- epilogue
        ptx::regs_inc<112>();
        const int q = warp & 3, half = (warp - 4) >> 2;  // TMEM lane quarter (rows 32 q ..), columns 64 half ..
        float* tr = reinterpret_cast<float*>(smem + kOffEpi) + (warp - 4) * 16 * 33;
        int gc = 0;
        bool stop = false;
        for (int t = blockIdx.x; t < a.n_tiles && !stop; t += gridDim.x) {
            const Tile w(a, t);
            float acc[64];
            for (int c = 0; c < nc; ++c, ++gc) {
                const int b = gc & 1;
                if (!warp_wait(&B.acc_full[b], (gc >> 1) & 1, abort_flag, tmo)) {
                    stop = true;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t taddr = tmem + (uint32_t(32 * q) << 16) + uint32_t(b * 256 + 64 * half);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t x[16], y[16];
                    ptx::tmem_ld16(taddr + 16 * j, x);
                    ptx::tmem_ld16(taddr + 128 + 16 * j, y);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float v = __uint_as_float(x[e]) + __uint_as_float(y[e]);
                        acc[16 * j + e] = c == 0 ? v : acc[16 * j + e] + v;
                    }
                }
                ptx::tc_fence_before();
                ptx::mbar_arrive(&B.acc_empty[b]);
            }
            if (stop) break;
            // (a select, not a.set[w.set]: a runtime index into the kernel arguments would copy them to the stack)
            float* C = (w.set ? a.set[1].C : a.set[0].C) + int64_t(w.batch) * a.M * a.N;
            const float* res = w.set ? a.set[1].residual : a.set[0].residual;
            const int64_t rs = a.set[0].residual_stride;
            if (res) res += w.batch * a.set[0].residual_batch;
            const float* table = a.table ? a.table + w.batch * a.table_stride : nullptr;
            const int row0 = w.m0 + 32 * q;
            int4 query = make_int4(0, 0, 0, 0);
            if (table) query = a.tile_num[min(row0 + lane, a.M - 1)];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int n = w.n0 + 64 * half + 32 * j + lane, nn = min(n, a.N - 1);
                int4 key = make_int4(0, 0, 0, 0);
                if (table) key = a.tile_num[nn];
                // sixteen rows at a time: the lanes that hold them lay them down, and what is added to them is loaded
                // while they do, from clamped places
#pragma unroll
                for (int r16 = 0; r16 < 32; r16 += 16) {
                    float more[16];
                    if (table) {
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            const int span = __shfl_sync(0xffffffffu, query.x, r16 + x);
                            const int num = __shfl_sync(0xffffffffu, query.z, r16 + x);
                            more[x] = __ldg(table + (key.x != span ? a.offsets + (key.x > span) : key.y + num));
                        }
                    } else if (res) {
#pragma unroll
                        for (int x = 0; x < 16; ++x) more[x] = __ldg(res + min(row0 + r16 + x, a.M - 1) * rs + nn);
                    } else {
#pragma unroll
                        for (int x = 0; x < 16; ++x) more[x] = 0.f;
                    }
                    if ((lane & 16) == r16) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) tr[(lane & 15) * 33 + e] = acc[32 * j + e];
                    }
                    __syncwarp();
                    float* dst = C + int64_t(row0 + r16) * a.N + n;
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const float v = tr[x * 33 + lane] * a.scale + more[x];
                        if (row0 + r16 + x < a.M && n < a.N) dst[int64_t(x) * a.N] = v;
                    }
                    __syncwarp();
                }
            }
        }
    } else {
        // ---------------------------------------------------------------------------- producers
        ptx::regs_inc<104>();
        const int i = threadIdx.x & (kGroup - 1), group = (warp - 12) >> 2;
        int g = 0;  // slices of the tiles before this one; a group takes every second slice of the CTA's sequence
        bool stop = false;
        for (int t = blockIdx.x; t < a.n_tiles && !stop; t += gridDim.x, g += nk) {
            const Tile w(a, t);
            const Reader ra(w.set ? a.set[1].a : a.set[0].a, w.batch, w.m0, i);
            const Reader rb(w.set ? a.set[1].b : a.set[0].b, w.batch, w.n0, i);
            for (int kk = (group ^ g) & 1; kk < nk; kk += 2) {
                float va[32], vb[32];
                ra.load(va, kk * kBK, a.K, i);
                rb.load(vb, kk * kBK, a.K, i);
                const int s = (g + kk) % kStages, ph = (g + kk) / kStages;
                if (!warp_wait(&B.empty[s], (ph & 1) ^ 1, abort_flag, tmo)) {
                    stop = true;
                    break;
                }
                uint8_t* st = smem + s * kStageBytes;
                store_slice(va, st, ra.layout, i);
                store_slice(vb, st + 2 * kPart, rb.layout, i);
                tf32x3::fence_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&B.full[s]);
            }
        }
    }

    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
    if (threadIdx.x == 0 && *abort_flag) atomicOr(a.err, kTimeoutBit);
}

}  // namespace train
}  // namespace veda
