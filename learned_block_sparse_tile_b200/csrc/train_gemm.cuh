// fp32 products of the predictor's scores and of their gradients on the tensor cores:
//     C[batch][n][m] = scale sum_k A[batch](m, k) B[batch](n, k)  (+ the relative position bias),
// the operands read where they are, in any of three layouts (no transposed copies).
//
// Each fp32 operand is split into two tf32 parts, x = hi + lo, and a b is taken as hi_a hi_b + hi_a lo_b +
// lo_a hi_b (what is left out is under 1.25 x 2^-20 |a b|; score.cuh has the bound). What keeps the sums at
// the level of fp32 rounding as well: the tensor core truncates when it adds into its accumulator, so the errors of a
// long sum all have one sign and add up. So the sums are cut at every slice of 32 values of K, and the epilogue warps add
// the slices' sums in registers in rounded fp32; and a slice's small products go first, into an accumulator that is still
// small. Scores of 819 tiles, 24 heads against 64 bits: 3.9e-6 with one accumulator, 1.0e-6 with sums of 64 values, 3.3e-7
// with these (97 us instead of 95 when it came in); fp32 products leave 4.5e-7.
//
// Times here are of runs of a few milliseconds, as each step was taken; the kernels now take 95 us (scores) and 97 us
// (gradients, both launches), 98 and 110 in half a second of calls from the host.
//
// The projections' residual, feats @ P + feats[:, :D] = feats @ (P + E) with E the identity in P's first D rows, is added to
// A as it is split.
//
// Both operands need the split, and it is shared memory that bounds the kernel (with both parts of both operands in
// shared memory an MMA of 128 x 128 x 8 takes 117 cycles instead of 64, measured). So A, whose row a thread can hold, goes
// to tensor memory straight from its registers, and only B is laid down in shared memory. The products are written
// so that A's rows are innermost in memory (a warp reads 32 neighbouring rows at one k), which also makes the
// lanes of an accumulator neighbours in C: the epilogue stores whole 128-byte lines without a transpose.
//
// Persistent CTAs walk 128 x 128 tiles; the tiles that do not fill the last round of CTAs are cut along K where that saves
// more slices than joining them costs (join_kernel). K runs in slices of 32:
//   warp 0       MMA issuer, 12 MMAs per slice; warp 1 owns the TMEM: the sums twice (columns 0-255) and kStages
//                stages of A's hi and lo parts (256-511)
//   warp 2       TMA producer: raw slices of both operands into the split groups' stages
//   warps 1, 3   the bias table that the score launch after this one reads, where it is asked for
//   8 or 16      epilogue warps, two or four per lane quarter with a part of the columns each; their sums start from the bias,
//                whose loads pass while the tile is computed. Scores, whose tiles have few slices for their 128 x 128
//                biases and stores, take four warps a quarter (104k rows, 24 heads: 93 us; two: 96), gradients two (uncut
//                along K 96 us; four: 102)
//   12           split warps, three groups with a stage each that take the slices in turn, so that one group's waits pass while
//                others work. Thread i of 128 has row i of both operands: it reads its 32 values of K (rows of K lie in
//                the 128-byte swizzle, so that 8 lanes' 16-byte pieces fall into 8 different banks; columns are
//                neighbours for neighbouring lanes), and writes A's parts to its TMEM lane and B's in the swizzle that
//                the MMA reads.
// A score gradient whose row length n is no multiple of four values has no tensor map of its own: its rows start off the
// 16-byte boundaries. But every fourth row does have one, with a stride of 4 n values, from the boundary before its first
// value: four maps, one for each remainder b of the row's number (over all batches), in which row 4 a + b begins at
// place (b n) % 4. A slice is four boxes, one value quad wider and one row higher than its share; a thread reads its
// values at their places. (The gradient of 819-tile scores, both kernels: 275 us with values copied one by one, 340 with
// a bulk copy per piece of a row, 127 with 16-byte copies by the split warps.)
// Every wait is bounded; a CTA that gives up lets its MMAs finish, frees its TMEM and returns.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "bias.cuh"
#include "ptx.cuh"
#include "tf32.cuh"
#include "wait.cuh"

namespace veda {
namespace train {

constexpr int kBM = 128, kBN = 128, kBK = 32;
constexpr int kPart = 128 * kBK * 4;    // 16 KB: one 128-row slice of an operand, raw or one part of it
constexpr int kStageBytes = 2 * kPart;  // B hi, B lo
constexpr int kStages = 3;              // of the raw slices (A, B) and of their parts; a split group has one of each
constexpr int kQuadRows = 33, kQuadWidth = 36;   // a box of a quarter of 128 rows x 32 K (kRows) ...
constexpr int kQuadK = 9, kQuadCols = 132;       // ... and of 32 K x 128 rows (kCols), in rows and values
constexpr int kQuadBytes = kQuadRows * kQuadWidth * 4, kQuadStep = 4864;  // boxes lie on 128-byte boundaries
static_assert(kQuadBytes == kQuadK * kQuadCols * 4 && kQuadBytes <= kQuadStep && kQuadStep % 128 == 0, "boxes of one size");
constexpr int kRawB = 4 * kQuadStep;      // 19 KB (a slice of a dense map takes 16)
constexpr int kRawBytes = kPart + kRawB;  // A, B
constexpr int kOffRaw = kStages * kStageBytes;
constexpr int kOffBar = kOffRaw + kStages * kRawBytes;
static_assert(kRawBytes % 1024 == 0, "raw slices lie in whole swizzle atoms");
constexpr int kGroup = 128;      // threads of one split group; as many groups as stages
constexpr uint32_t kStageA = 256;  // TMEM column of the first stage
constexpr int kTimeoutBit = 1;
constexpr uint64_t kDrainNs = 200000000ull;

struct Bars {
    uint64_t raw_full[kStages];   // TMA -> split (transaction bytes)
    uint64_t raw_empty[kStages];  // split (one arrival per warp) -> TMA
    uint64_t full[kStages];    // split (one arrival per warp) -> MMA
    uint64_t empty[kStages];   // MMA commit -> split
    uint64_t acc_full[2];      // MMA commit -> epilogue
    uint64_t acc_empty[2];     // epilogue (one arrival per thread) -> MMA
    uint64_t drain;
};
constexpr size_t kSmem = 1024 + size_t(kOffBar) + sizeof(Bars) + 16;

enum Layout : int {
    kRows = 0,  // element (r, k) at r * stride + k
    kCols = 1,  // element (r, k) at k * stride + r
};

struct Operand {
    const float* base;
    int64_t batch;   // elements between two batches
    int64_t stride;
    int rows;
    int layout;
    int dense;       // one tensor map; 0: four, one for every fourth row (B only)
};

struct Maps {
    CUtensorMap a[2];     // boxes of 32 K x 128 rows, 128-byte swizzle (kRows), or 128 rows x 32 K (kCols)
    CUtensorMap b[2][4];  // the same in b[set][0], or every fourth row's in boxes of kQuadWidth x kQuadRows or kQuadCols x kQuadK
};

struct Set {
    Operand a, b;
    float* C;  // [batch][N][M]
};

struct Args {
    Set set[2];
    int n_sets, nb;         // operand sets (1 or 2) of one shape, batches in each
    int M, N, K;
    int tiles_m, tiles_n;
    int full, parts, n_units;  // tiles of one unit each, then the others' K in `parts` units each
    float* partial;            // [units of split tiles][128 of N][128 of M]
    float scale;
    int identity;           // A(m, m) + 1 in the place of A(m, m)
    // the bias of score tiles (table null: none), m the key and n the query: scale table[batch][key number + query number]
    const float* table;
    const int4* tile_num;
    int64_t table_stride;
    int offsets, one_span;
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

// A work unit: slices [k0, k1) of a tile; the tiles that do not fill the last round of CTAs are cut along K.
struct Unit : Tile {
    int k0 = 0, k1, part = -1;  // part: the unit's place among those of split tiles, or -1
    __device__ __forceinline__ Unit(const Args& a, int u, int nk) : Tile(a, u), k1(nk) {
        if (u >= a.full) {
            part = u - a.full;
            const int t = part / a.parts, p = part - t * a.parts;
            static_cast<Tile&>(*this) = Tile(a, a.full + t);
            k0 = nk * p / a.parts;
            k1 = nk * (p + 1) / a.parts;
        }
    }
};
__device__ __forceinline__ int unit_slices(const Args& a, int u, int nk) {
    if (u < a.full) return nk;
    const int p = (u - a.full) % a.parts;
    return nk * (p + 1) / a.parts - nk * p / a.parts;
}

// C of the split tiles: their parts' sums, in order (a programmatic dependent launch; 16 CTAs a tile)
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Args a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Tile w(a, a.full + blockIdx.y);
    const float* p = a.partial + int64_t(blockIdx.y) * a.parts * (kBM * kBN);
    float* C = (w.set ? a.set[1].C : a.set[0].C) + int64_t(w.batch) * a.M * a.N;
    const int e = (blockIdx.x * 256 + threadIdx.x) * 4, n = w.n0 + e / kBM, m = w.m0 + e % kBM;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = 0; x < a.parts; ++x) {
        const float4 v = *reinterpret_cast<const float4*>(p + int64_t(x) * (kBM * kBN) + e);
        sum.x += v.x;
        sum.y += v.y;
        sum.z += v.z;
        sum.w += v.w;
    }
    const float v[4] = {sum.x, sum.y, sum.z, sum.w};
    if (n < a.N)
        for (int x = 0; x < 4; ++x)
            if (m + x < a.M) C[int64_t(n) * a.M + m + x] = v[x] * a.scale;
}

// Loads that stay where they are written, ahead of the waits that hide their latency.
__device__ __forceinline__ float load1(const float* p) {
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(p));
    return v;
}

// a box of a tensor map into L2
__device__ __forceinline__ void prefetch_3d(const void* desc, int32_t c0, int32_t c1, int32_t c2) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(desc)), "r"(c0),
                 "r"(c1), "r"(c2)
                 : "memory");
}

// Half h of this thread's row of a raw slice (row i, K from 16 h).
__device__ __forceinline__ void read_raw(float (&v)[16], const uint8_t* raw, int layout, int h, int i) {
    if (layout == kCols) {
        const float* p = reinterpret_cast<const float*>(raw) + 2048 * h + i;
#pragma unroll
        for (int x = 0; x < 16; ++x) v[x] = p[128 * x];
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float4 f = *reinterpret_cast<const float4*>(raw + i * 128 + (((4 * h + u) ^ (i & 7)) << 4));
            v[4 * u] = f.x;
            v[4 * u + 1] = f.y;
            v[4 * u + 2] = f.z;
            v[4 * u + 3] = f.w;
        }
    }
}

// The same of a slice of four boxes. `first`: the number over all batches of the slice's first row (kRows), or of its first
// k (kCols); n the row length; values from ks on are zero (with kCols a k past the operand's is the next batch's row).
// Neighbouring lanes read neighbouring banks: with kRows four rows share a bank group and begin at four different places.
__device__ __forceinline__ void read_quads(float (&v)[16], const uint8_t* raw, int layout, int first, int n, int ks, int h, int i) {
    const float* q = reinterpret_cast<const float*>(raw);
    constexpr int kStep = kQuadStep / 4;
    if (layout == kCols) {
        const float* p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int x = (first & 3) + j, b = x & 3;
            p[j] = q + b * kStep + ((b * n) & 3) + (x >> 2) * kQuadCols + i;
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) v[x] = p[x & 3][(4 * h + (x >> 2)) * kQuadCols];
        if (16 * h + 16 > ks) {
#pragma unroll
            for (int x = 0; x < 16; ++x)
                if (16 * h + x >= ks) v[x] = 0.f;
        }
    } else {
        const int x = (first & 3) + i, b = x & 3;
        const float* p = q + b * kStep + ((b * n) & 3) + (x >> 2) * kQuadWidth + 16 * h;
#pragma unroll
        for (int x = 0; x < 16; ++x) v[x] = p[x];
    }
}

// x rounded to the nearest tf32 value, ties away from zero, but no farther than the largest one: a finite value's remainder
// stays finite, an infinity's carries it, and a NaN's is NaN. Products with an infinity are then infinite as fp32's are; but
// the largest value times a partner's remainder may pass the type's range with the other sign, and the sum is NaN, where the
// partners add up to 2^11 or more. The bound is the third of the split's instructions (819 tiles, 24 heads: scores 93.7 ->
// 95.2 us, gradients 94.3 -> 97.0).
__device__ __forceinline__ float hi_part(float x) {
    float r = __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u);
    asm("min.xorsign.abs.f32 %0, %0, 0f7F7FE000;" : "+f"(r));
    return r;
}

// Half `half` of B's values of this thread's row as hi and lo parts in the 128-byte swizzle (16-byte piece c of row r at
// piece c ^ (r % 8))
__device__ __forceinline__ void store_b(const float (&v)[16], uint8_t* part, int half, int i) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        uint8_t* dst = part + i * 128 + (((4 * half + u) ^ (i & 7)) << 4);
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

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]),
        "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
        : "memory");
}

// Half of A's values of this thread's row (its TMEM lane): hi parts in 16 columns, lo parts 32 columns behind them
__device__ __forceinline__ void store_a(const float (&v)[16], uint32_t taddr) {
    float h[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) h[x] = hi_part(v[x]);
    tmem_st16(taddr, h);
#pragma unroll
    for (int x = 0; x < 16; ++x) h[x] = v[x] - h[x];
    tmem_st16(taddr + 32, h);
}

// D[tmem] (+)= A[tmem] * B[smem desc], kind::tf32: A (M x K) in lanes 0..M-1, one value per column
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t id, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(id), "r"(accumulate)
        : "memory");
}

// kParts: epilogue warps per lane quarter, and the parts of a tile's columns
constexpr int threads_of(int parts) { return 32 * (4 + 4 * parts) + kStages * kGroup; }
template <int kParts>
__global__ void __launch_bounds__(threads_of(kParts), 1) gemm_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a,
                                                           const __grid_constant__ BiasExpand expand) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars& B = *reinterpret_cast<Bars*>(smem + kOffBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(&B + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    constexpr int kWide = kBN / kParts, kSplitWarp = 4 + 4 * kParts;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nk = (a.K + kBK - 1) / kBK;
    const uint64_t tmo = a.timeout_ns;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&B.raw_full[s], 1);
            ptx::mbar_init(&B.raw_empty[s], kGroup / 32);
        }
        for (int s = 0; s < kStages; ++s) {
            ptx::mbar_init(&B.full[s], kGroup / 32);
            ptx::mbar_init(&B.empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            ptx::mbar_init(&B.acc_full[s], 1);
            ptx::mbar_init(&B.acc_empty[s], 128 * kParts);
        }
        ptx::mbar_init(&B.drain, 1);
        *abort_flag = 0;
        ptx::fence_barrier_init();
    }
    if (warp == 1) ptx::tmem_alloc(tmem_slot, 512);
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // (programmatic dependent launch: what is above may run while the launch before this one still does)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp < 4) {
        ptx::regs_dec<kParts == 2 ? 56 : 40>();
        if (warp == 0) {
            // ------------------------------------------------------------------------ MMA issuer
            constexpr uint32_t kId = tf32x3::idesc(kBM, kBN);
            int g = 0;  // slices consumed
            bool stop = false;
            for (int u = blockIdx.x; u < a.n_units && !stop; u += gridDim.x) {
                for (int left = unit_slices(a, u, nk); left > 0; --left, ++g) {
                    const int s = g % kStages, b = g & 1;
                    if (!warp_wait(&B.acc_empty[b], ((g >> 1) & 1) ^ 1, abort_flag, tmo) ||
                        !warp_wait(&B.full[s], (g / kStages) & 1, abort_flag, tmo)) {
                        stop = true;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t d = tmem + uint32_t(b * 128), ah = tmem + kStageA + uint32_t(s * 64);
                    const uint32_t base = ptx::smem_addr(smem + s * kStageBytes);
                    const uint64_t bh = ptx::smem_desc_sw128(base, 16, 1024);
                    const uint64_t bl = ptx::smem_desc_sw128(base + kPart, 16, 1024);
                    // 8 tf32 = 32 bytes of B per k-step (2 of the descriptor's 16-byte units), 8 columns of A
#pragma unroll
                    for (int k8 = 0; k8 < kBK / 8; ++k8) {
                        mma_ts(d, ah + 32 + 8 * k8, bh + uint64_t(2 * k8), kId, k8 > 0 ? 1u : 0u);
                        mma_ts(d, ah + 8 * k8, bl + uint64_t(2 * k8), kId, 1u);
                    }
#pragma unroll
                    for (int k8 = 0; k8 < kBK / 8; ++k8) mma_ts(d, ah + 8 * k8, bh + uint64_t(2 * k8), kId, 1u);
                    ptx::mma_commit_w(&B.empty[s]);
                    ptx::mma_commit_w(&B.acc_full[b]);
                }
            }
            // every product issued must be complete before the TMEM is released
            volatile int never = 0;
            ptx::mma_commit_w(&B.drain);
            ptx::mbar_wait(&B.drain, 0, &never, kDrainNs);
        } else if (warp == 2) {
            // ------------------------------------------------------------------------ TMA producer
            const uint64_t keep = ptx::policy_evict_last();  // operand rows are read by several tiles
            int g = 0;
            bool stop = false;
            for (int u = blockIdx.x; u < a.n_units && !stop; u += gridDim.x) {
                const Unit w(a, u, nk);
                const int la = w.set ? a.set[1].a.layout : a.set[0].a.layout;
                const int lb = w.set ? a.set[1].b.layout : a.set[0].b.layout;
                const int dense = w.set ? a.set[1].b.dense : a.set[0].b.dense;
                const int row0 = w.batch * (lb == kCols ? a.K : a.N);  // the batch's first row, over all of them
                const CUtensorMap *ma = w.set ? &maps.a[1] : &maps.a[0], *mb = w.set ? maps.b[1] : maps.b[0];
                for (int kk = w.k0; kk < w.k1; ++kk, ++g) {
                    const int s = g % kStages, ph = g / kStages, k0 = kk * kBK;
                    // a stage is refilled as soon as it is read, which leaves no time for memory's latency: the slice
                    // after the stages' comes into L2 meanwhile
                    if (kk + kStages < w.k1 && ptx::elect_one()) {
                        const int k1 = k0 + kStages * kBK;
                        prefetch_3d(ma, la == kCols ? w.m0 : k1, la == kCols ? k1 : w.m0, w.batch);
                        if (dense) {
                            prefetch_3d(mb, lb == kCols ? w.n0 : k1, lb == kCols ? k1 : w.n0, w.batch);
                        } else {
                            for (int b = 0; b < 4; ++b)
                                prefetch_3d(mb + b, lb == kCols ? w.n0 : k1, (row0 + (lb == kCols ? k1 : w.n0)) >> 2, 0);
                        }
                    }
                    __syncwarp();
                    if (!warp_wait(&B.raw_empty[s], (ph & 1) ^ 1, abort_flag, tmo)) {
                        stop = true;
                        break;
                    }
                    if (ptx::elect_one()) {
                        uint8_t* raw = smem + kOffRaw + s * kRawBytes;
                        ptx::mbar_arrive_expect_tx(&B.raw_full[s], kPart + (dense ? kPart : 4 * kQuadBytes));
                        ptx::tma_load_3d_hint(raw, ma, la == kCols ? w.m0 : k0, la == kCols ? k0 : w.m0, w.batch,
                                              &B.raw_full[s], keep);
                        if (dense) {
                            ptx::tma_load_3d_hint(raw + kPart, mb, lb == kCols ? w.n0 : k0, lb == kCols ? k0 : w.n0, w.batch,
                                                  &B.raw_full[s], keep);
                        } else {
                            for (int b = 0; b < 4; ++b)
                                ptx::tma_load_3d_hint(raw + kPart + b * kQuadStep, mb + b, lb == kCols ? w.n0 : k0,
                                                      (row0 + (lb == kCols ? k0 : w.n0)) >> 2, 0, &B.raw_full[s], keep);
                        }
                    }
                    __syncwarp();
                }
            }
            if (*abort_flag && lane == 0) {
                // every copy already issued must land before the CTA releases its shared memory
                volatile int never = 0;
                for (int k = (g > kStages ? g - kStages : 0); k < g; ++k)
                    ptx::mbar_wait(&B.raw_full[k % kStages], (k / kStages) & 1, &never, kDrainNs);
            }
        } else if (expand.bias) {
            // ------------------------------------------------------------------------ the bias table (warps 1 and 3)
            for (int i = (blockIdx.x * 2 + (warp >> 1)) * 32 + lane; i < expand.count + 2; i += gridDim.x * 64) bias_expand(expand, i);
        }
    } else if (warp < kSplitWarp) {
        // ---------------------------------------------------------------------------- epilogue
        if constexpr (kParts == 2) ptx::regs_inc<88>();
        else ptx::regs_dec<56>();
        const int q = warp & 3, part = (warp - 4) >> 2;  // TMEM lane quarter (m 32 q ..), columns kWide part ..
        int g = 0;
        bool stop = false;
        for (int u = blockIdx.x; u < a.n_units && !stop; u += gridDim.x) {
            const Unit w(a, u, nk);
            const uint32_t lanes = tmem + (uint32_t(32 * q) << 16) + uint32_t(kWide * part);
            const int m = w.m0 + 32 * q + lane, mm = min(m, a.M - 1), n0 = w.n0 + kWide * part;
            const int left = a.N - n0;
            float acc[kWide];  // what is added to the product, over its scale, then the sums; loads from clamped places
            if (a.table) {
                const float* table = a.table + w.batch * a.table_stride;
                const int4 key = a.tile_num[mm];
#pragma unroll
                for (int j = 0; j < kWide; j += 32) {
                    const int4 mine = a.tile_num[min(n0 + j + lane, a.N - 1)];
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        int o = key.y + __shfl_sync(0xffffffffu, mine.z, x);
                        if (!a.one_span) {
                            const int span = __shfl_sync(0xffffffffu, mine.x, x);
                            if (key.x != span) o = a.offsets + (key.x > span);
                        }
                        acc[j + x] = load1(table + o);
                    }
                }
            } else {
#pragma unroll
                for (int x = 0; x < kWide; ++x) acc[x] = 0.f;
            }
            const auto add = [&](uint32_t from) {
#pragma unroll
                for (int j = 0; j < kWide; j += 16) {
                    uint32_t x[16];
                    ptx::tmem_ld16(from + j, x);
                    ptx::tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[j + e] += __uint_as_float(x[e]);
                }
            };
            for (int kk = w.k0; kk < w.k1; ++kk, ++g) {
                const int b = g & 1;
                if (!warp_wait(&B.acc_full[b], (g >> 1) & 1, abort_flag, tmo)) {
                    stop = true;
                    break;
                }
                ptx::tc_fence_after();
                add(lanes + uint32_t(b * 128));
                ptx::tc_fence_before();
                ptx::mbar_arrive(&B.acc_empty[b]);
            }
            if (stop) break;
            if (w.part >= 0) {
                float* P = a.partial + (int64_t(w.part) * kBN + kWide * part) * kBM + (m - w.m0);
#pragma unroll
                for (int x = 0; x < kWide; ++x) P[x * kBM] = acc[x];
            } else if (m < a.M) {
                // (a select, not a.set[w.set]: a runtime index into the kernel arguments would copy them to the stack)
                float* C = (w.set ? a.set[1].C : a.set[0].C) + int64_t(w.batch) * a.M * a.N + int64_t(n0) * a.M + m;
                if (left >= kWide) {
#pragma unroll
                    for (int x = 0; x < kWide; ++x) C[uint32_t(x) * uint32_t(a.M)] = acc[x] * a.scale;
                } else {
#pragma unroll
                    for (int x = 0; x < kWide; ++x)
                        if (x < left) C[uint32_t(x) * uint32_t(a.M)] = acc[x] * a.scale;
                }
            }
        }
    } else {
        // ---------------------------------------------------------------------------- split
        if constexpr (kParts == 2) ptx::regs_dec<80>();
        else ptx::regs_inc<80>();
        const int s = (warp - kSplitWarp) >> 2, i = threadIdx.x & (kGroup - 1);  // the group's number is its stage's
        const uint32_t stage_a = tmem + kStageA + uint32_t(64 * s) + (uint32_t(32 * (warp & 3)) << 16);
        uint8_t* stage_b = smem + s * kStageBytes;
        const uint8_t* raw = smem + kOffRaw + s * kRawBytes;
        // this group's slices, every kStages-th of the CTA's sequence: unit u, its slice `at`, number `use` of the group
        int u = blockIdx.x, at = s, use = 0;
        int slices = u < a.n_units ? unit_slices(a, u, nk) : 0;
        const auto settle = [&] {  // `at` within its unit
            while (u < a.n_units && at >= slices) {
                at -= slices;
                u += gridDim.x;
                if (u < a.n_units) slices = unit_slices(a, u, nk);
            }
        };
        settle();
        int mine = -1;
        Unit w(a, min(u, a.n_units - 1), nk);
        while (u < a.n_units) {
            if (u != mine) {
                w = Unit(a, u, nk);
                mine = u;
            }
            const Operand& ob = w.set ? a.set[1].b : a.set[0].b;
            const int la = w.set ? a.set[1].a.layout : a.set[0].a.layout, kk = w.k0 + at;
            if (!warp_wait(&B.raw_full[s], use & 1, abort_flag, tmo) ||
                !warp_wait(&B.empty[s], (use & 1) ^ 1, abort_flag, tmo))
                break;
            ptx::tc_fence_after();
            if (ob.dense) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[16];
                    read_raw(v, raw + kPart, ob.layout, h, i);
                    store_b(v, stage_b, h, i);
                }
            } else {
                const int first = ob.layout == kCols ? w.batch * a.K + kk * kBK : w.batch * a.N + w.n0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v[16];
                    read_quads(v, raw + kPart, ob.layout, first, int(ob.stride), a.K - kk * kBK, h, i);
                    store_b(v, stage_b, h, i);
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float v[16];
                read_raw(v, raw, la, h, i);
                if (a.identity && kk * kBK < a.M) {
                    const int one = w.m0 + i - kk * kBK - 16 * h;
#pragma unroll
                    for (int x = 0; x < 16; ++x) v[x] += x == one ? 1.f : 0.f;
                }
                store_a(v, stage_a + 16 * h);
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&B.raw_empty[s]);
            tf32x3::fence_async_smem();
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&B.full[s]);
            at += kStages;
            settle();
            ++use;
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
