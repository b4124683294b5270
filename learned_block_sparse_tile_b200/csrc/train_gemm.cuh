// fp32 products of the predictor's scores with a bias and of their gradients:
// C[batch] = epilogue(A[batch] B[batch]^T), 128 x 128 tiles, 256 threads with 8 x 8 sums each.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace veda {
namespace train {

// element (row, k) of an operand at base + batch * sb + row * sr + k * sk; zero outside [rows) x [K)
template <class T>
struct Operand {
    const T* base;
    int64_t sb, sr, sk;
    int rows;
    __device__ __forceinline__ float at(int batch, int r, int k, int K) const {
        return r < rows && k < K ? float(base[batch * sb + r * sr + k * sk]) : 0.f;
    }
};

template <class T, class Epilogue>
__global__ void __launch_bounds__(256) gemm_kernel(const Operand<T> A, const Operand<T> B, const int K, const Epilogue epi) {
    __shared__ float as[16][132], bs[16][132];
    const int m0 = blockIdx.y * 128, n0 = blockIdx.x * 128, batch = blockIdx.z;
    const int tm = (threadIdx.x >> 4) * 8, tn = (threadIdx.x & 15) * 8;
    float c[8][8] = {};
    for (int k0 = 0; k0 < K; k0 += 16) {
        for (int e = threadIdx.x; e < 2048; e += 256) {
            const int ra = A.sk == 1 ? e >> 4 : e & 127, ka = A.sk == 1 ? e & 15 : e >> 7;
            const int rb = B.sk == 1 ? e >> 4 : e & 127, kb = B.sk == 1 ? e & 15 : e >> 7;
            as[ka][ra] = A.at(batch, m0 + ra, k0 + ka, K);
            bs[kb][rb] = B.at(batch, n0 + rb, k0 + kb, K);
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) c[i][j] = fmaf(as[k][tm + i], bs[k][tn + j], c[i][j]);
        __syncthreads();
    }
    epi(c, batch, m0, n0, tm, tn);
}

// C = scale * AB^T (+ residual[m][n] at its own stride)
struct StoreEpilogue {
    float* C;
    int64_t cb;
    int M, N;
    float scale;
    const float* residual;
    int64_t rb, rs;
    __device__ void operator()(float (&c)[8][8], int batch, int m0, int n0, int tm, int tn) const {
        for (int i = 0; i < 8; ++i)
            for (int j = 0; j < 8; ++j) {
                const int m = m0 + tm + i, n = n0 + tn + j;
                if (m < M && n < N)
                    C[batch * cb + int64_t(m) * N + n] = c[i][j] * scale + (residual ? residual[batch * rb + m * rs + n] : 0.f);
            }
    }
};

// scores = scale * AB^T + the pair's bias, from the table of all offsets (null: no bias)
struct BiasEpilogue {
    float* C;
    int n;
    float scale;
    const float* table;
    int64_t table_stride;
    const int4* tile_num;
    int count;
    __device__ void operator()(float (&c)[8][8], int batch, int m0, int n0, int tm, int tn) const {
        for (int i = 0; i < 8; ++i)
            for (int j = 0; j < 8; ++j) {
                const int m = m0 + tm + i, k = n0 + tn + j;
                if (m >= n || k >= n) continue;
                float b = 0.f;
                if (table) {
                    const int4 q = tile_num[m], p = tile_num[k];
                    b = table[batch * table_stride + (p.x != q.x ? count + (p.x > q.x) : p.y + q.z)];
                }
                C[(int64_t(batch) * n + m) * n + k] = c[i][j] * scale + b;
            }
    }
};

}  // namespace train
}  // namespace veda
