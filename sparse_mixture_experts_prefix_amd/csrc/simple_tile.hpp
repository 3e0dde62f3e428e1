// A 64 x 64 output tile of C[m][n] = sum_k A(m, k) B(n, k) in fp32 on the
// vector units, for any operands that a callable can give by index: 256
// threads with 4 x 4 outputs each, K in steps of 16 through LDS.
#pragma once
#include "device.hpp"

namespace moe {

// a(m, k) for m < M, b(n, k) for n < N, k < K; store(m, n, sum) for the tile at (m0, n0)
template <class FA, class FB, class FC>
__device__ __forceinline__ void simple_tile(FA a, FB b, FC store, int64_t M, int64_t N, int64_t K,
                                            int64_t m0, int64_t n0) {
  __shared__ float sa[16][68], sb[16][68];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += 16) {
    __syncthreads();
    for (int e = tid; e < 1024; e += 256) {
      const int k = e & 15, i = e >> 4;
      sa[k][i] = (m0 + i < M && k0 + k < K) ? a(m0 + i, k0 + k) : 0.f;
      sb[k][i] = (n0 + i < N && k0 + k < K) ? b(n0 + i, k0 + k) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m < M && n < N) store(m, n, acc[i][j]);
    }
}

}  // namespace moe
