// Weight gradients of the grouped products with ragged groups
// (moe_grouped_gemm_wgrad in moe.h): dW[g][n][k] = sum over the group's rows of
// dy[r][n] x[r][k], on the K loop of gemm_tile.hpp with both operands read
// K-major (the rows are the reduction) through the transposing LDS reads.
#include "gemm_tile.hpp"
#include "ops_launch.hpp"
#include "ragged.hpp"

namespace moe {
namespace {

__global__ __launch_bounds__(256) void moe_grouped_wgrad_kernel(RaggedWgrad p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  wgrad_whole_tile(p, blockIdx.x, lds);
}

}  // namespace

hipError_t launch_grouped_wgrad(const moe_gemm_shape& s, const void* dy, const void* x,
                                const int32_t* offsets, float* dw, hipStream_t st) {
  static std::atomic<uint64_t> done;
  const hipError_t e =
      allow_lds(reinterpret_cast<const void*>(moe_grouped_wgrad_kernel), kLdsBytes, done);
  if (e != hipSuccess) return e;
  RaggedWgrad p{static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(x), s.N, s.K, s.N, s.K,
                s.G, offsets, s.R, dw, (s.N + BM - 1) / BM, (s.K + BN - 1) / BN};
  hipLaunchKernelGGL(moe_grouped_wgrad_kernel, dim3((unsigned)(s.G * p.tiles_m * p.tiles_n)), dim3(256),
                     kLdsBytes, st, p);
  return hipGetLastError();
}

}  // namespace moe
