// Grouped products and weight gradients with ragged groups of many rows: the
// 256 x 256 x 64 tiles of gemm_tile.hpp on rows as they are (see grouped.hip).
#include "gemm_tile.hpp"
#include "ops_launch.hpp"
#include "ragged.hpp"

namespace moe {
namespace {

// KT: K may end inside a 64-wide K stage (see prefill_tile)
template <bool FP8, bool KT>
__global__ __launch_bounds__(256) void moe_grouped_prefill_kernel(RaggedGemm p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  prefill_tile<false, FP8, false, KT>(p, lds);
}

__global__ __launch_bounds__(256) void moe_grouped_kmajor_prefill_kernel(RaggedGemm p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  prefill_tile<false, false, true>(p, lds);
}

// FOLD: the product's kernel folds short last m-tiles (bf16 [N][K] weights)
template <bool FOLD>
__global__ __launch_bounds__(256) void moe_grouped_fixup_kernel(RaggedGemm p) {
  fixup_tiles<false, FOLD>(p);
}

template <class Kernel>
hipError_t launch_tiles(Kernel kernel, const RaggedGemm& p, int64_t blocks, std::atomic<uint64_t>& done,
                        hipStream_t s) {
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), kLdsBytes, done);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), kLdsBytes, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_prefill(RaggedGemm p, bool fp8, bool kn, int64_t mtiles, hipStream_t s) {
  static std::atomic<uint64_t> done[5];
  p.n_tiles_n = (p.N_routed + BN - 1) / BN;
  const int64_t blocks = (mtiles * p.n_tiles_n + 7) / 8 * 8 + p.ctas;
  const bool kt = p.K_routed % BK != 0;
  hipError_t e;
  if (kn)
    e = launch_tiles(moe_grouped_kmajor_prefill_kernel, p, blocks, done[0], s);
  else if (fp8)
    e = kt ? launch_tiles(moe_grouped_prefill_kernel<true, true>, p, blocks, done[1], s)
           : launch_tiles(moe_grouped_prefill_kernel<true, false>, p, blocks, done[2], s);
  else
    e = kt ? launch_tiles(moe_grouped_prefill_kernel<false, true>, p, blocks, done[3], s)
           : launch_tiles(moe_grouped_prefill_kernel<false, false>, p, blocks, done[4], s);
  if (e != hipSuccess || p.ctas <= 0) return e;
  const unsigned fix = (unsigned)p.ctas * kFixBlocksPerTile;
  if (kn || fp8)
    hipLaunchKernelGGL(moe_grouped_fixup_kernel<false>, dim3(fix), dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL(moe_grouped_fixup_kernel<true>, dim3(fix), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace moe
