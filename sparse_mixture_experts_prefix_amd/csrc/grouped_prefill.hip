// Grouped products and weight gradients with ragged groups of many rows: the
// 256 x 256 x 64 tiles of gemm_tile.hpp on rows as they are (see grouped.hip).
#include "gemm_tile.hpp"
#include "ops_launch.hpp"
#include "ragged.hpp"

namespace moe {
namespace {

// The output type fixed at compile time: with both epilogues in one kernel the
// folding K loop spilled 16 registers.
template <bool OUT16>
struct TypedGemm : RaggedGemm {
  static constexpr int out16 = OUT16;
};

// KT: K may end inside a 64-wide K stage (see prefill_tile)
template <bool FP8, bool KT, bool OUT16>
__global__ __launch_bounds__(256) void moe_grouped_prefill_kernel(TypedGemm<OUT16> p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  prefill_tile<false, FP8, false, KT>(p, lds);
}

template <bool OUT16>
__global__ __launch_bounds__(256) void moe_grouped_kmajor_prefill_kernel(TypedGemm<OUT16> p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  prefill_tile<false, false, true>(p, lds);
}

// FOLD: the product's kernel folds short last m-tiles (bf16 [N][K] weights)
template <bool FOLD>
__global__ __launch_bounds__(256) void moe_grouped_fixup_kernel(RaggedGemm p) {
  fixup_tiles<false, FOLD>(p);
}

template <bool OUT16>
hipError_t launch_tiles(void (*kernel)(TypedGemm<OUT16>), const RaggedGemm& g, int64_t blocks,
                        std::atomic<uint64_t>& done, hipStream_t s) {
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), kLdsBytes, done);
  if (e != hipSuccess) return e;
  TypedGemm<OUT16> p;
  static_cast<RaggedGemm&>(p) = g;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), kLdsBytes, s, p);
  return hipGetLastError();
}

template <bool OUT16>
hipError_t launch_typed(const RaggedGemm& p, bool fp8, bool kn, int64_t blocks, hipStream_t s) {
  static std::atomic<uint64_t> done[5];
  const bool kt = p.K_routed % BK != 0;
  if (kn) return launch_tiles<OUT16>(moe_grouped_kmajor_prefill_kernel<OUT16>, p, blocks, done[0], s);
  if (fp8)
    return kt ? launch_tiles<OUT16>(moe_grouped_prefill_kernel<true, true, OUT16>, p, blocks, done[1], s)
              : launch_tiles<OUT16>(moe_grouped_prefill_kernel<true, false, OUT16>, p, blocks, done[2], s);
  return kt ? launch_tiles<OUT16>(moe_grouped_prefill_kernel<false, true, OUT16>, p, blocks, done[3], s)
            : launch_tiles<OUT16>(moe_grouped_prefill_kernel<false, false, OUT16>, p, blocks, done[4], s);
}

}  // namespace

hipError_t launch_grouped_prefill(RaggedGemm p, bool fp8, bool kn, int64_t mtiles, hipStream_t s) {
  p.n_tiles_n = (p.N_routed + BN - 1) / BN;
  // enough workgroups for every XCD's run plus the pieces of a cut last round
  const int64_t blocks = (mtiles * p.n_tiles_n + 7) / 8 * 8 + p.ctas;
  const hipError_t e = p.out16 ? launch_typed<true>(p, fp8, kn, blocks, s) : launch_typed<false>(p, fp8, kn, blocks, s);
  if (e != hipSuccess || p.ctas <= 0) return e;
  const unsigned fix = (unsigned)p.ctas * kFixBlocksPerTile;
  if (kn || fp8)
    hipLaunchKernelGGL(moe_grouped_fixup_kernel<false>, dim3(fix), dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL(moe_grouped_fixup_kernel<true>, dim3(fix), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace moe
