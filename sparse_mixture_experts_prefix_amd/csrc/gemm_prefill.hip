// Prefill-sized grouped GEMMs (many rows per expert): 256 x 256 x 64 tiles.
//
// Same operation as the decode kernels in gemm_decode.hip (SwiGLU expert FFN of the
// glossary "MoE (Mixture of Experts - Mezcla de Expertos)", section 3 step 3;
// packed [E, 2F, D] gate/up tensor of "Transformers v5 El Secreto Detrás de
// los Modelos MoE Más Rápidos", section "La Solución: WeightConverter"), laid
// out for CDNA4:
//  - 4 wavefronts, each owning 128 x 128 outputs as 4 x 4 MFMA 32x32x16
//    tiles (256 fp32 accumulators per lane; in a partly filled tile its 4 row
//    blocks of 32 alternate with the other wave row's), so every 16-byte LDS
//    read feeds four MFMAs.
//  - Operands go HBM/L2 -> LDS with buffer_load ... lds (no registers, no
//    ds_write); A is double- and B triple-buffered, and a wave's loads of a
//    stage are spread evenly over the MFMA substeps (see k_loop).
//    Out-of-range buffer offsets read as zero, which handles padding rows,
//    gathered rows of -1 and N/K tails with no branches.
//  - LDS rows are 128 B (64 bf16 of K); the eight 16-byte chunks of row r are
//    stored XOR-swizzled by (r & 7) ^ ((r >> 3) & 1), which keeps both 8- and
//    16-lane phases of the b128 operand reads on distinct banks.
//  - The valid tiles are split into 8 equal runs, one per XCD (the hardware
//    deals workgroups to the 8 XCDs round-robin), each walked in blocks of
//    up to 4 m-tiles of one expert x 8 n-tiles, so the workgroups an XCD runs
//    together share their A and B tiles in its L2 and no XCD gets more tiles
//    than another.
//  - MFMA work of 32-row sub-tiles that hold only padding rows is skipped.
//  - A short, partial last round of tiles is cut along K (see split_of).
//  - A group's last m-tile of at most 32 rows is not a tile of its own: the
//    m-tile before it computes those rows too, with their A fragments loaded
//    straight into registers (see tile_rows and k_loop's XR).
//  - E4M3 weights (one fp32 scale per weight row): a B stage holds the codes,
//    64-byte rows of four 16-byte chunks swizzled by (r >> 1) & 3; a lane's
//    16-byte read carries its weights of two k-substeps (K is permuted the
//    same way for A), widened to bf16 exactly in registers, and each output
//    column is multiplied by its row's scale before the epilogue.  Half the
//    weight bytes and half the B loads of bf16, for the same MFMAs.
#include "gemm_tile.hpp"

namespace moe {
namespace {

template <bool FP8, bool KT, bool NTB>
__global__ __launch_bounds__(256) void moe_gemm_gate_up_prefill_kernel(GroupedGemm p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  prefill_tile<true, FP8, false, KT, NTB>(p, lds);
}

template <bool FP8, bool KT>
__global__ __launch_bounds__(256) void moe_gemm_down_prefill_kernel(GroupedGemm p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  prefill_tile<false, FP8, false, KT>(p, lds);
}

// rows x weight with the weight stored K-major ([K][N] per group): the
// backward pass's products with W_down and W_gate_up read in their own layout
__global__ __launch_bounds__(256) void moe_gemm_rows_kmajor_prefill_kernel(GroupedGemm p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  prefill_tile<false, false, true>(p, lds);
}

template <bool GATE_UP>
__global__ __launch_bounds__(256) void moe_gemm_split_fixup_kernel(GroupedGemm p) {
  if (p.b_kmajor || p.fp8)
    fixup_tiles<GATE_UP, false>(p);  // the K-major and E4M3 kernels' m-tiles do not fold
  else
    fixup_tiles<GATE_UP, true>(p);
}

template <bool FP8, bool KT>
hipError_t launch_fmt(bool gate_up, GroupedGemm g, hipStream_t s) {
  constexpr int lds = lds_bytes<FP8>();
  // set once per process (a function-local static is initialised thread-safely)
  static const hipError_t attr = [] {
    hipError_t e = hipFuncSetAttribute((const void*)moe_gemm_gate_up_prefill_kernel<FP8, KT, false>,
                                       hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e == hipSuccess)
      e = hipFuncSetAttribute((const void*)moe_gemm_gate_up_prefill_kernel<FP8, KT, true>,
                              hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e == hipSuccess)
      e = hipFuncSetAttribute((const void*)moe_gemm_down_prefill_kernel<FP8, KT>,
                              hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e == hipSuccess && !FP8)
      e = hipFuncSetAttribute((const void*)moe_gemm_rows_kmajor_prefill_kernel,
                              hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    return e;
  }();
  if (attr != hipSuccess) return attr;
  const int nmax = g.N_routed > g.N_shared ? g.N_routed : g.N_shared;
  const int NB = gate_up ? BN / 2 : BN;
  g.n_tiles_n = (nmax + NB - 1) / NB;
  // No split (and no second kernel) when the device could never choose one:
  // too many tiles for any routing, or K too short to cut.  With ids outside
  // [0, E) the bound may overstate the tiles; that only forgoes the split.
  {
    const int kmin = g.B_shared && g.K_shared < g.K_routed ? g.K_shared : g.K_routed;
    const bool short_k = ((kmin + BK - 1) / BK) / kMinPieceStages < 2;
    if (short_k || g.min_tiles * g.n_tiles_n >= (int64_t)kSplitRounds * g.ctas) g.ctas = 0;
  }
  // enough workgroups for every XCD's run plus the pieces of a split last
  // round (at most ctas of them; see prefill_tile)
  const int64_t blocks = (g.max_tiles * g.n_tiles_n + 7) / 8 * 8 + (g.ctas > 0 ? g.ctas : 0);
  if (blocks == 0) return hipSuccess;
  if (gate_up && g.stream_b)
    hipLaunchKernelGGL((moe_gemm_gate_up_prefill_kernel<FP8, KT, true>), dim3((unsigned)blocks),
                       dim3(256), lds, s, g);
  else if (gate_up)
    hipLaunchKernelGGL((moe_gemm_gate_up_prefill_kernel<FP8, KT, false>), dim3((unsigned)blocks),
                       dim3(256), lds, s, g);
  else if (g.b_kmajor)
    hipLaunchKernelGGL(moe_gemm_rows_kmajor_prefill_kernel, dim3((unsigned)blocks), dim3(256), lds,
                       s, g);
  else
    hipLaunchKernelGGL((moe_gemm_down_prefill_kernel<FP8, KT>), dim3((unsigned)blocks), dim3(256), lds,
                       s, g);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || g.ctas <= 0) return e;
  const unsigned fix_blocks = (unsigned)g.ctas * kFixBlocksPerTile;
  if (gate_up)
    hipLaunchKernelGGL(moe_gemm_split_fixup_kernel<true>, dim3(fix_blocks), dim3(256), 0, s, g);
  else
    hipLaunchKernelGGL(moe_gemm_split_fixup_kernel<false>, dim3(fix_blocks), dim3(256), 0, s, g);
  return hipGetLastError();
}

hipError_t launch(bool gate_up, const GroupedGemm& g, hipStream_t s) {
  if (g.b_kmajor && (gate_up || g.fp8)) return hipErrorInvalidValue;  // no such variant
  // a K of some group that ends inside a 64-wide K-stage needs the masked loads
  const bool kt = g.K_routed % BK != 0 || (g.B_shared && g.K_shared % BK != 0);
  if (g.fp8)
    return kt ? launch_fmt<true, true>(gate_up, g, s) : launch_fmt<true, false>(gate_up, g, s);
  return kt ? launch_fmt<false, true>(gate_up, g, s) : launch_fmt<false, false>(gate_up, g, s);
}

// ------------------------------------------------------------ weight gradients
__global__ __launch_bounds__(256) void moe_gemm_wgrad_kernel(WgradGemm p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  wgrad_whole_tile<false>(p, blockIdx.x, lds, NoHook{});
}

// The same products when every group has at most 64 rows (a token picks an
// expert once, so T <= 64 guarantees it): one K stage per tile.  With 256
// accumulators per lane a CU runs one workgroup, which would wait for each
// tile's loads with nothing else to do; here a workgroup walks tiles
// blockIdx.x, + gridDim.x, ... and issues the next tile's stage into the other
// LDS buffer before storing the current tile, so the loads fly under the
// stores.
__global__ __launch_bounds__(256) void moe_gemm_wgrad_one_stage_kernel(WgradGemm p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int64_t total = (int64_t)p.G * p.tiles_m * p.tiles_n;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  auto no_issue = [](int, int, int, int) {};
  f32x16 acc[4][4];
  int64_t t = blockIdx.x;
  int buf = 0;
  if (t < total) {
    const WgradTile w = wgrad_tile(p, t);
    if (w.valid && w.K > 0) {
      wgrad_issue(p, w, lds, false, 0, 0, 0, 8, wave, lane);
      wgrad_issue(p, w, lds, true, 0, 0, 0, 8, wave, lane);
    }
  }
  for (; t < total; t += gridDim.x) {
    const WgradTile w = wgrad_tile(p, t);
    zero_acc(acc);
    if (w.valid && w.K > 0)  // its stage is in buffer buf (issued one tile earlier)
      k_loop<false, 4, false, decltype(no_issue), decltype(no_issue), true, true, true>(
          lds + buf * kABytes, 0, 1, wm, wn, false, lane, no_issue, no_issue, acc);
    // every wave is done reading this tile's stage (and the one before, in
    // the other buffer) before the next tile's loads go there
    __syncthreads();
    const int64_t tn = t + gridDim.x;
    if (tn < total) {
      const WgradTile wn_ = wgrad_tile(p, tn);
      if (wn_.valid && wn_.K > 0) {
        wgrad_issue(p, wn_, lds, false, 0, buf ^ 1, 0, 8, wave, lane);
        wgrad_issue(p, wn_, lds, true, 0, buf ^ 1, 0, 8, wave, lane);
      }
    }
    if (w.valid) wgrad_store<false>(w, wm, wn, lane, acc);
    buf ^= 1;
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // no load may still be writing LDS at exit
}

}  // namespace

hipError_t launch_gemm_wgrad(const WgradGemm& g, hipStream_t s) {
  static const hipError_t attr = hipFuncSetAttribute(
      (const void*)moe_gemm_wgrad_kernel, hipFuncAttributeMaxDynamicSharedMemorySize, kLdsBytes);
  if (attr != hipSuccess) return attr;
  static const hipError_t attr1 =
      hipFuncSetAttribute((const void*)moe_gemm_wgrad_one_stage_kernel,
                          hipFuncAttributeMaxDynamicSharedMemorySize, kLdsBytes);
  if (attr1 != hipSuccess) return attr1;
  const int64_t blocks = (int64_t)g.G * g.tiles_m * g.tiles_n;
  if (blocks == 0) return hipSuccess;
  if (g.one_stage_ctas > 0) {
    const int64_t grid = blocks < g.one_stage_ctas ? blocks : g.one_stage_ctas;
    hipLaunchKernelGGL(moe_gemm_wgrad_one_stage_kernel, dim3((unsigned)grid), dim3(256), kLdsBytes, s,
                       g);
  } else {
    hipLaunchKernelGGL(moe_gemm_wgrad_kernel, dim3((unsigned)blocks), dim3(256), kLdsBytes, s, g);
  }
  return hipGetLastError();
}

hipError_t launch_gemm_gate_up_prefill(const GroupedGemm& g, hipStream_t s) {
  return launch(true, g, s);
}

hipError_t launch_gemm_down_prefill(const GroupedGemm& g, hipStream_t s) {
  return launch(false, g, s);
}

}  // namespace moe
