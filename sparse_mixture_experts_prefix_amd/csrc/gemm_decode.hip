// Decode-sized grouped GEMMs (a few rows per expert): weight streaming.
//
// Same operation as the prefill kernels (SwiGLU expert FFN of the glossary
// "MoE (Mixture of Experts - Mezcla de Expertos)", section 3 step 3; packed
// [E, 2F, D] gate/up tensor of "Transformers v5 El Secreto Detrás de los
// Modelos MoE Más Rápidos", section "La Solución: WeightConverter").  With
// 16-32 rows per expert every weight byte feeds only 16-32 MACs, so the time
// is the time to stream the touched experts' weights from HBM (the pages'
// "decode time follows active bytes over bandwidth", "Mixture of Experts
// optimiza Transformers y LLMs", section "¿Por qué MoEs importan ...").
//  - A workgroup owns one m-tile (16*MT rows of one expert) and 16*NG weight
//    rows (gate/up: NG/2 groups of gate rows with the matching up rows);
//    its 4 waves split K and their partial sums are added in LDS in a fixed
//    order (deterministic).  All loads of a trip are issued before its
//    MFMAs (a scheduling barrier), so each wave keeps two chunks in flight.
//  - MFMA 16x16x32 bf16.  The K order inside a chunk is permuted the same
//    way for A and B: lane (col c, group g) holds 128 / 4 bytes of weights of
//    its row (16 bf16 or 32 E4M3 values) for two or four consecutive MFMAs,
//    so the four lanes of a row read one full 128-byte line.  Weights go
//    straight from HBM to registers (each byte is used once); the loads of
//    several chunks are in flight per wave.
//  - Out-of-range buffer offsets read as zero: padding rows, rows past the
//    group's count and K tails need no branches.  Weight rows of tiles that
//    lie wholly in bounds are read with plain global loads instead (faster).
//  - E4M3 weights (one fp32 scale per weight row): a lane's 32 weights of a
//    chunk are two 16-byte loads, widened to bf16 exactly in registers
//    (v_cvt_scalef32_pk_bf16_fp8 with scale 1; every E4M3 value is a bf16
//    value), and each output column's sum is multiplied by its row's scale
//    after the reduction: sum_k x_k (q_k s) = s sum_k x_k q_k.  Half the
//    weight bytes of bf16, for the same MFMAs.
//  - bf16 weights with the wide column tiles, and the backward pass's
//    products with the weights as stored (contracting over their row index),
//    stage the weights through LDS instead; see the staged tile below.
#include "gemm_decode_tile.hpp"

namespace moe {
namespace {

template <int MT, bool FP8, bool NARROW>
__global__ __launch_bounds__(kKw * 64) void moe_gemm_gate_up_decode_kernel(GroupedGemm p) {
  decode_tile<true, MT, ng_gate_up<FP8, NARROW>(), kKw, unroll<FP8>(), FP8>(p);
}

template <int MT, bool FP8, bool NARROW>
__global__ __launch_bounds__(kKw * 64) void moe_gemm_down_decode_kernel(GroupedGemm p) {
  decode_tile<false, MT, ng_down<FP8, NARROW>(), kKw, unroll<FP8>(), FP8>(p);
}

template <bool FP8, bool NARROW>
int column_tile(bool gate_up) {
  return gate_up ? ng_gate_up<FP8, NARROW>() / 2 * 16 : ng_down<FP8, NARROW>() * 16;
}

template <int MT, bool FP8, bool NARROW>
hipError_t launch_mt(bool gate_up, GroupedGemm g, hipStream_t s) {
  const int nmax = g.N_routed > g.N_shared ? g.N_routed : g.N_shared;
  const int nout = column_tile<FP8, NARROW>(gate_up);
  g.n_tiles_n = (nmax + nout - 1) / nout;
  const int64_t blocks = g.max_tiles * g.n_tiles_n;
  if (blocks == 0) return hipSuccess;
  if (gate_up)
    hipLaunchKernelGGL((moe_gemm_gate_up_decode_kernel<MT, FP8, NARROW>), dim3((unsigned)blocks),
                       dim3(kKw * 64), 0, s, g);
  else
    hipLaunchKernelGGL((moe_gemm_down_decode_kernel<MT, FP8, NARROW>), dim3((unsigned)blocks),
                       dim3(kKw * 64), 0, s, g);
  return hipGetLastError();
}

template <int MT, bool GATE_UP, int NG>
hipError_t launch_staged(const GroupedGemm& g0, hipStream_t s);

template <int MT, bool FP8>
hipError_t launch_width(bool gate_up, const GroupedGemm& g, hipStream_t s) {
  const int nmax = g.N_routed > g.N_shared ? g.N_routed : g.N_shared;
  const int nout = column_tile<FP8, false>(gate_up);
  const bool narrow = g.busy_tiles * ((nmax + nout - 1) / nout) < kFillBlocks;
  // bf16 weights stream through LDS (narrow tiles: the register path's
  // column groups), E4M3 codes into registers
  if constexpr (!FP8) {
    if (narrow)
      return gate_up ? launch_staged<MT, true, kNgGateUpNarrow>(g, s)
                     : launch_staged<MT, false, kNgDownNarrow>(g, s);
    return gate_up ? launch_staged<MT, true, 4>(g, s) : launch_staged<MT, false, 4>(g, s);
  } else {
    if (narrow) return launch_mt<MT, FP8, true>(gate_up, g, s);
    return launch_mt<MT, FP8, false>(gate_up, g, s);
  }
}

template <int MT>
__global__ __launch_bounds__(kKw * 64) void moe_gemm_rows_kmajor_decode_kernel(GroupedGemm p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  decode_tile_staged<MT, true, false>(p, lds);
}

template <int MT, bool GATE_UP, int NG>
__global__ __launch_bounds__(kKw * 64) void moe_gemm_staged_decode_kernel(GroupedGemm p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  decode_tile_staged<MT, false, GATE_UP, NG>(p, lds);
}

// bf16 weights: the weights stream through LDS, NG column groups per tile
template <int MT, bool GATE_UP, int NG>
hipError_t launch_staged(const GroupedGemm& g0, hipStream_t s) {
  static const hipError_t attr =
      hipFuncSetAttribute((const void*)moe_gemm_staged_decode_kernel<MT, GATE_UP, NG>,
                          hipFuncAttributeMaxDynamicSharedMemorySize, km_lds_bytes<MT, NG>());
  if (attr != hipSuccess) return attr;
  const int64_t brows = GATE_UP ? 2 : 1;
  if (brows * g0.K_routed * g0.N_routed * 2 >= (int64_t(1) << 31) ||
      brows * g0.K_shared * g0.N_shared * 2 >= (int64_t(1) << 31))
    return hipErrorInvalidValue;
  GroupedGemm g = g0;
  const int nmax = g.N_routed > g.N_shared ? g.N_routed : g.N_shared;
  const int nout = GATE_UP ? 8 * NG : 16 * NG;
  g.n_tiles_n = (nmax + nout - 1) / nout;
  const int64_t blocks = g.max_tiles * g.n_tiles_n;
  if (blocks == 0) return hipSuccess;
  constexpr int lds = km_lds_bytes<MT, NG>();
  hipLaunchKernelGGL((moe_gemm_staged_decode_kernel<MT, GATE_UP, NG>), dim3((unsigned)blocks),
                     dim3(kKw * 64), lds, s, g);
  return hipGetLastError();
}

template <int MT>
hipError_t launch_kmajor(const GroupedGemm& g0, hipStream_t s) {
  static const hipError_t attr =
      hipFuncSetAttribute((const void*)moe_gemm_rows_kmajor_decode_kernel<MT>,
                          hipFuncAttributeMaxDynamicSharedMemorySize, km_lds_bytes<MT>());
  if (attr != hipSuccess) return attr;
  // a group's slab is addressed with 32-bit offsets
  if ((int64_t)g0.K_routed * g0.N_routed * 2 >= (int64_t(1) << 31) ||
      (int64_t)g0.K_shared * g0.N_shared * 2 >= (int64_t(1) << 31))
    return hipErrorInvalidValue;
  GroupedGemm g = g0;
  const int nmax = g.N_routed > g.N_shared ? g.N_routed : g.N_shared;
  g.n_tiles_n = (nmax + 63) / 64;
  const int64_t blocks = g.max_tiles * g.n_tiles_n;
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL((moe_gemm_rows_kmajor_decode_kernel<MT>), dim3((unsigned)blocks), dim3(kKw * 64),
                     km_lds_bytes<MT>(), s, g);
  return hipGetLastError();
}

template <int MT>
hipError_t launch_fmt(bool gate_up, const GroupedGemm& g, hipStream_t s) {
  return g.fp8 ? launch_width<MT, true>(gate_up, g, s) : launch_width<MT, false>(gate_up, g, s);
}

}  // namespace

hipError_t launch_gemm_gate_up_decode(const GroupedGemm& g, hipStream_t s) {
  if (g.b_kmajor) return hipErrorInvalidValue;
  if (g.BM == 16) return launch_fmt<1>(true, g, s);
  if (g.BM == 32) return launch_fmt<2>(true, g, s);
  return hipErrorInvalidValue;
}

hipError_t launch_gemm_down_decode(const GroupedGemm& g, hipStream_t s) {
  if (g.b_kmajor) {
    if (g.fp8) return hipErrorInvalidValue;  // K-major weights: bf16 only
    if (g.BM == 16) return launch_kmajor<1>(g, s);
    if (g.BM == 32) return launch_kmajor<2>(g, s);
    return hipErrorInvalidValue;
  }
  if (g.BM == 16) return launch_fmt<1>(false, g, s);
  if (g.BM == 32) return launch_fmt<2>(false, g, s);
  return hipErrorInvalidValue;
}

}  // namespace moe
