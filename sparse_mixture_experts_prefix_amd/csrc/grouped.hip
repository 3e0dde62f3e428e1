// Grouped products with ragged row groups and their weight gradient
// (moe_grouped_gemm, moe_grouped_gemm_wgrad in moe.h).
//
// The tile kernels are the layer's: 256 x 256 x 64 tiles for many rows per
// group (gemm_tile.hpp), weight-streaming tiles of 16 or 32 rows for few
// (gemm_decode_tile.hpp), here on rows as they are: no padding, no align
// step, one launch (two when the last round of tiles is cut along K).  Every
// wave numbers the m-tiles from the group offsets itself.
#include "device.hpp"
#include "gemm_decode_tile.hpp"
#include "launch.hpp"
#include "ops_launch.hpp"
#include "ragged.hpp"

namespace moe {
namespace {

// M-tile m (of BMD rows) of a few-row call: a wave's lanes hold GPL groups
// each, add their tile counts up and pick the group that holds tile m.
template <int BMD, int GPL>
__device__ __forceinline__ bool find_mtile(const RaggedGemm& p, int64_t m, DecodeRows& r) {
  const int lane = threadIdx.x & 63;
  int cnt[GPL], first[GPL], tot = 0;
#pragma unroll
  for (int q = 0; q < GPL; ++q) {
    const int g = lane * GPL + q;
    cnt[q] = g < p.E ? group_rows(p, g) : 0;
    first[q] = g < p.E ? group_first(p, g) : 0;
    tot += (cnt[q] + BMD - 1) / BMD;
  }
  int incl = tot;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(incl, off);
    if (lane >= off) incl += y;
  }
  int run = incl - tot, g = -1, row0 = 0, valid = 0;
#pragma unroll
  for (int q = 0; q < GPL; ++q) {
    const int t = (cnt[q] + BMD - 1) / BMD;
    if (m >= run && m < run + t) {
      const int j = (int)m - run;
      g = lane * GPL + q;
      row0 = first[q] + j * BMD;
      valid = min(BMD, cnt[q] - j * BMD);
    }
    run += t;
  }
  const uint64_t hit = __ballot(g >= 0);
  if (!hit) return false;
  const int src = (int)__builtin_ctzll(hit);
  r.g = __builtin_amdgcn_readlane(g, src);
  r.row0 = __builtin_amdgcn_readlane(row0, src);
  r.valid = __builtin_amdgcn_readlane(valid, src);
  return true;
}

template <int BMD>
__device__ __forceinline__ bool decode_rows(const RaggedGemm& p, int64_t m, DecodeRows& r) {
  return p.E <= 64 ? find_mtile<BMD, 1>(p, m, r) : find_mtile<BMD, 5>(p, m, r);
}
template <int BMD>
__device__ __forceinline__ int decode_valid(const RaggedGemm&, const DecodeRows& r) {
  return r.valid;
}

template <int MT, int NG>
__global__ __launch_bounds__(kKw * 64) void moe_grouped_decode_kernel(RaggedGemm p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  decode_tile_staged<MT, false, false, NG>(p, lds);
}

template <int MT>
__global__ __launch_bounds__(kKw * 64) void moe_grouped_kmajor_decode_kernel(RaggedGemm p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  decode_tile_staged<MT, true, false>(p, lds);
}

template <int MT, bool NARROW>
__global__ __launch_bounds__(kKw * 64) void moe_grouped_e4m3_decode_kernel(RaggedGemm p) {
  decode_tile<false, MT, ng_down<true, NARROW>(), kKw, unroll<true>(), true>(p);
}

// columns: output columns per tile; lds: dynamic bytes
template <class Kernel>
hipError_t launch_columns(Kernel kernel, RaggedGemm p, int64_t mtiles, int columns, int lds,
                          std::atomic<uint64_t>& done, hipStream_t s) {
  if (lds > 0) {
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), lds, done);
    if (e != hipSuccess) return e;
  }
  p.n_tiles_n = (p.N_routed + columns - 1) / columns;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(mtiles * p.n_tiles_n)), dim3(kKw * 64), lds, s, p);
  return hipGetLastError();
}

// Few rows per group: BM = 16 MT rows per tile.  Column tiles as the layer's
// (64 columns, or 16 when few row tiles would leave CUs idle; K-major stages
// are always 64 columns wide).
template <int MT>
hipError_t launch_decode(const RaggedGemm& p, bool fp8, bool kn, int64_t mtiles, hipStream_t s) {
  static std::atomic<uint64_t> done[5];
  const int64_t rows = (p.R + 16 * MT - 1) / (16 * MT), groups = p.E < p.R ? p.E : p.R;
  const int64_t busy = rows > groups ? rows : groups;  // row tiles that can hold rows, about
  const bool narrow = busy * ((p.N_routed + 63) / 64) < kFillBlocks;
  if (fp8)
    return narrow ? launch_columns(moe_grouped_e4m3_decode_kernel<MT, true>, p, mtiles, 16, 0, done[0], s)
                  : launch_columns(moe_grouped_e4m3_decode_kernel<MT, false>, p, mtiles, 64, 0, done[1], s);
  if (kn)
    return launch_columns(moe_grouped_kmajor_decode_kernel<MT>, p, mtiles, 64, km_lds_bytes<MT>(), done[2], s);
  if (narrow)
    return launch_columns(moe_grouped_decode_kernel<MT, kNgDownNarrow>, p, mtiles, 16 * kNgDownNarrow,
                          km_lds_bytes<MT, kNgDownNarrow>(), done[3], s);
  return launch_columns(moe_grouped_decode_kernel<MT, 4>, p, mtiles, 64, km_lds_bytes<MT, 4>(), done[4], s);
}

}  // namespace

hipError_t launch_grouped_gemm(const moe_gemm_shape& s, const GemmPlan& plan, const void* x,
                               const int32_t* offsets, const void* w, const float* w_scale, void* y,
                               void* ws, hipStream_t st) {
  const bool fp8 = s.weight_format == MOE_WEIGHTS_FP8_E4M3, kn = s.weight_layout == MOE_LAYOUT_KN;
  RaggedGemm p{};
  p.A = static_cast<const uint16_t*>(x);
  p.lda = s.K;
  p.B_routed = w;
  p.S_routed = w_scale;
  p.E = s.G;
  p.N_routed = s.N;
  p.K_routed = s.K;
  p.offsets = offsets;
  p.R = s.R;
  p.C = y;
  p.ldc = s.N;
  p.out16 = s.out_dtype == MOE_DTYPE_BF16;
  // a y beyond the 256 MB Infinity Cache would only push the weights out of it (10007 x
  // 7168, 64 groups of width 2048: 478 -> 453 us); a smaller one may stay for its reader
  p.stream_out = (int64_t)s.R * s.N * 4 > (int64_t(256) << 20);
  // m-tiles that can hold rows: full ones and one ragged end per group
  int64_t mtiles = s.R / plan.BM + s.G;
  if (mtiles > s.R) mtiles = s.R;
  if (plan.BM == 16) return launch_decode<1>(p, fp8, kn, mtiles, st);
  if (plan.BM == 32) return launch_decode<2>(p, fp8, kn, mtiles, st);
  if (plan.split) {
    const hipError_t e = split_ctas(&p.ctas);
    if (e != hipSuccess) return e;
    p.partial = static_cast<float*>(ws);
  }
  return launch_grouped_prefill(p, fp8, kn, mtiles, st);
}

}  // namespace moe
