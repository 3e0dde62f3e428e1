// Grouped products with ragged row groups and their weight gradient
// (moe_grouped_gemm, moe_grouped_gemm_wgrad in moe.h).
#include "device.hpp"
#include "ops_launch.hpp"
#include "simple_tile.hpp"

namespace moe {
namespace {

// Rows [begin, end) of group g, kept inside [0, R] whatever the offsets hold.
struct Rows {
  int64_t begin, end;
};
__device__ __forceinline__ Rows group_rows(const int32_t* offsets, int g, int R) {
  const int b = min(max(offsets[g], 0), R);
  return {b, max(b, min(offsets[g + 1], R))};
}

__device__ __forceinline__ float e4m3_value(uint8_t c) {
  return __builtin_amdgcn_cvt_f32_fp8((int)c, 0);
}

struct GemmArgs {
  const bf16_t* x;
  const int32_t* offsets;
  const void* w;
  const float* w_scale;
  void* y;
  int R, G, N, K, fp8, kn, out_bf16;
};

// block (n-tile, m-tile): the m-tiles of 64 rows are numbered group by group
__global__ __launch_bounds__(256) void moe_grouped_gemm_kernel(GemmArgs p) {
  int64_t t = blockIdx.y;
  for (int g = 0; g < p.G; ++g) {
    const Rows r = group_rows(p.offsets, g, p.R);
    const int64_t tiles = (r.end - r.begin + 63) / 64;
    if (t >= tiles) {
      t -= tiles;
      continue;
    }
    const int64_t K = p.K, N = p.N;
    const bf16_t* wb = static_cast<const bf16_t*>(p.w) + (int64_t)g * N * K;
    const uint8_t* w8 = static_cast<const uint8_t*>(p.w) + (int64_t)g * N * K;
    auto a = [&](int64_t m, int64_t k) { return bf16_to_f32(p.x[(r.begin + m) * K + k]); };
    auto b = [&](int64_t n, int64_t k) {
      return p.fp8 ? e4m3_value(w8[n * K + k]) : bf16_to_f32(p.kn ? wb[k * N + n] : wb[n * K + k]);
    };
    auto store = [&](int64_t m, int64_t n, float v) {
      if (p.fp8) v *= p.w_scale[(int64_t)g * N + n];
      const int64_t at = (r.begin + m) * N + n;
      if (p.out_bf16)
        static_cast<bf16_t*>(p.y)[at] = f32_to_bf16(v);
      else
        static_cast<float*>(p.y)[at] = v;
    };
    simple_tile(a, b, store, r.end - r.begin, N, K, t * 64, (int64_t)blockIdx.x * 64);
    return;
  }
}

// block (k-tile, n-tile, group)
__global__ __launch_bounds__(256) void moe_grouped_wgrad_kernel(const bf16_t* dy, const bf16_t* x,
                                                                const int32_t* offsets, float* dw,
                                                                int R, int N, int K) {
  const int g = blockIdx.z;
  const Rows r = group_rows(offsets, g, R);
  auto a = [&](int64_t n, int64_t t) { return bf16_to_f32(dy[(r.begin + t) * N + n]); };
  auto b = [&](int64_t k, int64_t t) { return bf16_to_f32(x[(r.begin + t) * K + k]); };
  auto store = [&](int64_t n, int64_t k, float v) { dw[((int64_t)g * N + n) * K + k] = v; };
  simple_tile(a, b, store, N, K, r.end - r.begin, (int64_t)blockIdx.y * 64, (int64_t)blockIdx.x * 64);
}

}  // namespace

hipError_t launch_grouped_gemm(const moe_gemm_shape& s, const GemmPlan&, const void* x,
                               const int32_t* offsets, const void* w, const float* w_scale, void* y,
                               void*, hipStream_t st) {
  const GemmArgs p{static_cast<const bf16_t*>(x), offsets, w, w_scale, y, s.R, s.G, s.N, s.K,
                   s.weight_format == MOE_WEIGHTS_FP8_E4M3, s.weight_layout == MOE_LAYOUT_KN,
                   s.out_dtype == MOE_DTYPE_BF16};
  const unsigned mt = (unsigned)(s.R / 64 + s.G);
  hipLaunchKernelGGL(moe_grouped_gemm_kernel, dim3((unsigned)((s.N + 63) / 64), mt), dim3(256), 0, st, p);
  return hipGetLastError();
}

hipError_t launch_grouped_wgrad(const moe_gemm_shape& s, const void* dy, const void* x,
                                const int32_t* offsets, float* dw, hipStream_t st) {
  const dim3 grid((unsigned)((s.K + 63) / 64), (unsigned)((s.N + 63) / 64), (unsigned)s.G);
  hipLaunchKernelGGL(moe_grouped_wgrad_kernel, grid, dim3(256), 0, st, static_cast<const bf16_t*>(dy),
                     static_cast<const bf16_t*>(x), offsets, dw, s.R, s.N, s.K);
  return hipGetLastError();
}

}  // namespace moe
