// Low-rank adapters of many requests beside one shared projection
// (moe_lora_forward, moe_lora_backward in moe.h).
#include "device.hpp"
#include "ops_launch.hpp"
#include "simple_tile.hpp"

namespace moe {
namespace {

struct LoraArgs {
  const bf16_t *x, *w, *a, *b;
  const int32_t* adapter;
  const float* scale;
  int T, D, N, L, r, out_bf16;
};

__device__ __forceinline__ bool has_adapter(const LoraArgs& p, int l) { return l >= 0 && l < p.L; }
__device__ __forceinline__ float scale_of(const LoraArgs& p, int l) { return p.scale ? p.scale[l] : 1.f; }

__device__ __forceinline__ void store_as(void* y, int64_t at, float v, int out_bf16) {
  if (out_bf16)
    static_cast<bf16_t*>(y)[at] = f32_to_bf16(v);
  else
    static_cast<float*>(y)[at] = v;
}

// xa[t] = A[a] x[t] (one wave per row and rank)
__global__ void moe_lora_shrink_kernel(LoraArgs p, float* xa) {
  const int64_t t = blockIdx.x;
  const int l = p.adapter[t], j = blockIdx.y;
  float s = 0.f;
  if (has_adapter(p, l)) {
    const bf16_t* a = p.a + ((int64_t)l * p.r + j) * p.D;
    for (int k = threadIdx.x; k < p.D; k += 64) s += bf16_to_f32(a[k]) * bf16_to_f32(p.x[t * p.D + k]);
    for (int off = 32; off; off >>= 1) s += __shfl_xor(s, off);
  }
  if (threadIdx.x == 0) xa[t * p.r + j] = s;
}

// u[t] = scale B[a]^T dy[t]
__global__ void moe_lora_shrink_back_kernel(LoraArgs p, const bf16_t* dy, float* u) {
  const int64_t t = blockIdx.x;
  const int l = p.adapter[t], j = blockIdx.y;
  float s = 0.f;
  if (has_adapter(p, l)) {
    const bf16_t* b = p.b + (int64_t)l * p.N * p.r + j;
    for (int n = threadIdx.x; n < p.N; n += 64)
      s += bf16_to_f32(b[(int64_t)n * p.r]) * bf16_to_f32(dy[t * p.N + n]);
    for (int off = 32; off; off >>= 1) s += __shfl_xor(s, off);
    s *= scale_of(p, l);
  }
  if (threadIdx.x == 0) u[t * p.r + j] = s;
}

__global__ __launch_bounds__(256) void moe_lora_forward_kernel(LoraArgs p, const float* xa, void* y) {
  auto a = [&](int64_t t, int64_t k) { return bf16_to_f32(p.x[t * p.D + k]); };
  auto b = [&](int64_t n, int64_t k) { return bf16_to_f32(p.w[n * p.D + k]); };
  auto store = [&](int64_t t, int64_t n, float v) {
    const int l = p.adapter[t];
    if (has_adapter(p, l)) {
      const bf16_t* bl = p.b + ((int64_t)l * p.N + n) * p.r;
      float s = 0.f;
      for (int j = 0; j < p.r; ++j) s += bf16_to_f32(bl[j]) * xa[t * p.r + j];
      v += scale_of(p, l) * s;
    }
    store_as(y, t * p.N + n, v, p.out_bf16);
  };
  simple_tile(a, b, store, p.T, p.N, p.D, (int64_t)blockIdx.y * 64, (int64_t)blockIdx.x * 64);
}

__global__ __launch_bounds__(256) void moe_lora_dx_kernel(LoraArgs p, const bf16_t* dy, const float* u,
                                                          void* dx) {
  auto a = [&](int64_t t, int64_t n) { return bf16_to_f32(dy[t * p.N + n]); };
  auto b = [&](int64_t d, int64_t n) { return bf16_to_f32(p.w[n * p.D + d]); };
  auto store = [&](int64_t t, int64_t d, float v) {
    const int l = p.adapter[t];
    if (has_adapter(p, l))
      for (int j = 0; j < p.r; ++j)
        v += bf16_to_f32(p.a[((int64_t)l * p.r + j) * p.D + d]) * u[t * p.r + j];
    store_as(dx, t * p.D + d, v, p.out_bf16);
  };
  simple_tile(a, b, store, p.T, p.D, p.N, (int64_t)blockIdx.y * 64, (int64_t)blockIdx.x * 64);
}

// out[l][j][c] (DB: out[l][c][j]) = sum over l's rows of v[t][j] * z[t][c] (DB: * scale)
template <bool DB>
__global__ void moe_lora_wgrad_kernel(LoraArgs p, const float* v, const bf16_t* z, int C, float* out) {
  const int l = blockIdx.z, j = blockIdx.y;
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= C) return;
  float s = 0.f;
  for (int64_t t = 0; t < p.T; ++t)
    if (p.adapter[t] == l) s += v[t * p.r + j] * bf16_to_f32(z[t * C + c]);
  if (DB)
    out[((int64_t)l * C + c) * p.r + j] = s * scale_of(p, l);
  else
    out[((int64_t)l * p.r + j) * C + c] = s;
}

LoraArgs args_of(const moe_lora_shape& s, const moe_lora_tensors& t) {
  return {static_cast<const bf16_t*>(t.x), static_cast<const bf16_t*>(t.w),
          static_cast<const bf16_t*>(t.lora_a), static_cast<const bf16_t*>(t.lora_b), t.adapter, t.scale,
          s.T, s.D, s.N, s.L, s.r, s.out_dtype == MOE_DTYPE_BF16};
}

}  // namespace

hipError_t launch_lora_forward(const moe_lora_shape& s, const LoraPlan& p, const moe_lora_tensors& t,
                               void* y, float* xa, void* ws, hipStream_t st) {
  const LoraArgs a = args_of(s, t);
  if (!xa) xa = reinterpret_cast<float*>(static_cast<char*>(ws) + p.off_xa);
  hipLaunchKernelGGL(moe_lora_shrink_kernel, dim3(s.T, s.r), dim3(64), 0, st, a, xa);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(moe_lora_forward_kernel, dim3((s.N + 63) / 64, (s.T + 63) / 64), dim3(256), 0, st, a,
                     static_cast<const float*>(xa), y);
  return hipGetLastError();
}

hipError_t launch_lora_backward(const moe_lora_shape& s, const LoraBwdPlan& p,
                                const moe_lora_tensors& t, const void* dy, const float* xa,
                                const moe_lora_grads& g, void* ws, hipStream_t st) {
  const LoraArgs a = args_of(s, t);
  const bf16_t* d = static_cast<const bf16_t*>(dy);
  float* u = reinterpret_cast<float*>(static_cast<char*>(ws) + p.off_u);
  hipLaunchKernelGGL(moe_lora_shrink_back_kernel, dim3(s.T, s.r), dim3(64), 0, st, a, d, u);
  hipLaunchKernelGGL(moe_lora_dx_kernel, dim3((s.D + 63) / 64, (s.T + 63) / 64), dim3(256), 0, st, a, d,
                     static_cast<const float*>(u), g.dx);
  hipLaunchKernelGGL(moe_lora_wgrad_kernel<false>, dim3((s.D + 255) / 256, s.r, s.L), dim3(256), 0, st, a,
                     static_cast<const float*>(u), a.x, s.D, g.da);
  hipLaunchKernelGGL(moe_lora_wgrad_kernel<true>, dim3((s.N + 255) / 256, s.r, s.L), dim3(256), 0, st, a,
                     xa, d, s.N, g.db);
  return hipGetLastError();
}

}  // namespace moe
