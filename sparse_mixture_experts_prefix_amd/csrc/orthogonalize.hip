// Orthogonalised updates by Newton-Schulz products (moe_orthogonalize in moe.h).
#include "device.hpp"
#include "ops_launch.hpp"
#include "simple_tile.hpp"

namespace moe {
namespace {

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;

__device__ __forceinline__ float g_at(const void* g, int dtype, int64_t i) {
  return dtype == MOE_DTYPE_F32 ? static_cast<const float*>(g)[i]
                                : bf16_to_f32(static_cast<const bf16_t*>(g)[i]);
}

// norm[e] = |G_e|_F, summed in double so that no gradient's squares under- or overflow
__global__ __launch_bounds__(256) void moe_orth_norm_kernel(const void* g, int dtype, int64_t mn, float* norm) {
  __shared__ double sum[256];
  const int64_t base = blockIdx.x * mn;
  double s = 0;
  for (int64_t i = threadIdx.x; i < mn; i += 256) {
    const double v = g_at(g, dtype, base + i);
    s += v * v;
  }
  sum[threadIdx.x] = s;
  __syncthreads();
  for (int o = 128; o; o >>= 1) {
    if (threadIdx.x < o) sum[threadIdx.x] += sum[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) norm[blockIdx.x] = (float)sqrt(sum[0]);
}

__global__ void moe_orth_scale_kernel(const void* g, int dtype, int64_t mn, const float* norm, float eps, float* x) {
  const int64_t e = blockIdx.y, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= mn) return;
  const float d = norm[e] + eps;
  x[e * mn + i] = d > 0.f ? g_at(g, dtype, e * mn + i) / d : 0.f;
}

// P = X X^T (tall: X^T X), one tile per block, z: matrix
__global__ __launch_bounds__(256) void moe_orth_gram_kernel(const float* x, float* p, int m, int n, int tall) {
  const float* X = x + (int64_t)blockIdx.z * m * n;
  float* P = p + (int64_t)blockIdx.z * m * m;
  auto a = [&](int64_t i, int64_t k) { return tall ? X[k * m + i] : X[i * n + k]; };
  auto st = [&](int64_t i, int64_t j, float v) { P[i * m + j] = v; };
  simple_tile(a, a, st, m, m, n, (int64_t)blockIdx.y * 64, (int64_t)blockIdx.x * 64);
}

// Q = b P + c P P
__global__ __launch_bounds__(256) void moe_orth_poly_kernel(const float* p, float* q, int m) {
  const float* P = p + (int64_t)blockIdx.z * m * m;
  float* Q = q + (int64_t)blockIdx.z * m * m;
  auto a = [&](int64_t i, int64_t k) { return P[i * m + k]; };
  auto st = [&](int64_t i, int64_t j, float v) { Q[i * m + j] = kB * P[i * m + j] + kC * v; };
  simple_tile(a, a, st, m, m, m, (int64_t)blockIdx.y * 64, (int64_t)blockIdx.x * 64);
}

// X' = a X + Q X (tall: a X + X Q)
__global__ __launch_bounds__(256) void moe_orth_apply_kernel(const float* x, const float* q, float* xo,
                                                             bf16_t* out, int m, int n, int tall) {
  const float* X = x + (int64_t)blockIdx.z * m * n;
  const float* Q = q + (int64_t)blockIdx.z * m * m;
  const int64_t rows = tall ? n : m, cols = tall ? m : n, at0 = (int64_t)blockIdx.z * m * n;
  auto a = [&](int64_t i, int64_t k) { return tall ? X[i * m + k] : Q[i * m + k]; };
  auto b = [&](int64_t j, int64_t k) { return tall ? Q[j * m + k] : X[k * n + j]; };
  auto st = [&](int64_t i, int64_t j, float v) {
    const int64_t at = i * cols + j;
    v += kA * X[at];
    if (out)
      out[at0 + at] = f32_to_bf16(v);
    else
      xo[at0 + at] = v;
  };
  simple_tile(a, b, st, rows, cols, m, (int64_t)blockIdx.y * 64, (int64_t)blockIdx.x * 64);
}

}  // namespace

hipError_t launch_orthogonalize(int E, int M, int N, const OrthPlan& p, const void* g, int g_dtype,
                                int steps, float eps, void* out, void* ws, hipStream_t st) {
  char* w = static_cast<char*>(ws);
  float* x[2] = {reinterpret_cast<float*>(w + p.off_x[0]), reinterpret_cast<float*>(w + p.off_x[1])};
  float* P = reinterpret_cast<float*>(w + p.off_p);
  float* Q = reinterpret_cast<float*>(w + p.off_q);
  float* norm = reinterpret_cast<float*>(w + p.off_norm);
  const int64_t mn = (int64_t)M * N;
  const unsigned tm = (p.m + 63) / 64;
  hipLaunchKernelGGL(moe_orth_norm_kernel, dim3(E), dim3(256), 0, st, g, g_dtype, mn, norm);
  hipLaunchKernelGGL(moe_orth_scale_kernel, dim3((unsigned)((mn + 255) / 256), E), dim3(256), 0, st, g,
                     g_dtype, mn, norm, eps, x[0]);
  for (int i = 0; i < steps; ++i) {
    hipLaunchKernelGGL(moe_orth_gram_kernel, dim3(tm, tm, E), dim3(256), 0, st, x[i & 1], P, p.m, p.n, p.tall);
    hipLaunchKernelGGL(moe_orth_poly_kernel, dim3(tm, tm, E), dim3(256), 0, st, P, Q, p.m);
    hipLaunchKernelGGL(moe_orth_apply_kernel, dim3((N + 63) / 64, (M + 63) / 64, E), dim3(256), 0, st,
                       x[i & 1], Q, x[~i & 1], i + 1 == steps ? static_cast<bf16_t*>(out) : nullptr, p.m,
                       p.n, p.tall);
  }
  return hipGetLastError();
}

}  // namespace moe
