// Parameter blocks of the tile kernels for ragged row groups: groups follow
// each other without padding, their rows given by offsets on the device.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace moe {

// Rows [offsets[g], offsets[g + 1]) of group g, kept inside [0, R] whatever
// the offsets hold.
__device__ __forceinline__ int ragged_first(const int32_t* offsets, int g, int R) {
  return min(max(offsets[g], 0), R);
}
__device__ __forceinline__ int ragged_rows(const int32_t* offsets, int g, int R) {
  const int first = ragged_first(offsets, g, R);
  return max(first, min(offsets[g + 1], R)) - first;  // no difference of unclamped values: it could wrap
}

// C = A W[g]^T (or A W[g], K-major) over the groups' rows, for prefill_tile,
// decode_tile and decode_tile_staged (field names as GroupedGemm's).
struct RaggedGemm {
  static constexpr bool kRagged = true, kFold = true, kLora = false;
  static constexpr const int32_t* row_token = nullptr;  // rows are not gathered
  static constexpr int64_t a_bytes = 0, ld_gu = 0;
  static constexpr uint16_t* gu_out = nullptr;
  static constexpr const void* B_shared = nullptr;      // no shared expert
  static constexpr const float* S_shared = nullptr;
  static constexpr int N_shared = 0, K_shared = 0, BM = 256;
  const uint16_t* A;
  int64_t lda;
  const void* B_routed;
  const float* S_routed;
  int E, N_routed, K_routed;
  const int32_t* offsets;
  int R;
  void* C;
  int64_t ldc;
  int out16;       // C is bf16 (else fp32)
  int stream_out;  // fp32 C is stored non-temporal
  int64_t n_tiles_n;
  int ctas;
  float* partial;
};
__device__ __forceinline__ int group_rows(const RaggedGemm& p, int g) {
  return ragged_rows(p.offsets, g, p.R);
}
__device__ __forceinline__ int group_first(const RaggedGemm& p, int g) {
  return ragged_first(p.offsets, g, p.R);
}

// dW[g][m][n] = sum over the group's rows of A[r][m] B[r][n], for the weight
// gradient's tiles (field names as WgradGemm's).
struct RaggedWgrad {
  static constexpr int M_shared = 0, N_shared = 0;
  static constexpr float* C_shared = nullptr;
  const uint16_t* A;
  const uint16_t* B;
  int64_t lda, ldb;
  int M_routed, N_routed, E;
  const int32_t* offsets;
  int R;
  float* C_routed;
  int64_t tiles_m, tiles_n;
};
__device__ __forceinline__ int group_rows(const RaggedWgrad& p, int g) {
  return ragged_rows(p.offsets, g, p.R);
}
__device__ __forceinline__ int group_first(const RaggedWgrad& p, int g) {
  return ragged_first(p.offsets, g, p.R);
}

// Allows `kernel` `bytes` of dynamic LDS on the current device; `done` (one per
// kernel, zero at first) remembers the devices it was done on.
inline hipError_t allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return hipSuccess;
  e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace moe
