// Parameter blocks and small device helpers of the adapter kernels.
#pragma once
#include "device.hpp"

namespace moe {

// One adapter call as the kernels see it.  In the backward pass x is dy, w is
// read K-major, and the roles of A and B change: K and N are always the lengths
// of the product at hand (rows of `in` have K values, rows of `out` N).
struct LoraCall {
  const bf16_t* in;       // [T][K]: x, or dy
  const bf16_t* w;        // [N][K], or (K-major) [K][N]
  const bf16_t* shrink;   // [L][r][K] (A), or (K-major) [L][K][r] (B)
  const bf16_t* expand;   // [L][N][r] (B), or (K-major) [L][r][N] (A)
  const int32_t* adapter; // [T]
  const float* scale;     // [L] or NULL
  int T, K, N, L, r;
  void* out;              // [T][N]
  int out16;              // out is bf16 (else fp32)
};

// The rows of each adapter: counts[l] of them from offsets[l] of `sorted` on.
struct LoraLists {
  int32_t *counts, *offsets, *sorted;
};

// Outputs of the first product; each but one may be NULL.
struct ShrinkOut {
  float* v;           // fp32 [T][r], unscaled (zero rows without an adapter)
  uint16_t* parts;    // bf16 [T][2 r]: scaled, upper parts then lower parts
  const float* xa;    // fp32 [T][r] in ...
  uint16_t* xa_parts; // ... and its parts (all rows), written on the way
};

// the row's adapter, or -1
__device__ __forceinline__ int lora_id(const LoraCall& c, int64_t t) {
  const int l = c.adapter[t];
  return (uint32_t)l < (uint32_t)c.L ? l : -1;
}
__device__ __forceinline__ float lora_scale(const LoraCall& c, int l) {
  return c.scale ? c.scale[l] : 1.f;
}

// v as two bf16 parts: hi carries 8 bits of it, lo the next 8 (v = hi + lo to 2^-16)
__device__ __forceinline__ void split_bf16(float v, bf16_t& hi, bf16_t& lo) {
  hi = f32_to_bf16(v);
  lo = f32_to_bf16(v - bf16_to_f32(hi));
}

// 16-byte buffer loads with out-of-range offsets reading as zero
__device__ __forceinline__ __amdgpu_buffer_rsrc_t lora_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

}  // namespace moe
