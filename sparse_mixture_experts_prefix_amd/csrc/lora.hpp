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
  uint16_t* parts;    // bf16 [T][np][r]: scaled, in np parts
  int np;
  const float* xa;    // fp32 [T][r] in ...
  uint16_t* xa_parts; // ... and its kParts32 parts (all rows), written on the way
};

// the row's adapter, or -1
__device__ __forceinline__ int lora_id(const LoraCall& c, int64_t t) {
  const int l = c.adapter[t];
  return (uint32_t)l < (uint32_t)c.L ? l : -1;
}
__device__ __forceinline__ float lora_scale(const LoraCall& c, int l) {
  return c.scale ? c.scale[l] : 1.f;
}

// v as NP bf16 parts of 8 bits each, upper first: v = their sum to 2^-16 (two parts) or
// 2^-24 (three), stored `step` elements apart.
__device__ __forceinline__ void split_bf16(float v, int np, bf16_t* at, int step) {
  for (int q = 0; q < np; ++q) {
    const bf16_t part = f32_to_bf16(v);
    at[q * step] = part;
    v -= bf16_to_f32(part);
  }
}
// Parts of a factor whose product is returned in bf16 (2^-16 is 1/128 of its half step),
// and in fp32.
constexpr int kParts16 = 2, kParts32 = 3;

// 16-byte buffer loads with out-of-range offsets reading as zero
__device__ __forceinline__ __amdgpu_buffer_rsrc_t lora_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

}  // namespace moe
