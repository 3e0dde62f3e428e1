// The first product of the adapters, v[t] = M[a] in[t] with M = A [r][K]
// (forward) or B^T, B stored [K][r] (backward), for tiles of 16 rows whose
// adapters may all differ.
//
// One workgroup takes the rows of a tile that name one adapter after the
// other: MFMA 16x16x32 products of all 16 rows with that adapter, of which only
// its own rows' results are stored, so other rows (and other adapters' values)
// never meet.  The four waves split K in chunks of 64, and their sums are added
// in wave order.  A wave streams its chunks through a ring of LDS stages of its
// own (16 rows x 64 k, and 64 k of 16 RB ranks), so loads of several chunks are in
// flight and no barrier sits in the loop; K-major adapters are read back
// transposed.  (Loading operands straight into registers, two chunks ahead,
// took 1.5 us per trip: adapters_decode 13.6 us in its first launch against
// 10.0 us.)  Bound by reading the rows and the live adapters once (2 K bytes per
// row, 2 r K per adapter and tile), and by latency for few rows.
#pragma once
#include "lora.hpp"

namespace moe {
namespace {

constexpr uint32_t kShrinkOob = 0x80000000u;
constexpr int kShrinkWaves = 4;

// Stages of a wave's ring, 2 KB of rows and 2 KB per block of 16 ranks each: at
// least two, and 16 KB or more in flight per wave.
template <int RB> constexpr int shrink_stages() { return RB <= 2 ? 4 : RB == 4 ? 3 : 2; }
template <int RB> constexpr int shrink_stage_bytes() { return 2048 * (1 + RB); }
template <int RB> constexpr int shrink_lds_bytes() {
  return kShrinkWaves * shrink_stages<RB>() * shrink_stage_bytes<RB>();
}

// 16-byte chunk c (8 k) of row r of a row-major stage block sits at c ^ shrink_swz(r)
__device__ __forceinline__ int shrink_swz(int r) { return (r >> 1) & 7; }

template <int N>
__device__ __forceinline__ void shrink_wait() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Ranks 16 rb .. 16 (rb + RB) - 1 (those below r).  slot, slots: this workgroup
// takes the tile's distinct adapters slot, slot + slots, ... (in order of first row).
// Chunks q0 .. q1 - 1 of K; PART: their sums go to o.v as they are (rows without an
// adapter are left out), to be added up by the caller's next kernel.
template <int RB, bool KMAJ, bool PART>
__device__ __forceinline__ void lora_shrink_tile(const LoraCall& c, const ShrinkOut& o, int tile, int rb,
                                                 int slot, int slots, int q0, int q1, char* lds) {
  constexpr int S = shrink_stages<RB>(), SB = shrink_stage_bytes<RB>(), V = 2 + 2 * RB;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, gq = lane >> 4;
  const int64_t t0 = (int64_t)tile * 16;
  const int rows = (int)min((int64_t)16, c.T - t0);
  const int my = col < rows ? lora_id(c, t0 + col) : -1;  // adapter of row `col`, in every lane group
  if (!PART && slot == 0 && rb == 0 && o.v) {  // rows without an adapter
    for (int e = threadIdx.x; e < rows * c.r; e += blockDim.x)
      if (lora_id(c, t0 + e / c.r) < 0) o.v[t0 * c.r + e] = 0.f;
  }
  if (slot == 0 && rb == 0 && q0 == 0 && o.xa) {
    for (int e = threadIdx.x; e < rows * c.r; e += blockDim.x) {
      const int64_t t = t0 + e / c.r;
      const int j = e % c.r;
      split_bf16(o.xa[t * c.r + j], kParts32, o.xa_parts + t * kParts32 * c.r + j, c.r);
    }
  }
  // distinct adapters: bit `row` of `left` is a row whose adapter is yet to come
  uint32_t left = (uint32_t)__ballot(lane < 16 && my >= 0);
  const __amdgpu_buffer_rsrc_t rsX = lora_rsrc(c.in + t0 * c.K, (uint32_t)(rows * c.K * 2));
  char* ring = lds + wave * (S * SB);
  const int nq = q1 - q0;
  const int nm = wave < nq ? (nq - 1 - wave) / kShrinkWaves + 1 : 0;  // this wave's chunks
  for (int n = 0; left; ++n) {
    const int l = __builtin_amdgcn_readlane(my, __builtin_ctz(left));
    const uint32_t same = (uint32_t)__ballot(lane < 16 && my == l);
    left &= ~same;
    if (n % slots != slot) continue;
    f32x4 acc[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const __amdgpu_buffer_rsrc_t rsM =
        lora_rsrc(c.shrink + (int64_t)l * c.r * c.K, (uint32_t)(c.r * c.K * 2));
    // chunk m of this wave into ring slot s; loads past K or the ranks bring zeros
    auto issue = [&](int m, int s) {
      const int k0 = (q0 + wave + kShrinkWaves * m) * 64;
      char* st = ring + __builtin_amdgcn_readfirstlane(s * SB);
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const int r = 8 * d + (lane >> 3), k = k0 + 8 * ((lane & 7) ^ shrink_swz(r));
        lds_dma16(rsX, st + d * 1024, r < rows && k < c.K ? (uint32_t)((r * c.K + k) * 2) : kShrinkOob, 0);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          uint32_t off;
          if constexpr (KMAJ) {  // 32 k-rows of 16 ranks, 32 bytes each
            const int kk = k0 + 32 * d + (lane >> 1), j = 16 * (rb + b) + 8 * (lane & 1);
            off = kk < c.K && j < c.r ? (uint32_t)((kk * c.r + j) * 2) : kShrinkOob;
          } else {
            const int j = 16 * (rb + b) + r;
            off = k < c.K && j < c.r ? (uint32_t)((j * c.K + k) * 2) : kShrinkOob;
          }
          lds_dma16(rsM, st + 2048 * (1 + b) + d * 1024, off, 0);
        }
      }
    };
#pragma unroll
    for (int m = 0; m < S; ++m)
      if (m < nm) issue(m, m);
    int s = 0;
    for (int m = 0; m < nm; ++m) {
      const int later = min(nm - 1 - m, S - 1);  // chunks issued after this one
      if (S > 3 && later >= 3)
        shrink_wait<(S > 3 ? 3 : 1) * V>();
      else if (S > 2 && later >= 2)
        shrink_wait<(S > 2 ? 2 : 1) * V>();
      else if (later >= 1)
        shrink_wait<V>();
      else
        shrink_wait<0>();
      const char* st = ring + s * SB;
      typedef short i16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) i16x4 lds_v4;
      typedef __attribute__((address_space(3))) char lds_char;
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // step h takes k = 32 h + 8 gq + (0 .. 7)
        const int at = col * 128 + 16 * ((4 * h + gq) ^ shrink_swz(col));
        const bf16x8 x = *reinterpret_cast<const bf16x8*>(st + at);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          const char* mb = st + 2048 * (1 + b);
          if constexpr (KMAJ) {
            // lane col of a 16-lane group points at k-row 8 gq + col / 4 (+ 4) and ranks
            // 4 (col % 4) .. + 3 and gets rank `col` at four consecutive k
            const char* q = mb + (32 * h + 8 * gq + (col >> 2)) * 32 + 8 * (col & 3);
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)((lds_char*)q));
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)((lds_char*)(q + 128)));
            acc[b] = mfma16(
                x, __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7)), acc[b]);
          } else {
            acc[b] = mfma16(x, *reinterpret_cast<const bf16x8*>(mb + at), acc[b]);
          }
        }
      }
      if (m + S < nm) {
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this stage's reads are done
        issue(m + S, s);
      }
      s = s == S - 1 ? 0 : s + 1;
    }
    // sum over the waves in order; lane (col, gq) then holds rows 4 gq + i, rank 16 b + col
    f32x4* red = reinterpret_cast<f32x4*>(lds);
    __syncthreads();  // every wave is done with its ring
    if (wave > 0) {
#pragma unroll
      for (int b = 0; b < RB; ++b) red[((wave - 1) * RB + b) * 64 + lane] = acc[b];
    }
    __syncthreads();
    if (wave == 0) {
      const float sc = lora_scale(c, l);
#pragma unroll
      for (int b = 0; b < RB; ++b) {
#pragma unroll
        for (int w = 0; w < kShrinkWaves - 1; ++w) acc[b] += red[(w * RB + b) * 64 + lane];
        const int j = 16 * (rb + b) + col;
        if (j >= c.r) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 4 * gq + i;
          if (!((same >> row) & 1)) continue;
          const int64_t t = t0 + row;
          if (PART || o.v) o.v[t * c.r + j] = acc[b][i];
          if constexpr (PART) continue;
          const float v = acc[b][i] * sc;
          if (o.parts) split_bf16(v, o.np, o.parts + t * o.np * c.r + j, c.r);
        }
      }
    }
    __syncthreads();  // the sums are read before the next adapter's chunks
  }
}

}  // namespace
}  // namespace moe
