// The first product of the adapters, v[t] = M[a] in[t] with M = A [r][K]
// (forward) or B^T, B stored [K][r] (backward), for tiles of 16 rows whose
// adapters may all differ.
//
// One workgroup takes the rows of a tile that name one adapter after the
// other: MFMA 16x16x32 products of all 16 rows with that adapter, of which only
// its own rows' results are stored, so other rows (and other adapters' values)
// never meet.  The four waves split K in chunks of 64 and their sums are added
// in wave order.  Rows and adapters are read straight from memory into
// operands, with K permuted inside a chunk so that a row's four lanes read one
// full 128-byte line.  Bound by reading the rows and the live adapters once
// (2 K bytes per row, 2 r K per adapter and tile).
#pragma once
#include "lora.hpp"

namespace moe {
namespace {

struct ShrinkOut {
  float* v;        // fp32 [T][r], unscaled (zero rows without an adapter), or NULL
  float* sv;       // fp32 [T][r], scaled, or NULL
  uint16_t* parts; // bf16 [T][2 r]: scaled, upper parts then lower parts, or NULL
};

constexpr uint32_t kShrinkOob = 0x80000000u;
constexpr int kShrinkWaves = 4;

// Chunk bytes of K-major adapters (64 k-rows of r values) with room for the
// last row's reads past r, which only reach columns that are not stored.
__host__ __device__ constexpr int shrink_stage_bytes(int r) { return 64 * r * 2 + 256; }
// LDS: the waves' sums [3][RB][64] f32x4, or (K-major) the four waves' chunks
template <int RB>
__host__ __device__ constexpr int shrink_lds_bytes(int r, bool kmajor) {
  const int red = (kShrinkWaves - 1) * RB * 64 * 16;
  const int st = kmajor ? kShrinkWaves * shrink_stage_bytes(r) : 0;
  return red > st ? red : st;
}

// RB: blocks of 16 ranks (16 RB >= r).  slot, slots: this workgroup takes the
// tile's distinct adapters slot, slot + slots, ... (in order of first row).
template <int RB, bool KMAJ>
__device__ __forceinline__ void lora_shrink_tile(const LoraCall& c, const ShrinkOut& o, int tile, int slot,
                                                 int slots, char* lds) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, gq = lane >> 4;
  const int64_t t0 = (int64_t)tile * 16;
  const int rows = (int)min((int64_t)16, c.T - t0);
  const int my = col < rows ? lora_id(c, t0 + col) : -1;  // adapter of row `col`, in every lane group
  if (slot == 0 && o.v) {  // rows without an adapter
    for (int e = threadIdx.x; e < rows * c.r; e += blockDim.x) {
      const int row = e / c.r;
      if (lora_id(c, t0 + row) < 0) o.v[(t0 + row) * c.r + e % c.r] = 0.f;
    }
  }
  // distinct adapters: bit `row` of `left` is a row whose adapter is yet to come
  uint32_t left = (uint32_t)__ballot(lane < 16 && my >= 0);
  const __amdgpu_buffer_rsrc_t rsX = lora_rsrc(c.in + t0 * c.K, (uint32_t)(rows * c.K * 2));
  const uint32_t offX = col < rows ? (uint32_t)(col * c.K * 2) + gq * 32 : kShrinkOob;
  const int nq = (c.K + 63) / 64;
  for (int n = 0; left; ++n) {
    const int first = __builtin_ctz(left);
    const int l = __builtin_amdgcn_readlane(my, first);
    const uint32_t same = (uint32_t)__ballot(lane < 16 && my == l);
    left &= ~same;
    if (n % slots != slot) continue;
    f32x4 acc[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[b] = f32x4{0.f, 0.f, 0.f, 0.f};
    const __amdgpu_buffer_rsrc_t rsM =
        lora_rsrc(c.shrink + (int64_t)l * c.r * c.K, (uint32_t)(c.r * c.K * 2));
    if constexpr (!KMAJ) {
      uint32_t offM[RB];
#pragma unroll
      for (int b = 0; b < RB; ++b)
        offM[b] = 16 * b + col < c.r ? (uint32_t)((16 * b + col) * c.K * 2) + gq * 32 : kShrinkOob;
      constexpr int U = RB >= 4 ? 1 : 2;  // chunks whose loads go out together
      for (int q = wave; q < nq; q += U * kShrinkWaves) {
        u32x4 x[U][2], m[U][RB][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k0 = (q + u * kShrinkWaves) * 64;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bool in = k0 + gq * 16 + 8 * h < c.K;
            x[u][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                    rsX, in ? offX + 16 * h : kShrinkOob, k0 * 2, 0));
#pragma unroll
            for (int b = 0; b < RB; ++b)
              m[u][b][h] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                         rsM, in ? offM[b] + 16 * h : kShrinkOob, k0 * 2, 0));
          }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int b = 0; b < RB; ++b) acc[b] = mfma16(as_bf16x8(x[u][h]), as_bf16x8(m[u][b][h]), acc[b]);
      }
    } else {
      // a chunk's 64 k-rows of the adapter are contiguous: staged through the
      // wave's own LDS and read transposed (see decode_tile_staged): lane col of
      // a 16-lane group points at k-row 8 gq + col / 4 (+ 4) and ranks
      // 4 (col % 4) .. + 3 and gets rank `col` at four consecutive k
      char* st = lds + wave * shrink_stage_bytes(c.r);
      const int rowb = c.r * 2;
      typedef short i16x4 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) i16x4 lds_v4;
      typedef __attribute__((address_space(3))) char lds_char;
      for (int q = wave; q < nq; q += kShrinkWaves) {
        const int k0 = q * 64;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the last chunk's reads are done
        for (int b = 0; b < c.r / 8; ++b)
          lds_dma16(rsM, st + b * 1024, (uint32_t)(k0 * rowb + b * 1024 + lane * 16), 0);
        u32x4 x[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // step h takes k = 32 h + 8 gq + (0 .. 7)
          const bool in = k0 + 32 * h + 8 * gq < c.K;
          x[h] = __builtin_bit_cast(
              u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                         rsX, in && col < rows ? (uint32_t)(col * c.K * 2 + 64 * h + 16 * gq) : kShrinkOob,
                         k0 * 2, 0));
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int b = 0; b < RB; ++b) {
            const char* at = st + (32 * h + 8 * gq + (col >> 2)) * rowb + 32 * b + 8 * (col & 3);
            const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)((lds_char*)at));
            const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)((lds_char*)(at + 4 * rowb)));
            acc[b] = mfma16(as_bf16x8(x[h]),
                            __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7)),
                            acc[b]);
          }
      }
    }
    // sum over the waves in order; lane (col, gq) then holds rows 4 gq + i, rank 16 b + col
    f32x4* red = reinterpret_cast<f32x4*>(lds);
    __syncthreads();  // every wave is done with the LDS (chunks, the adapter before)
    if (wave > 0) {
#pragma unroll
      for (int b = 0; b < RB; ++b) red[((wave - 1) * RB + b) * 64 + lane] = acc[b];
    }
    __syncthreads();
    if (wave == 0) {
      const float s = lora_scale(c, l);
#pragma unroll
      for (int b = 0; b < RB; ++b) {
#pragma unroll
        for (int w = 0; w < kShrinkWaves - 1; ++w) acc[b] += red[(w * RB + b) * 64 + lane];
        const int j = 16 * b + col;
        if (j >= c.r) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 4 * gq + i;
          if (!((same >> row) & 1)) continue;
          const int64_t t = t0 + row;
          if (o.v) o.v[t * c.r + j] = acc[b][i];
          const float v = acc[b][i] * s;
          if (o.sv) o.sv[t * c.r + j] = v;
          if (o.parts) {
            bf16_t hi, lo;
            split_bf16(v, hi, lo);
            o.parts[t * 2 * c.r + j] = hi;
            o.parts[t * 2 * c.r + c.r + j] = lo;
          }
        }
      }
    }
    __syncthreads();  // the sums are read before the next adapter's chunks or sums
  }
}

}  // namespace
}  // namespace moe
