// The adapters' gradients, over the rows of each adapter (lora_rows.hpp):
//   da[l][j][d] = sum over l's rows of u[t][j] x[t][d]
//   db[l][n][j] = scale[l] sum over l's rows of xa[t][j] dy[t][n]
// One workgroup owns 128 columns (of x or dy) of one adapter and walks its
// rows in stages of 64: the rows' values (gathered, each row's 256 bytes) and
// their three bf16 parts of u or xa go through a ring of LDS stages, and both
// operands are read transposed, the rows being the reduction.  MFMA 16x16x32,
// 16 ranks x 32 columns per wave.  Row numbers come through LDS too, 1024 at a
// time, so the loop has no load that it waits for out of turn.  Bound by reading
// x and dy once (2 bytes per row and column) and writing the fp32 gradients.
#include "gemm_tile.hpp"
#include "lora.hpp"
#include "ops_launch.hpp"

namespace moe {
namespace {

struct LoraWgrad {
  LoraLists rows;
  const uint16_t* z[2];    // x [T][D], dy [T][N]
  const uint16_t* v[2];    // parts of u and of xa [T][3][r]
  float* out[2];           // da, db
  int width[2];            // D, N
  const float* scale;      // [L] or NULL
  int T, r;
  unsigned tiles0;         // column tiles of da; the others are db's
};

constexpr int kWgCols = 128;
constexpr int kWgZ = 64 * kWgCols * 2;  // 16 KB: a stage's rows
constexpr int kWgIds = 1024;            // row numbers held at a time
constexpr int kNP = kParts32;
// A stage's parts: each wave's 16 rows of 6 r bytes in wg_v() KB of its own.
template <int RB> constexpr int wg_v() { return (16 * 2 * kNP * 16 * RB + 1023) / 1024; }
template <int RB> constexpr int wg_stage_bytes() { return kWgZ + 4 * wg_v<RB>() * 1024; }
// (two workgroups per CU up to rank 32)
template <int RB> constexpr int wg_stages() { return RB == 1 || RB == 4 ? 3 : 2; }
template <int RB> constexpr int wg_lds_bytes() { return wg_stages<RB>() * wg_stage_bytes<RB>() + kWgIds * 4; }

// 16-byte chunk c of a stage's row (16 chunks of 8 columns) sits at c ^ wg_swz(row):
// a 32-lane half of a transposing read covers rows R .. R + 3 and R + 8 .. R + 11,
// two chunks each, which then fall on 16 different chunk positions.
__device__ __forceinline__ int wg_swz(int row) { return 2 * (row & 3) + 8 * ((row >> 3) & 1); }

template <int RB>
__global__ __launch_bounds__(256) void moe_lora_wgrad_kernel(LoraWgrad p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  constexpr int S = wg_stages<RB>(), SB = wg_stage_bytes<RB>(), NV = wg_v<RB>(), V = 4 + NV;
  int* ids = reinterpret_cast<int*>(lds + S * SB);
  const int l = blockIdx.y;
  const int which = blockIdx.x >= p.tiles0;
  const int C = which ? p.width[1] : p.width[0];
  const int c0 = (int)(blockIdx.x - (which ? p.tiles0 : 0)) * kWgCols;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, gq = lane >> 4;
  const int r = p.r, rowb = 2 * kNP * r;  // bytes of a row's parts
  const int rows = __builtin_amdgcn_readfirstlane(p.rows.counts[l]);
  const int32_t* list = p.rows.sorted + __builtin_amdgcn_readfirstlane(p.rows.offsets[l]);
  const __amdgpu_buffer_rsrc_t rsZ = make_rsrc(which ? p.z[1] : p.z[0], (uint32_t)((int64_t)p.T * C * 2));
  const __amdgpu_buffer_rsrc_t rsV = make_rsrc(which ? p.v[1] : p.v[0], (uint32_t)((int64_t)p.T * rowb));
  f32x4 acc[RB][2];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[b][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // A stage's loads: wave w brings rows 16 w .. + 15.  Load i: rows 4 i + lane / 16 of
  // them, 256 bytes each; then NV loads of their parts, 16 bytes per lane in row
  // order.  Rows past the adapter's last (-1) read as zero.
  auto issue = [&](int stage, int slot) {
    char* st = lds + __builtin_amdgcn_readfirstlane(slot * SB);
    const int* id = ids + stage * 64 + 16 * wave;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = 4 * i + (lane >> 4), row = 16 * wave + q;
      const int t = id[q];
      const int n = c0 + 8 * ((lane & 15) ^ wg_swz(row));
      lds_dma16(rsZ, st + (4 * wave + i) * 1024,
                t >= 0 && n < C ? (uint32_t)t * (uint32_t)(C * 2) + (uint32_t)n * 2 : kOob, 0);
    }
#pragma unroll
    for (int b = 0; b < NV; ++b) {
      const int at = b * 1024 + lane * 16, q = at / rowb;
      const int t = q < 16 ? id[q & 15] : -1;
      lds_dma16(rsV, st + kWgZ + (NV * wave + b) * 1024,
                t >= 0 ? (uint32_t)t * (uint32_t)rowb + (uint32_t)(at % rowb) : kOob, 0);
    }
  };
  typedef __attribute__((address_space(3))) i16x4 lds_v4;
  typedef __attribute__((address_space(3))) char lds_char;
  auto read_tr = [](const char* lo_at, const char* hi_at) {
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)((lds_char*)lo_at));
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)((lds_char*)hi_at));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  for (int i0 = 0; i0 < rows; i0 += kWgIds) {
    const int n = min(kWgIds, rows - i0), stages = (n + 63) / 64;
    __syncthreads();  // the last stages' reads, and their row numbers, are done with
    for (int i = threadIdx.x; i < stages * 64; i += 256) ids[i] = i < n ? list[i0 + i] : -1;
    __syncthreads();
#pragma unroll
    for (int s = 0; s < S - 1; ++s)
      if (s < stages) issue(s, s);
    int slot = 0;
    for (int s = 0; s < stages; ++s) {
      if (S > 2 && stages - 1 - s >= 1)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(V) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();  // stage s is whole, and every wave has read stage s - 1
      asm volatile("" ::: "memory");
      if (s + S - 1 < stages) issue(s + S - 1, slot == 0 ? S - 1 : slot - 1);
      const char* st = lds + slot * SB;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = 32 * h + 8 * gq + (col >> 2);  // row of this lane's words, and 4 further
        bf16x8 z[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int cc = wave * 32 + 16 * j + 4 * (col & 3);
          auto at = [&](int row) { return st + row * 256 + ((cc >> 3) ^ wg_swz(row)) * 16 + (cc & 7) * 2; };
          z[j] = read_tr(at(k), at(k + 4));
        }
        const char* v0 = st + kWgZ + (k >> 4) * (NV * 1024) + (k & 15) * rowb + 8 * (col & 3);
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int part = 0; part < kNP; ++part) {
            // (ranks past r read the neighbour's values: they reach results that are not stored)
            const char* at = v0 + part * 2 * r + 32 * b;
            const bf16x8 v = read_tr(at, at + 4 * rowb);
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[b][j] = mfma16(v, z[j], acc[b][j]);
          }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this wave's reads of stage s are done
      slot = slot == S - 1 ? 0 : slot + 1;
    }
  }
  // lane (col, gq) holds ranks 16 b + 4 gq + i of column c0 + 32 wave + 16 j + col
  // (without rows the scale is not read: a NaN there would reach the zeros)
  const float sc = which && p.scale && rows > 0 ? p.scale[l] : 1.f;
  float* out = (which ? p.out[1] : p.out[0]) + (int64_t)l * r * C;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int n = c0 + wave * 32 + 16 * j + col;
    if (n >= C) continue;
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int j0 = 16 * b + 4 * gq;
      if (j0 >= r) continue;  // r is a multiple of 8: four ranks are in or out together
      if (which) {
        *reinterpret_cast<f32x4*>(out + (int64_t)n * r + j0) = acc[b][j] * sc;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) out[(int64_t)(j0 + i) * C + n] = acc[b][j][i];
      }
    }
  }
}

template <int RB>
hipError_t launch(const LoraWgrad& p, int L, hipStream_t s) {
  static std::atomic<uint64_t> done;
  const hipError_t e =
      allow_lds(reinterpret_cast<const void*>(moe_lora_wgrad_kernel<RB>), wg_lds_bytes<RB>(), done);
  if (e != hipSuccess) return e;
  const unsigned tiles = p.tiles0 + (unsigned)((p.width[1] + kWgCols - 1) / kWgCols);
  hipLaunchKernelGGL(moe_lora_wgrad_kernel<RB>, dim3(tiles, (unsigned)L), dim3(256), wg_lds_bytes<RB>(), s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_wgrad(const LoraLists& rows, const void* x, const void* dy, const uint16_t* u,
                             const uint16_t* xa, const float* scale, int T, int D, int N, int L, int r,
                             float* da, float* db, hipStream_t s) {
  LoraWgrad p{rows, {static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(dy)}, {u, xa}, {da, db}, {D, N},
              scale, T, r, (unsigned)((D + kWgCols - 1) / kWgCols)};
  if (r <= 16) return launch<1>(p, L, s);
  if (r <= 32) return launch<2>(p, L, s);
  if (r <= 64) return launch<4>(p, L, s);
  return launch<8>(p, L, s);
}

}  // namespace moe
