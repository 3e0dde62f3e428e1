// The adapters' products for few rows (at most 64): two launches.
//
// First, in one launch: the projection's weights are streamed once (tiles of all
// rows x 64 columns of decode_tile_staged, K cut into parts so that the grid
// fills the chip, fp32 partial sums), while other workgroups compute the
// adapters' first product.  Then each output is its partial sums, in part
// order, plus its row's second product in fp32.  Bound by streaming W (2 N K
// bytes) and the live adapters.
#include "gemm_decode_tile.hpp"
#include "lora_shrink.hpp"
#include "ops_launch.hpp"
#include "ragged.hpp"

namespace moe {
namespace {

// One part of K of the projection for decode_tile_staged: m-tile index = part.
struct LoraParts {
  static constexpr bool kRagged = true, kFold = false, kLora = false, kParts = true;
  static constexpr const int32_t* row_token = nullptr;
  static constexpr int64_t a_bytes = 0, ld_gu = 0;
  static constexpr uint16_t* gu_out = nullptr;
  static constexpr const void* B_shared = nullptr;
  static constexpr int N_shared = 0, K_shared = 0, E = 1;
  const uint16_t* A;
  int64_t lda;
  const void* B_routed;
  int N_routed, K_routed;
  float* C;  // [parts][T][N]
  int64_t ldc;
  int64_t n_tiles_n;
  int T, parts;
  int64_t first_block;
  // 64-wide K chunks of part dr.g_part: first one, and how many
  __device__ __forceinline__ void k_range(const DecodeRows& r, int& q0, int& nq) const {
    const int all = nq;
    q0 = (int)((int64_t)r.part * all / parts);
    nq = (int)((int64_t)(r.part + 1) * all / parts) - q0;
  }
  __device__ __forceinline__ float* part_out(const DecodeRows& r) const {
    return C + (int64_t)r.part * T * ldc;
  }
};
template <int BMD>
__device__ __forceinline__ bool decode_rows(const LoraParts& p, int64_t m, DecodeRows& r) {
  if (m >= p.parts) return false;
  r.g = 0;
  r.part = (int)m;
  r.row0 = 0;
  r.valid = p.T;
  return true;
}
template <int BMD>
__device__ __forceinline__ int decode_valid(const LoraParts&, const DecodeRows& r) {
  return r.valid;
}

// Blocks 0 .. first_block - 1 compute the first product, one per block of 16 ranks,
// tile of 16 rows and slot of 16 (the tile's distinct adapters); the others the
// projection.
template <int MT, bool KMAJ>
__global__ __launch_bounds__(256) void moe_lora_decode_kernel(LoraParts p, LoraCall c, ShrinkOut o) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  if (blockIdx.x < p.first_block) {
    const int tiles = (c.T + 15) / 16, b = blockIdx.x / 16;
    lora_shrink_tile<1, KMAJ>(c, o, b % tiles, b / tiles, blockIdx.x % 16, 16, lds);
    return;
  }
  decode_tile_staged<MT, KMAJ, false>(p, lds);
}

// out[t][n] = sum of the parts (in part order) + sum_j sv[t][j] expand[a][n][j]
// (K-major: expand[a][j][n]); one row and 256 columns per workgroup
template <bool KMAJ>
__global__ __launch_bounds__(256) void moe_lora_finish_kernel(LoraCall c, const float* partial, int parts,
                                                              const float* sv) {
  const int t = blockIdx.y;
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= c.N) return;
  const int l = lora_id(c, t);
  float s = 0.f;
#pragma unroll 4
  for (int q = 0; q < parts; ++q) s += partial[((int64_t)q * c.T + t) * c.N + n];
  if (l >= 0) {
    const float* v = sv + (int64_t)t * c.r;  // uniform: scalar loads
    float e = 0.f;
    if constexpr (KMAJ) {
      const bf16_t* m = c.expand + (int64_t)l * c.r * c.N + n;
#pragma unroll 8
      for (int j = 0; j < c.r; ++j) e = fmaf(v[j], bf16_to_f32(m[(int64_t)j * c.N]), e);
    } else {
      const u32x4* m = reinterpret_cast<const u32x4*>(c.expand + ((int64_t)l * c.N + n) * c.r);
#pragma unroll 8
      for (int j = 0; j < c.r / 8; ++j) {
        const u32x4 b = m[j];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          e = fmaf(v[8 * j + 2 * h], __builtin_bit_cast(float, b[h] << 16), e);
          e = fmaf(v[8 * j + 2 * h + 1], __builtin_bit_cast(float, b[h] & 0xFFFF0000u), e);
        }
      }
    }
    s += e;
  }
  const int64_t at = (int64_t)t * c.N + n;
  if (c.out16)
    static_cast<bf16_t*>(c.out)[at] = f32_to_bf16(s);
  else
    static_cast<float*>(c.out)[at] = s;
}

template <int MT, bool KMAJ>
hipError_t launch(const LoraCall& c, const LoraParts& p, const ShrinkOut& o, hipStream_t s) {
  static std::atomic<uint64_t> done;
  constexpr int lds = km_lds_bytes<MT>() > shrink_lds_bytes<1>() ? km_lds_bytes<MT>() : shrink_lds_bytes<1>();
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(moe_lora_decode_kernel<MT, KMAJ>), lds, done);
  if (e != hipSuccess) return e;
  const int64_t blocks = p.first_block + p.parts * p.n_tiles_n;
  hipLaunchKernelGGL((moe_lora_decode_kernel<MT, KMAJ>), dim3((unsigned)blocks), dim3(256), lds, s, p, c, o);
  return hipGetLastError();
}

template <int MT>
hipError_t launch_layout(const LoraCall& c, bool kmajor, const LoraParts& p, const ShrinkOut& o, hipStream_t s) {
  return kmajor ? launch<MT, true>(c, p, o, s) : launch<MT, false>(c, p, o, s);
}

}  // namespace

hipError_t launch_lora_decode(const LoraCall& c, bool kmajor, float* v, float* sv, uint16_t* parts16,
                              float* partial, int parts, hipStream_t s) {
  LoraParts p{};
  p.A = c.in;
  p.lda = c.K;
  p.B_routed = c.w;
  p.N_routed = c.N;
  p.K_routed = c.K;
  p.C = partial;
  p.ldc = c.N;
  p.n_tiles_n = (c.N + 63) / 64;
  p.T = c.T;
  p.parts = parts;
  p.first_block = (c.T + 15) / 16 * ((c.r + 15) / 16) * 16;
  const ShrinkOut o{v, sv, parts16};
  hipError_t e;
  if (c.T <= 16)
    e = launch_layout<1>(c, kmajor, p, o, s);
  else if (c.T <= 32)
    e = launch_layout<2>(c, kmajor, p, o, s);
  else
    e = launch_layout<4>(c, kmajor, p, o, s);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((c.N + 255) / 256), (unsigned)c.T);
  if (kmajor)
    hipLaunchKernelGGL(moe_lora_finish_kernel<true>, grid, dim3(256), 0, s, c, partial, parts, sv);
  else
    hipLaunchKernelGGL(moe_lora_finish_kernel<false>, grid, dim3(256), 0, s, c, partial, parts, sv);
  return hipGetLastError();
}

}  // namespace moe
