// The adapters' products for few rows (lora_few_rows in ops_plan.hpp says which calls):
// two launches.
//
// First, in one launch: the projection's weights are streamed once (tiles of up to 64
// rows x 64 columns, K cut into parts so that the grid fills the chip, fp32 partial
// sums; more rows take several tiles, which share the weights in an XCD's L2), while
// other workgroups compute the adapters' first product (and, for the backward pass,
// the rows' lists).  Then each output is its partial sums, in part order, plus its
// row's second product in fp32.  Bound by streaming W (2 N K bytes) and the live
// adapters.
#include "lora_rows.hpp"
#include "lora_shrink.hpp"
#include "ops_launch.hpp"
#include "ragged.hpp"

namespace moe {
namespace {

// Projection tile: `rows` <= 16 MT rows from t0 on x 64 columns, chunks q0 .. q1 - 1 of
// 64 k.  A stage (all rows, 64 columns) is shared by the four waves, 16 columns each, in a
// ring of four (64 rows) or six stages, all but one in flight, one barrier per stage.  64
// or 72 KB of LDS per workgroup, so two share a CU (each wave with its own ring of whole
// stages took 128 KB at 64 rows: one workgroup per CU, 24 us against 15 us for
// 64 rows x 5760 columns x 2880).
// (a multiple of 4 KB: the waves issue equally many 1-KB loads)
template <int MT> constexpr int tile_stage_bytes() { return (MT * 2048 + 8192 + 4095) / 4096 * 4096; }
template <int MT> constexpr int tile_stages() { return MT == 4 ? 4 : 6; }
template <int MT> constexpr int tile_lds_bytes() { return tile_stages<MT>() * tile_stage_bytes<MT>(); }

__device__ __forceinline__ int row_swz(int r) { return (r >> 1) & 7; }
// K-major weights: 64 k-rows of 64 columns, chunk c (8 columns) of k-row r at c ^ col_swz(r), so
// that a 32-lane half of a transposing read (k-rows R .. R + 3 and R + 8 .. R + 11,
// two chunks each) hits every bank once
__device__ __forceinline__ int col_swz(int r) { return 2 * ((r >> 1) & 1) + 4 * ((r >> 3) & 1); }

template <int MT, bool KMAJ>
__device__ __forceinline__ void project_tile(const LoraCall& c, int t0, int rows, int n0, int q0, int q1, float* out,
                                             char* lds) {
  constexpr int SB = tile_stage_bytes<MT>(), AB = MT * 2048, S = tile_stages<MT>();
  constexpr int LA = MT * 2;            // 1-KB blocks of rows
  constexpr int V = SB / 4096;          // loads per wave and stage
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, gq = lane >> 4, ir = lane >> 3, ip = lane & 7;
  const int K = c.K, N = c.N;
  const __amdgpu_buffer_rsrc_t rsA = lora_rsrc(c.in + (int64_t)t0 * K, (uint32_t)(rows * K * 2));
  const __amdgpu_buffer_rsrc_t rsB = lora_rsrc(c.w, (uint32_t)((int64_t)N * K * 2));
  // block b of a stage: rows 8 b + ir (b < LA), else weight rows (or k-rows) 8 (b - LA) + ir
  auto issue = [&](int q, int slot) {
    const int k0 = q * 64;
    char* st = lds + __builtin_amdgcn_readfirstlane(slot * SB);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int b = wave + 4 * i;  // uniform
      if (b < LA) {
        const int r = 8 * b + ir, k = k0 + 8 * (ip ^ row_swz(r));
        lds_dma16(rsA, st + b * 1024, r < rows && k < K ? (uint32_t)((r * K + k) * 2) : kShrinkOob, 0);
      } else if (b < LA + 8) {
        const int r = 8 * (b - LA) + ir;
        uint32_t off;
        if constexpr (KMAJ) {
          const int k = k0 + r, n = n0 + 8 * (ip ^ col_swz(r));
          off = k < K && n < N ? (uint32_t)((k * N + n) * 2) : kShrinkOob;
        } else {
          const int k = k0 + 8 * (ip ^ row_swz(r)), n = n0 + r;
          off = k < K && n < N ? (uint32_t)((n * K + k) * 2) : kShrinkOob;
        }
        lds_dma16<true>(rsB, st + b * 1024, off, 0);  // read once: non-temporal
      } else {  // zeros into the stage's unused end: the waves' counts of loads stay equal
        lds_dma16(rsA, st + b * 1024, kShrinkOob, 0);
      }
    }
  };
  static_assert(4 * V * 1024 == SB, "a stage is the waves' loads");
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int n = q1 - q0;
#pragma unroll
  for (int s = 0; s < S - 1; ++s)
    if (s < n) issue(q0 + s, s);
  for (int s = 0; s < n; ++s) {
    const int later = min(n - 1 - s, S - 2);
    if (S > 5 && later >= 4)
      shrink_wait<(S > 5 ? 4 : 2) * V>();
    else if (S > 4 && later == 3)
      shrink_wait<(S > 4 ? 3 : 2) * V>();
    else if (later >= 2)
      shrink_wait<2 * V>();
    else if (later == 1)
      shrink_wait<V>();
    else
      shrink_wait<0>();
    __builtin_amdgcn_s_barrier();  // stage s is whole; every wave has read stage s - 1
    asm volatile("" ::: "memory");
    if (s + S - 1 < n) issue(q0 + s + S - 1, (s + S - 1) % S);
    const char* st = lds + (s % S) * SB;
    typedef short i16x4 __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) i16x4 lds_v4;
    typedef __attribute__((address_space(3))) char lds_char;
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // step h takes k = 32 h + 8 gq + (0 .. 7)
      bf16x8 b;
      if constexpr (KMAJ) {
        const int r = 32 * h + 8 * gq + (col >> 2), ch = 2 * wave + ((col & 3) >> 1);
        const char* q = st + AB + r * 128 + 16 * (ch ^ col_swz(r)) + 8 * (col & 1);
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)((lds_char*)q));
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4*)((lds_char*)(q + 4 * 128)));
        b = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      } else {
        const int r = 16 * wave + col;
        b = *reinterpret_cast<const bf16x8*>(st + AB + r * 128 + 16 * ((4 * h + gq) ^ row_swz(r)));
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int r = 16 * i + col;
        const bf16x8 a = *reinterpret_cast<const bf16x8*>(st + r * 128 + 16 * ((4 * h + gq) ^ row_swz(r)));
        acc[i] = mfma16(a, b, acc[i]);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this wave's reads of stage s are done
  }
  // lane (col, gq) holds rows 16 i + 4 gq + r of column n0 + 16 wave + col
  const int cn = n0 + 16 * wave + col;
  if (cn >= N) return;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = 16 * i + 4 * gq + r;
      if (t < rows) out[(int64_t)(t0 + t) * N + cn] = acc[i][r];
    }
}

struct FewRows {
  int shrink, lists;  // workgroups of the first product, and of the rows' lists
  int tiles, parts;   // column tiles, parts of K
  int blocks;         // blocks of 64 rows
  int v_parts;        // parts of K of the first product
  float* v;           // [v_parts][T][r]
  float* partial;     // [parts][T][N]
};

// Workgroups: the first product, one per block of 16 ranks, tile of 16 rows, part of K
// and slot of 16 (the tile's distinct adapters); the rows' lists; the projection.  The
// first product's parts are short, so that all of a wave's loads are in flight from the
// start: beside the weights' stream each wait takes several microseconds (whole rows
// of 4096 k took 11.3 us with the projection, which alone takes 8.2).
template <int MT, bool KMAJ>
__global__ __launch_bounds__(256) void moe_lora_decode_kernel(LoraCall c, ShrinkOut o, LoraLists rows, FewRows f) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  int b = blockIdx.x;
  if (b < f.shrink) {
    const int tiles = (c.T + 15) / 16, u = b / 16, q = u / tiles, part = q % f.v_parts, nq = (c.K + 63) / 64;
    ShrinkOut op = o;
    op.v = f.v + (int64_t)part * c.T * c.r;
    lora_shrink_tile<1, KMAJ, true>(c, op, u % tiles, q / f.v_parts, b % 16, 16, (int)((int64_t)part * nq / f.v_parts),
                                    (int)((int64_t)(part + 1) * nq / f.v_parts), lds);
    return;
  }
  b -= f.shrink;
  if (b < f.lists) {
    lora_list(c, rows, b, reinterpret_cast<int*>(lds));
    return;
  }
  b -= f.lists;
  // eight column tiles side by side (one per XCD), their row blocks behind them
  const int per = (f.tiles + 7) / 8 * 8 * f.blocks, part = b / per, u = b % per / 8;
  const int tile = u / f.blocks * 8 + b % 8, t0 = u % f.blocks * 64, nq = (c.K + 63) / 64;
  if (tile >= f.tiles) return;
  project_tile<MT, KMAJ>(c, t0, min(64, c.T - t0), tile * 64, (int)((int64_t)part * nq / f.parts),
                         (int)((int64_t)(part + 1) * nq / f.parts),
                         f.partial + (int64_t)part * c.T * c.N, lds);
}

__device__ __forceinline__ void store_out(const LoraCall& c, int64_t at, float v) {
  if (c.out16)
    static_cast<bf16_t*>(c.out)[at] = f32_to_bf16(v);
  else
    static_cast<float*>(c.out)[at] = v;
}

// The row's first product at rank j: its parts added in order.
__device__ __forceinline__ float sum_v(const LoraCall& c, const FewRows& f, int t, int j) {
  float v = f.v[(int64_t)t * c.r + j];
  for (int q = 1; q < f.v_parts; ++q) v += f.v[((int64_t)q * c.T + t) * c.r + j];
  return v;
}
// ... kept where asked for, by the row's first workgroup.
__device__ __forceinline__ void keep_v(const LoraCall& c, const ShrinkOut& o, const FewRows& f, int t, int l) {
  const int j = threadIdx.x;
  if (blockIdx.x != 0 || j >= c.r) return;
  const float v = l >= 0 ? sum_v(c, f, t, j) : 0.f;
  if (o.v) o.v[(int64_t)t * c.r + j] = v;
  if (o.parts) {
    const float s = l >= 0 ? v * lora_scale(c, l) : 0.f;
    split_bf16(s, o.np, o.parts + (int64_t)t * o.np * c.r + j, c.r);
  }
}

__device__ __forceinline__ float sum_parts(const LoraCall& c, const FewRows& f, int t, int n) {
  float s = 0.f;
#pragma unroll 4
  for (int q = 0; q < f.parts; ++q) s += f.partial[((int64_t)q * c.T + t) * c.N + n];
  return s;
}

// out[t][n] = sum of the parts (in part order) + sum_j sv[t][j] expand[a][n][j], one
// row and 256 columns per workgroup.  G lanes share a row of expand (16 bytes each, 8 G >=
// r), so a wave's loads are one contiguous piece (a row per lane read 16 bytes of 64
// different lines per load: 11 us against 10 us at 64 rows x 5760 columns, rank 64); the
// lanes' sums are added in a fixed tree.
template <int G, int VP>
__global__ __launch_bounds__(256) void moe_lora_finish_kernel(LoraCall c, ShrinkOut o, FewRows f) {
  __shared__ float es[256];
  const int t = blockIdx.y, lane = threadIdx.x & 63, w0 = threadIdx.x & ~63;
  const int n0 = blockIdx.x * 256 + w0;  // first column of this wave
  const int l = lora_id(c, t);
  const int n = n0 + lane, g = lane % G, row = lane / G;
  float s = n < c.N ? sum_parts(c, f, t, n) : 0.f;
  if (l >= 0) {  // uniform
    const float sc = lora_scale(c, l);
    float v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = 0.f;
    if (8 * g < c.r) {
#pragma unroll
      for (int q = 0; q < VP; ++q) {
        const float4* src = reinterpret_cast<const float4*>(f.v + ((int64_t)q * c.T + t) * c.r + 8 * g);
        const float4 x = src[0], y = src[1];
        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w, v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] *= sc;
    u32x4 b[G];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const int m = n0 + i * (64 / G) + row;
      b[i] = u32x4{0, 0, 0, 0};
      if (m < c.N && 8 * g < c.r) b[i] = ld16(c.expand + ((int64_t)l * c.N + m) * c.r + 8 * g);
    }
#pragma unroll
    for (int i = 0; i < G; ++i) {
      float e = 0.f;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        e = fmaf(v[2 * h], __builtin_bit_cast(float, b[i][h] << 16), e);
        e = fmaf(v[2 * h + 1], __builtin_bit_cast(float, b[i][h] & 0xFFFF0000u), e);
      }
#pragma unroll
      for (int off = 1; off < G; off <<= 1) e += __shfl_xor(e, off);
      if (g == 0) es[w0 + i * (64 / G) + row] = e;
    }
    __builtin_amdgcn_wave_barrier();  // the wave's own results, in its own words
    s += es[threadIdx.x];
  }
  if (n < c.N) store_out(c, (int64_t)t * c.N + n, s);
  if (o.v || o.parts) keep_v(c, o, f, t, l);
}

// ... K-major: expand[a][j][n] (the row's v is the same for all: scalar loads)
__global__ __launch_bounds__(256) void moe_lora_finish_kmajor_kernel(LoraCall c, ShrinkOut o, FewRows f) {
  const int t = blockIdx.y;
  const int n = blockIdx.x * 256 + threadIdx.x;
  const int l = lora_id(c, t);
  keep_v(c, o, f, t, l);
  if (n >= c.N) return;
  float s = sum_parts(c, f, t, n);
  if (l >= 0) {
    const bf16_t* m = c.expand + (int64_t)l * c.r * c.N + n;
    const float sc = lora_scale(c, l);
    float e = 0.f;
#pragma unroll 8
    for (int j = 0; j < c.r; ++j) e = fmaf(sum_v(c, f, t, j) * sc, bf16_to_f32(m[(int64_t)j * c.N]), e);
    s += e;
  }
  store_out(c, (int64_t)t * c.N + n, s);
}

template <int MT, bool KMAJ>
hipError_t launch(const LoraCall& c, const ShrinkOut& o, const LoraLists& rows, const FewRows& f, hipStream_t s) {
  static std::atomic<uint64_t> done;
  constexpr int lds = tile_lds_bytes<MT>() > shrink_lds_bytes<1>() ? tile_lds_bytes<MT>() : shrink_lds_bytes<1>();
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(moe_lora_decode_kernel<MT, KMAJ>), lds, done);
  if (e != hipSuccess) return e;
  const int64_t blocks = f.shrink + f.lists + (int64_t)(f.tiles + 7) / 8 * 8 * f.blocks * f.parts;
  hipLaunchKernelGGL((moe_lora_decode_kernel<MT, KMAJ>), dim3((unsigned)blocks), dim3(256), lds, s, c, o, rows, f);
  return hipGetLastError();
}

template <int G>
hipError_t launch_finish(const LoraCall& c, const ShrinkOut& o, const FewRows& f, dim3 grid, hipStream_t s) {
  if (f.v_parts == 2)
    hipLaunchKernelGGL((moe_lora_finish_kernel<G, 2>), grid, dim3(256), 0, s, c, o, f);
  else
    hipLaunchKernelGGL((moe_lora_finish_kernel<G, 1>), grid, dim3(256), 0, s, c, o, f);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora_decode(const LoraCall& c, bool kmajor, const ShrinkOut& o, const LoraLists& rows,
                              float* v, int v_parts, float* partial, int parts, hipStream_t s) {
  const FewRows f{(c.T + 15) / 16 * ((c.r + 15) / 16) * v_parts * 16, rows.counts ? c.L : 0, (c.N + 63) / 64,
                  parts, (c.T + 63) / 64, v_parts, v, partial};
  hipError_t e;
  if (c.T <= 16)
    e = kmajor ? launch<1, true>(c, o, rows, f, s) : launch<1, false>(c, o, rows, f, s);
  else if (c.T <= 32)
    e = kmajor ? launch<2, true>(c, o, rows, f, s) : launch<2, false>(c, o, rows, f, s);
  else
    e = kmajor ? launch<4, true>(c, o, rows, f, s) : launch<4, false>(c, o, rows, f, s);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((c.N + 255) / 256), (unsigned)c.T);
  if (kmajor) {
    hipLaunchKernelGGL(moe_lora_finish_kmajor_kernel, grid, dim3(256), 0, s, c, o, f);
    return hipGetLastError();
  }
  if (c.r <= 8) return launch_finish<1>(c, o, f, grid, s);
  if (c.r <= 16) return launch_finish<2>(c, o, f, grid, s);
  if (c.r <= 32) return launch_finish<4>(c, o, f, grid, s);
  if (c.r <= 64) return launch_finish<8>(c, o, f, grid, s);
  return launch_finish<16>(c, o, f, grid, s);
}

}  // namespace moe
