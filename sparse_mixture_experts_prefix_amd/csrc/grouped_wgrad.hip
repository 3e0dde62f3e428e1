// Weight gradients of the grouped products with ragged groups
// (moe_grouped_gemm_wgrad in moe.h): dW[g][n][k] = sum over the group's rows of
// dy[r][n] x[r][k], both operands read K-major (the rows are the reduction)
// through the transposing LDS reads.
//
// Many rows per group: the 256 x 256 x 64 tiles of gemm_tile.hpp, MFMA-bound.
// Few (mostly one K stage): 128 x 128 tiles, of which two share a CU, so that one's
// stores overlap the other's loads and products.  Also where 256 x 256 tiles would
// leave half the CUs idle: a tile walks its group's rows alone, the smaller one in
// less time (2 groups of 4367 rows, 216 x 128: 60 us against 105; 4 of 2048 rows, 1024 x
// 1024: 41 against 65; with 160 tiles, 10 of 205 rows, 18.4 against 17.4).  Up to a few hundred rows the time
// is the gradient's stores (4 G N K bytes).  They are non-temporal (nothing of a
// gradient this size stays in a cache: 541 -> 449 us for 64 x 2048 x 4096 at 156 rows
// each, held in a cache), and the tiles go in row order, so that what the chip stores
// at a time is whole rows (an eighth of the tiles per XCD instead: 602 us).
#include "gemm_tile.hpp"
#include "ops_launch.hpp"
#include "ragged.hpp"

namespace moe {
namespace {

constexpr int kAhead = 256;  // tiles that run at once
// Reads one word of each line of a share of the rows that the tiles one round ahead
// will load (tile t + ahead: its group's lines, dealt to that group's tiles), between a
// tile's products and its stores.  The stores keep the memory's queues full, and a
// group's first read behind them took several microseconds of every tile.
struct TouchAhead {
  const RaggedWgrad& p;
  int64_t t;
  __device__ __forceinline__ int before() const {
    const int64_t per = p.tiles_m * p.tiles_n;
    const int g = (int)(t / per);
    if (g >= p.E) return 0;
    const int64_t rows = group_rows(p, g), first = group_first(p, g);
    const int64_t la = (rows * p.lda + 63) / 64, lb = (rows * p.ldb + 63) / 64;  // 128-byte lines
    const uint16_t *A = p.A + first * p.lda, *B = p.B + first * p.ldb;
    int x = 0;
    for (int64_t i = (t - g * per) * 256 + threadIdx.x; i < la + lb; i += per * 256)
      x ^= i < la ? A[i * 64] : B[(i - la) * 64];
    return x;
  }
  __device__ __forceinline__ void after(int x) const { asm volatile("" ::"v"(x)); }
};

__global__ __launch_bounds__(256) void moe_grouped_wgrad_kernel(RaggedWgrad p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  wgrad_whole_tile<true>(p, blockIdx.x, lds, TouchAhead{p, (int64_t)blockIdx.x + kAhead});
}

// 128 x 128 tiles: 4 waves of 64 x 64 (2 x 2 MFMA blocks), two K stages of 64 rows.
constexpr int kSmallOp = 64 * 128 * 2;  // 16 KB: a stage of one operand
constexpr int kSmallLds = 2 * 2 * kSmallOp;
__global__ __launch_bounds__(256) void moe_grouped_wgrad_small_kernel(RaggedWgrad p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int64_t t = blockIdx.x, per = p.tiles_m * p.tiles_n;
  const int g = (int)(t / per);
  const int rem = (int)(t - g * per);
  const int m0 = rem / (int)p.tiles_n * 128, n0 = rem % (int)p.tiles_n * 128;
  const int M = p.M_routed, N = p.N_routed;
  const int64_t r0 = __builtin_amdgcn_readfirstlane(group_first(p, g));
  const int rows = __builtin_amdgcn_readfirstlane(group_rows(p, g));
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1, lr = lane & 31, kh = lane >> 5;
  const __amdgpu_buffer_rsrc_t rsA = make_rsrc(p.A + r0 * p.lda, (uint32_t)((int64_t)rows * p.lda * 2));
  const __amdgpu_buffer_rsrc_t rsB = make_rsrc(p.B + r0 * p.ldb, (uint32_t)((int64_t)rows * p.ldb * 2));
  // 1-KB block 4 wave + j of an operand's stage: 4 rows of 256 bytes, chunk c (8
  // columns) of row k at c ^ 4 (k % 4)
  auto issue_op = [&](const __amdgpu_buffer_rsrc_t rs, int c0, int lim, int64_t ld, int k0, char* st) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int kr = 4 * (wave * 4 + j) + (lane >> 4), c = c0 + 8 * kmaj_chunk(kr, lane & 15);
      const uint32_t off = k0 + kr < rows && c < lim ? (uint32_t)(k0 + kr) * (uint32_t)(ld * 2) + (uint32_t)c * 2 : kOob;
      lds_dma16(rs, st + (wave * 4 + j) * 1024, off, 0);
    }
  };
  auto issue = [&](int s) {
    char* st = lds + __builtin_amdgcn_readfirstlane((s & 1) * 2 * kSmallOp);
    issue_op(rsA, m0, M, p.lda, s * 64, st);
    issue_op(rsB, n0, N, p.ldb, s * 64, st + kSmallOp);
  };
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  typedef __attribute__((address_space(3))) char lds_char;
  auto read = [&](const char* st, int c0, int ks) {
    const int q = lane & 15, k = 16 * ks + 8 * kh + (q >> 2), c = c0 + 16 * ((lane >> 4) & 1) + 4 * (q & 3);
    const char* at = st + k * 256 + kmaj_chunk(k, c >> 3) * 16 + (c & 7) * 2;
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)((lds_char*)at));
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)((lds_char*)(at + 4 * 256)));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  f32x16 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  const int n = (rows + 63) / 64;
  if (n > 0) issue(0);
  for (int s = 0; s < n; ++s) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();  // stage s is whole; every wave has read stage s - 1
    asm volatile("" ::: "memory");
    if (s + 1 < n) issue(s + 1);
    const char* st = lds + (s & 1) * 2 * kSmallOp;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      bf16x8 a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) a[i] = read(st, wm * 64 + 32 * i, ks);
#pragma unroll
      for (int j = 0; j < 2; ++j) b[j] = read(st + kSmallOp, wn * 64 + 32 * j, ks);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma32(a[i], b[j], acc[i][j]);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this wave's reads of stage s are done
  }
  // register r of a block: row 8 (r / 4) + 4 kh + r % 4, column lr
  float* C = p.C_routed + (int64_t)g * M * N;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int m = m0 + wm * 64 + 32 * i + 8 * (r >> 2) + 4 * kh + (r & 3);
      if (m >= M) continue;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = n0 + wn * 64 + 32 * j + lr;
        if (c < N) __builtin_nontemporal_store(acc[i][j][r], C + (int64_t)m * N + c);
      }
    }
}

}  // namespace

hipError_t launch_grouped_wgrad(const moe_gemm_shape& s, const void* dy, const void* x,
                                const int32_t* offsets, float* dw, hipStream_t st) {
  static std::atomic<uint64_t> done[2];
  int ctas = 0;
  hipError_t e = split_ctas(&ctas);
  if (e != hipSuccess) return e;
  const int64_t large = (int64_t)s.G * ((s.N + BM - 1) / BM) * ((s.K + BM - 1) / BM);
  const bool small = (int64_t)s.R <= (int64_t)kWgradSmallRows * s.G || large * 2 <= ctas;
  const int ts = small ? 128 : BM, lds = small ? kSmallLds : kLdsBytes;
  void (*kernel)(RaggedWgrad) = small ? moe_grouped_wgrad_small_kernel : moe_grouped_wgrad_kernel;
  e = allow_lds(reinterpret_cast<const void*>(kernel), lds, done[small]);
  if (e != hipSuccess) return e;
  RaggedWgrad p{static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(x), s.N, s.K, s.N, s.K,
                s.G, offsets, s.R, dw, (s.N + ts - 1) / ts, (s.K + ts - 1) / ts};
  const int64_t tiles = s.G * p.tiles_m * p.tiles_n;
  hipLaunchKernelGGL(kernel, dim3((unsigned)tiles), dim3(256), lds, st, p);
  return hipGetLastError();
}

}  // namespace moe
