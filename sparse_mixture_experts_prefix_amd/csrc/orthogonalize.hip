// Orthogonalised updates by Newton-Schulz products (moe_orthogonalize in moe.h).
//
// Per step and matrix, m the smaller side, n the larger:
//   P = X X^T (or X^T X)      symmetric, m^2 n multiply-adds, half of them needed
//   Q = b P + c P P           symmetric, m^3, half needed
//   X' = a X + Q X (or X Q)   m^2 n
// Every product runs on MFMA tiles (256 x 256 x 64 with the K loop of gemm_tile.hpp;
// 128 x 128 or 64 x 64 where those would leave most CUs idle) in the layout X has: rows
// or columns as the reduction, so nothing is transposed.  The symmetric ones
// compute the tiles on and below the diagonal and store each twice.
//
// Numbers.  Operands are fp16 (11 bits; bf16's 8 showed 1 to 17% error on
// gradients of falling singular values) with power-of-two scales: X times
// S = 2^ceil(log2 sqrt(M N)) (at most 2^15: |X| stays below about 1.2), P and Q
// times SP = 2^13 (|P| <= 1.45, |Q| <= 2.81).  X is carried in two fp16 parts:
// the products read the upper one, and the step adds a (hi + lo), so the rounding of
// X does not feed the directions that later steps amplify by up to 3.4 each
// (with one part 1.5 to 5% error on such gradients, with two 0.2 to 0.4%,
// most of it the bf16 result's own rounding).
#include "gemm_tile.hpp"
#include "launch.hpp"
#include "ops_launch.hpp"
#include "ragged.hpp"

namespace moe {
namespace {

typedef _Float16 f16;
typedef f16 f16x4 __attribute__((ext_vector_type(4)));

constexpr float kA = 3.4445f, kB = -4.7750f, kC = 2.0315f;
constexpr float kSP = 8192.f;

// -------------------------------------------------------- norm and first X
__device__ __forceinline__ float g_at(const void* g, int dtype, int64_t i) {
  return dtype == MOE_DTYPE_F32 ? static_cast<const float*>(g)[i]
                                : bf16_to_f32(static_cast<const bf16_t*>(g)[i]);
}

// eight consecutive values (the matrices' sizes are multiples of 8)
__device__ __forceinline__ void load8(const void* g, int dtype, int64_t i, float (&v)[8]) {
  if (dtype == MOE_DTYPE_F32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(g) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const u32x4 q = ld16(static_cast<const bf16_t*>(g) + i);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      v[2 * h] = __builtin_bit_cast(float, q[h] << 16);
      v[2 * h + 1] = __builtin_bit_cast(float, q[h] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ void load4(const void* g, int dtype, int64_t i, float (&v)[4]) {
  if (dtype == MOE_DTYPE_F32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(g) + i);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  } else {
    const uint64_t q = *reinterpret_cast<const uint64_t*>(static_cast<const bf16_t*>(g) + i);
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = bf16_to_f32((bf16_t)(q >> (16 * u)));
  }
}

// part[e][b] = sum of squares of block b's share of matrix e, in double so that no
// gradient's squares under- or overflow; fixed order.  Bound by reading G.
__global__ __launch_bounds__(256) void moe_orth_norm_kernel(const void* g, int dtype, int64_t mn, double* part) {
  __shared__ double sum[4];
  const int64_t base = (int64_t)blockIdx.y * mn;
  double s = 0;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < mn; i += (int64_t)gridDim.x * 2048) {
    float v[8];
    load8(g, dtype, base + i, v);
#pragma unroll
    for (int u = 0; u < 8; ++u) s = fma((double)v[u], (double)v[u], s);
  }
  for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
  if ((threadIdx.x & 63) == 0) sum[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0)
    part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = ((sum[0] + sum[1]) + sum[2]) + sum[3];
}

// hi + lo = S G / (|G| + eps), zeros for a matrix of zeros
__global__ __launch_bounds__(256) void moe_orth_scale_kernel(const void* g, int dtype, int64_t mn,
                                                             const double* part, int parts, float eps,
                                                             float S, f16* hi, f16* lo) {
  const int64_t e = blockIdx.y;
  double s = 0;
  for (int b = 0; b < parts; ++b) s += part[e * parts + b];
  const double d = sqrt(s) + (double)eps;
  const double f = d > 0 ? (double)S / d : 0.0 * d;  // NaN stays NaN
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; i < mn; i += (int64_t)gridDim.x * 2048) {
    float v[8];
    load8(g, dtype, e * mn + i, v);
    f16x8 h, l;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float x = (float)((double)v[u] * f);
      h[u] = (f16)x;
      l[u] = (f16)(x - (float)h[u]);
    }
    *reinterpret_cast<f16x8*>(hi + e * mn + i) = h;
    *reinterpret_cast<f16x8*>(lo + e * mn + i) = l;
  }
}

// ----------------------------------------------------------------- products
// C = A B^T per matrix, A: M rows, B: N rows of K values; row-major operands have
// K contiguous ([rows][K]), K-major ones are [K][rows].  sym: C is symmetric (M = N).
// Results: sym: d0 = alpha acc (+ beta c0 when set); else with v = alpha acc +
// beta (c0 + c1): out = bf16(gamma v) when set, or d0 + d1 = v in two parts.
struct OrthProduct {
  const f16 *A, *B;
  int64_t sA, sB;  // elements per matrix
  int lda, ldb;
  int M, N, K, sym;
  int tm, tn, per;     // tiles down, across and per matrix
  int64_t n_dp;        // tiles run whole (the first ones)
  int R, S;            // tiles cut along K, pieces each
  float* partial;      // [R][S][tile][tile]
  const f16 *c0, *c1;
  f16 *d0, *d1;
  bf16_t* out;
  float alpha, beta, gamma;
};

// Tile t of a matrix: m-tile, n-tile.  sym: the tiles on and below the diagonal, row
// by row; a ragged last m-tile then meets every n-tile as the shorter operand.
// Else blocks of 4 m-tiles x 8 n-tiles, m fastest, for operand reuse in L2.
__device__ __forceinline__ void orth_coords(const OrthProduct& p, int t, int& i, int& j) {
  if (p.sym) {
    i = (int)((sqrtf(8.f * t + 1.f) - 1.f) * 0.5f);
    while (i * (i + 1) / 2 > t) --i;
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    j = t - i * (i + 1) / 2;
    return;
  }
  const int col = t / (p.tm * 8), u = t - col * p.tm * 8;  // columns of 8 n-tiles
  const int cw = min(8, p.tn - col * 8);
  const int blk = u / (4 * cw), v = u - blk * 4 * cw;
  const int mh = min(4, p.tm - blk * 4);
  i = blk * 4 + v % mh;
  j = col * 8 + v / mh;
}

struct OrthTile {
  int e, m0, n0, s0, s1;  // matrix, corner, K stages [s0, s1)
  int piece;              // index of the partial tile, or -1
};

// Workgroup b's tile: whole tiles in 8 runs, one per XCD (workgroup b runs on XCD
// b % 8), then the pieces.  False: nothing to do.
template <int TS>
__device__ __forceinline__ bool orth_tile(const OrthProduct& p, int64_t b, OrthTile& t) {
  const int64_t run = (p.n_dp + 7) / 8;
  int64_t L;
  int part = 0;
  t.piece = -1;
  if (b < 8 * run) {
    L = (b % 8) * run + b / 8;
    if (L >= p.n_dp) return false;
  } else {
    const int64_t q = b - 8 * run;
    if (q >= (int64_t)p.R * p.S) return false;
    L = p.n_dp + q % p.R;
    part = (int)(q / p.R);
    t.piece = (int)(q % p.R) * p.S + part;
  }
  t.e = (int)(L / p.per);
  int i, j;
  orth_coords(p, (int)(L - (int64_t)t.e * p.per), i, j);
  t.m0 = i * TS;
  t.n0 = j * TS;
  const int nk = (p.K + BK - 1) / BK;
  t.s0 = t.piece < 0 ? 0 : (int)((int64_t)part * nk / p.S);
  t.s1 = t.piece < 0 ? nk : (int)((int64_t)(part + 1) * nk / p.S);
  return true;
}

// The addends of eight results (c0, and c1 where SYM is false, at element i), and the
// results: all reads and writes are 16 bytes wide.
template <bool SYM>
struct Addend {
  f16x8 h, l;
};
template <>
struct Addend<true> {
  f16x8 h;
};
template <bool SYM>
__device__ __forceinline__ Addend<SYM> load_addend(const OrthProduct& p, int64_t i, bool in) {
  Addend<SYM> a;
#pragma unroll
  for (int u = 0; u < 8; ++u) a.h[u] = (f16)0.f;
  if constexpr (SYM) {
    if (in && p.c0) a.h = *reinterpret_cast<const f16x8*>(p.c0 + i);
  } else {
    a.l = a.h;
    if (in) {
      a.h = *reinterpret_cast<const f16x8*>(p.c0 + i);
      a.l = *reinterpret_cast<const f16x8*>(p.c1 + i);
    }
  }
  return a;
}
// v becomes the result
template <bool SYM>
__device__ __forceinline__ void emit8(const OrthProduct& p, int64_t i, const Addend<SYM>& a, float (&v)[8]) {
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    float x = (float)a.h[u];
    if constexpr (!SYM) x += (float)a.l[u];
    v[u] = fmaf(p.beta, x, v[u] * p.alpha);
  }
  if constexpr (!SYM) {
    if (p.out) {
      u32x4 w;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        w[u] = (uint32_t)f32_to_bf16(v[2 * u] * p.gamma) | ((uint32_t)f32_to_bf16(v[2 * u + 1] * p.gamma) << 16);
      st16(p.out + i, w);
      return;
    }
  }
  f16x8 h;
#pragma unroll
  for (int u = 0; u < 8; ++u) h[u] = (f16)v[u];
  *reinterpret_cast<f16x8*>(p.d0 + i) = h;
  if constexpr (!SYM) {
    f16x8 l;
#pragma unroll
    for (int u = 0; u < 8; ++u) l[u] = (f16)(v[u] - (float)h[u]);
    *reinterpret_cast<f16x8*>(p.d1 + i) = l;
  }
}

// The results of ROWS x TS accumulators at rows m, columns n: fill(tile) writes them to
// LDS (fp32, rows of TS + 8 so that row and column accesses spread over the banks),
// from where they leave in 16-byte rows; mirror: also as rows of the transposed place.
// A tile's end is not hidden behind another tile (the accumulators allow one
// workgroup per CU), so its waits count: all addends of the piece are requested before
// the accumulators go to LDS, and the transposed rows are made of finished results.
// (Addends loaded four at a time as they were needed, and again for the transposed
// place: a third of the X step's time and 40% of the symmetric products'.)
template <int TS>
constexpr int tile_pitch() { return TS + 8; }
template <bool SYM, int ROWS, int TS, class Fill>
__device__ __forceinline__ void emit_tile(const OrthProduct& p, int64_t at, int m, int n, float* tile, bool mirror,
                                          Fill fill) {
  const int rows = min(ROWS, p.M - m), cols = min(TS, p.N - n);  // multiples of 8
  constexpr int PIECES = (ROWS * TS / 8 + 255) / 256;  // (past ROWS: past `rows` too)
  Addend<SYM> a[PIECES];
  const int64_t base = at + (int64_t)m * p.N + n;
#pragma unroll
  for (int u = 0; u < PIECES; ++u) {
    const int q = u * 256 + threadIdx.x, r = q / (TS / 8), c = q % (TS / 8) * 8;
    a[u] = load_addend<SYM>(p, base + (int64_t)r * p.N + c, r < rows && c < cols);
  }
  fill(tile);
  __syncthreads();
#pragma unroll
  for (int u = 0; u < PIECES; ++u) {
    const int q = u * 256 + threadIdx.x, r = q / (TS / 8), c = q % (TS / 8) * 8;
    if (r >= rows || c >= cols) continue;
    float* src = tile + r * tile_pitch<TS>() + c;
    float v[8];
    const float4 x = *reinterpret_cast<const float4*>(src);
    const float4 y = *reinterpret_cast<const float4*>(src + 4);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    emit8<SYM>(p, base + (int64_t)r * p.N + c, a[u], v);
    if constexpr (SYM) {
      if (mirror) {
        *reinterpret_cast<float4*>(src) = float4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<float4*>(src + 4) = float4{v[4], v[5], v[6], v[7]};
      }
    }
  }
  if constexpr (SYM) {
    if (!mirror) return;
    __syncthreads();
#pragma unroll 4
    for (int u = 0; u < PIECES; ++u) {
      const int q = u * 256 + threadIdx.x, c = q % TS, r = q / TS * 8;
      if (r >= rows || c >= cols) continue;
      f16x8 h;
#pragma unroll
      for (int w = 0; w < 8; ++w) h[w] = (f16)tile[(r + w) * tile_pitch<TS>() + c];
      *reinterpret_cast<f16x8*>(p.d0 + at + (int64_t)(n + c) * p.N + m + r) = h;
    }
  }
}

// 256 x 256 tiles.  KB: B is K-major, KA: A is too.
template <bool KA, bool KB, bool SYM>
__global__ __launch_bounds__(256) void moe_orth_tile256_kernel(OrthProduct p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  OrthTile t;
  if (!orth_tile<256>(p, blockIdx.x, t)) return;
  const int lane = threadIdx.x & 63, sub = lane >> 3;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int valid = min(256, p.M - t.m0);
  const __amdgpu_buffer_rsrc_t rsA =
      make_rsrc(p.A + t.e * p.sA, (uint32_t)((KA ? p.K : p.M) * p.lda * 2));
  const __amdgpu_buffer_rsrc_t rsB =
      make_rsrc(p.B + t.e * p.sB, (uint32_t)((KB ? p.K : p.N) * p.ldb * 2));
  // load slots as in prefill_tile (rows) and wgrad_issue (K-major)
  uint32_t offA[8], offB[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int kr = 2 * (wave * 8 + j) + (lane >> 5), kc = 8 * kmaj_chunk(kr, lane & 31);
    const int ra = (j * 4 + wave) * 8 + sub, rb = (wave * 8 + j) * 8 + sub;
    if (KA)
      offA[j] = t.m0 + kc < p.M ? (uint32_t)((kr * p.lda + t.m0 + kc) * 2) : kOob;
    else
      offA[j] = ra < valid ? (uint32_t)(((t.m0 + ra) * p.lda + 8 * ((lane & 7) ^ swz(ra))) * 2) : kOob;
    if (KB)
      offB[j] = t.n0 + kc < p.N ? (uint32_t)((kr * p.ldb + t.n0 + kc) * 2) : kOob;
    else
      offB[j] = t.n0 + rb < p.N ? (uint32_t)(((t.n0 + rb) * p.ldb + 8 * ((lane & 7) ^ swz(rb))) * 2) : kOob;
  }
  auto issue = [&](bool isB, int stage, int buf, int j0, int j1) {
    const int k0 = stage * BK;
    const bool kmaj = isB ? KB : KA;
    const bool tail = k0 + BK > p.K;
    char* base = isB ? lds + 2 * kABytes + buf * kBBytes : lds + buf * kABytes;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j < j0 || j >= j1) continue;
      uint32_t o = isB ? offB[j] : offA[j];
      const int blk = isB || kmaj ? wave * 8 + j : j * 4 + wave;
      if (tail) {
        if (kmaj) {
          if (k0 + 2 * (wave * 8 + j) + (lane >> 5) >= p.K) o = kOob;
        } else if (k0 + 8 * ((lane & 7) ^ swz(blk * 8 + sub)) >= p.K) {
          o = kOob;
        }
      }
      const uint32_t soff = (uint32_t)(kmaj ? k0 * (isB ? p.ldb : p.lda) * 2 : k0 * 2);
      if (KA || KB)
        lds_dma16(isB ? rsB : rsA, base + blk * 1024, o, soff);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(isB ? rsB : rsA, (lds_void*)(base + blk * 1024), 16, o,
                                                 (int)soff, 0, 0);
    }
  };
  auto issue_a = [&](int stage, int buf, int j0, int j1) { issue(false, stage, buf, j0, j1); };
  auto issue_b = [&](int stage, int buf, int j0, int j1) { issue(true, stage, buf, j0, j1); };
  f32x16 acc[4][4];
  zero_acc(acc);
  const int n = t.s1 - t.s0;
  const bool il = !KA && valid < 256;
  int act = 4;
  if constexpr (KA) {
    k_loop<false, 4, false, decltype(issue_a), decltype(issue_b), true, true, false, 8, false, 0, true>(
        lds, t.s0, n, wm, wn, il, lane, issue_a, issue_b, acc);
  } else {
    // a ragged last m-tile skips the loads and products of its missing rows (see prefill_tile)
    if (il) act = min(4, max(0, ((valid + 31) / 32 - wm + 1) / 2));
    const int tier = min(4, max(1, (valid + 63) / 64));
#define MOE_KL(A_, N_)                                                                             \
  k_loop<false, A_, false, decltype(issue_a), decltype(issue_b), KB, false, false, N_, false, 0, true>( \
      lds, t.s0, n, wm, wn, il, lane, issue_a, issue_b, acc)
    switch (tier * 8 + act) {
      case 4 * 8 + 4: MOE_KL(4, 8); break;
      case 4 * 8 + 3: MOE_KL(3, 8); break;
      case 3 * 8 + 3: MOE_KL(3, 6); break;
      case 3 * 8 + 2: MOE_KL(2, 6); break;
      case 2 * 8 + 2: MOE_KL(2, 4); break;
      case 2 * 8 + 1: MOE_KL(1, 4); break;
      case 1 * 8 + 1: MOE_KL(1, 2); break;
      default: MOE_KL(0, 2); break;
    }
#undef MOE_KL
  }
  const int lr = lane & 31, kh = lane >> 5;
  if (t.piece >= 0) {
    float* P = p.partial + (int64_t)t.piece * 65536;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= act) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          P[(a_row_of(wm, i, il) + 8 * (r >> 2) + 4 * kh + (r & 3)) * 256 + b_row_of<false>(wn, j) + lr] =
              acc[i][j][r];
    }
    return;
  }
  // the K loop's LDS takes the results, 128 rows at a time
  float* tile = reinterpret_cast<float*>(lds);
  static_assert(128 * tile_pitch<256>() * 4 <= kLdsBytes, "half a tile of results must fit");
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (half * 128 >= valid) break;
    __syncthreads();  // the K loop's reads, or the first half's, are done
    emit_tile<SYM, 128, 256>(
        p, (int64_t)t.e * p.M * p.N, t.m0 + 128 * half, t.n0, tile, SYM && t.m0 != t.n0, [&](float* d) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = a_row_of(wm, i, il) - 128 * half;
            if (row < 0 || row >= 128) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int r = 0; r < 16; ++r)
                d[(row + 8 * (r >> 2) + 4 * kh + (r & 3)) * tile_pitch<256>() + b_row_of<false>(wn, j) + lr] =
                    acc[i][j][r];
          }
        });
  }
}

// 128 x 128 or 64 x 64 tiles (TS): 4 waves of 2 x 2 or one MFMA block of 32 x 32, three
// K stages of 32 or 16 KB in LDS, two of them in flight.  Taken where the larger tiles
// are too few for the chip; what a launch takes then is one tile's chain of loads,
// products and stores, which the smaller tile shortens: 7 to 12 us with TS 128, 4 to 6
// with TS 64 for matrices of a few hundred rows and columns.
template <int TS>
constexpr int small_stage_bytes() { return 2 * TS * BK * 2; }
// K-major rows of 64 columns are 128 bytes: chunk c of k-row k sits at c ^ 4 (k / 2 % 2), so
// that the four k-rows of a transposing read hit every bank once; of 128 columns as kmaj_chunk
template <int TS>
__device__ __forceinline__ int small_chunk(int k, int c) {
  return TS == 128 ? kmaj_chunk(k, c) : c ^ (4 * ((k >> 1) & 1));
}
template <int TS, bool KA, bool KB, bool SYM>
__global__ __launch_bounds__(256) void moe_orth_tile_kernel(OrthProduct p) {
  constexpr int SB = small_stage_bytes<TS>(), NB = TS / 64, CH = TS / 8;  // MFMA blocks a side; chunks of a k-row
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  OrthTile t;
  if (!orth_tile<TS>(p, blockIdx.x, t)) return;
  const int lane = threadIdx.x & 63, sub = lane >> 3;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int lr = lane & 31, kh = lane >> 5;
  const __amdgpu_buffer_rsrc_t rsA =
      make_rsrc(p.A + t.e * p.sA, (uint32_t)((KA ? p.K : p.M) * p.lda * 2));
  const __amdgpu_buffer_rsrc_t rsB =
      make_rsrc(p.B + t.e * p.sB, (uint32_t)((KB ? p.K : p.N) * p.ldb * 2));
  // a stage's operand is TS / 8 blocks of 1 KB, a quarter per wave: 8 rows of 128 bytes,
  // or (K-major) k-rows of 2 TS bytes
  auto issue_op = [&](const __amdgpu_buffer_rsrc_t rs, bool kmaj, int r0, int rows, int ld, int stage, char* st) {
    const int k0 = stage * BK;
#pragma unroll
    for (int j = 0; j < TS / 32; ++j) {
      const int blk = wave * (TS / 32) + j;
      uint32_t o;
      if (kmaj) {
        const int kr = blk * (64 / CH) + lane / CH, k = k0 + kr, c = r0 + 8 * small_chunk<TS>(kr, lane % CH);
        o = k < p.K && c < rows ? (uint32_t)((k * ld + c) * 2) : kOob;
      } else {
        const int r = blk * 8 + sub, k = k0 + 8 * ((lane & 7) ^ swz(r));
        o = k < p.K && r0 + r < rows ? (uint32_t)(((r0 + r) * ld + k) * 2) : kOob;
      }
      lds_dma16(rs, st + blk * 1024, o, 0);
    }
  };
  auto issue = [&](int stage, int buf) {
    char* st = lds + __builtin_amdgcn_readfirstlane(buf * SB);
    issue_op(rsA, KA, t.m0, p.M, p.lda, stage, st);
    issue_op(rsB, KB, t.n0, p.N, p.ldb, stage, st + SB / 2);
  };
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  typedef __attribute__((address_space(3))) char lds_char;
  auto read = [&](const char* st, bool kmaj, int r0, int ks) {
    if (kmaj) {
      const int q = lane & 15, k = 16 * ks + 8 * kh + (q >> 2), c = r0 + 16 * ((lane >> 4) & 1) + 4 * (q & 3);
      const char* at = st + k * (2 * TS) + small_chunk<TS>(k, c >> 3) * 16 + (c & 7) * 2;
      const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)((lds_char*)at));
      const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)((lds_char*)(at + 4 * 2 * TS)));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    const int r = r0 + lr;
    return *reinterpret_cast<const bf16x8*>(st + r * 128 + ((2 * ks + kh) ^ swz(r)) * 16);
  };
  f32x16 acc[NB][NB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  const int n = t.s1 - t.s0;
  issue(t.s0, 0);
  if (n > 1) issue(t.s0 + 1, 1);
  int buf = 0;
  for (int s = 0; s < n; ++s) {
    if (s + 1 < n && TS == 128)
      asm volatile("s_waitcnt vmcnt(8)" ::: "memory");  // stage s landed, s + 1 may fly
    else if (s + 1 < n)
      asm volatile("s_waitcnt vmcnt(4)" ::: "memory");
    else
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();  // every wave's part of stage s; all have left stage s - 1
    asm volatile("" ::: "memory");
    const int b2 = buf == 0 ? 2 : buf - 1;
    if (s + 2 < n) issue(t.s0 + s + 2, b2);
    const char* sa = lds + buf * SB;
    const char* sb = sa + SB / 2;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      bf16x8 a[NB], b[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i) a[i] = read(sa, KA, wm * (TS / 2) + 32 * i, ks);
#pragma unroll
      for (int j = 0; j < NB; ++j) b[j] = read(sb, KB, wn * (TS / 2) + 32 * j, ks);
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < NB; ++j) acc[i][j] = mfma32<true>(a[i], b[j], acc[i][j]);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this wave's reads of stage s are done
    buf = buf == 2 ? 0 : buf + 1;
  }
  if (t.piece >= 0) {
    float* P = p.partial + (int64_t)t.piece * (TS * TS);
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          P[(wm * (TS / 2) + 32 * i + 8 * (r >> 2) + 4 * kh + (r & 3)) * TS + wn * (TS / 2) + 32 * j + lr] = acc[i][j][r];
    return;
  }
  float* tile = reinterpret_cast<float*>(lds);
  static_assert(TS * tile_pitch<TS>() * 4 <= 3 * SB, "the results must fit");
  __syncthreads();  // the last stage's reads are done
  emit_tile<SYM, TS, TS>(p, (int64_t)t.e * p.M * p.N, t.m0, t.n0, tile, SYM && t.m0 != t.n0, [&](float* d) {
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          d[(wm * (TS / 2) + 32 * i + 8 * (r >> 2) + 4 * kh + (r & 3)) * tile_pitch<TS>() + wn * (TS / 2) + 32 * j + lr] =
              acc[i][j][r];
  });
}

// Finishes the cut tiles, 16 rows of one per workgroup: the pieces' sums are added
// in K order.
template <int TS, bool SYM>
__global__ __launch_bounds__(256) void moe_orth_fixup_kernel(OrthProduct p) {
  __shared__ float tile[16 * tile_pitch<TS>()];
  const int k = blockIdx.x / (TS / 16), r0 = blockIdx.x % (TS / 16) * 16;
  const int64_t L = p.n_dp + k;
  const int e = (int)(L / p.per);
  int ti, tj;
  orth_coords(p, (int)(L - (int64_t)e * p.per), ti, tj);
  if (ti * TS + r0 >= p.M) return;
  const float* P = p.partial + ((int64_t)k * p.S * TS + r0) * TS;
  emit_tile<SYM, 16, TS>(p, (int64_t)e * p.M * p.N, ti * TS + r0, tj * TS, tile, SYM && ti != tj, [&](float* d) {
    for (int q = threadIdx.x; q < 16 * TS / 4; q += 256) {
      const float4* src = reinterpret_cast<const float4*>(P) + q;
      float4 a = src[0];
      for (int s = 1; s < p.S; ++s) {
        const float4 b = src[(int64_t)s * TS * TS / 4];
        a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
      }
      *reinterpret_cast<float4*>(d + q * 4 / TS * tile_pitch<TS>() + q * 4 % TS) = a;
    }
  });
}

// --------------------------------------------------- one matrix per workgroup
// All steps of a small matrix (m <= 128, n <= 256) in one workgroup: X in fp32
// registers (in the layout of the X step's results, whose sums start from a X), its
// fp16 copy, P and Q in LDS.  A tall matrix is loaded and stored transposed.  Rows and
// columns past m and n are zeros and stay zeros.  Bound by the chain of products of one
// tile each and the vector work between them (conversions of up to 128 results per
// lane): 8 matrices of 256 x 128 take 48 us, in 17 launches of 64 x 64 tiles 67 us;
// 64 of 128 x 256 47 us against 89 us.
constexpr int kSmallM = 128, kSmallN = 256;
constexpr int kPitchX = kSmallN + 8, kPitchP = kSmallM + 8;  // fp16 elements; 16-byte reads of 16 rows spread
constexpr int kSmallLds = (kSmallM * kPitchX + 2 * kSmallM * kPitchP) * 2 + 64;
template <int dtype>
__global__ __launch_bounds__(256) void moe_orth_small_kernel(const void* g, int M, int N, int steps, float eps,
                                                             float S, bf16_t* out) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  f16* X = reinterpret_cast<f16*>(lds);
  f16* P = X + kSmallM * kPitchX;
  f16* Q = P + kSmallM * kPitchP;
  double* sum = reinterpret_cast<double*>(Q + kSmallM * kPitchP);
  const int lane = threadIdx.x & 63, lr = lane & 31, kh = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const bool tall = M > N;
  const int m = tall ? N : M, n = tall ? M : N;
  const int64_t base = (int64_t)blockIdx.x * M * N;
  // Blocks are computed transposed (operands exchanged), so that a lane's four
  // consecutive registers are four consecutive elements of a row in LDS: block (i, j) of
  // this wave: row 64 wm + 32 i + lr of X, registers 4 q .. 4 q + 3 its columns
  // 128 wn + 32 j + 8 q + 4 kh .. + 3 (P and Q: 64 wn + ..).
  f32x16 x[2][4];
  double sq = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = 64 * wm + 32 * i + lr, c = 128 * wn + 32 * j + 8 * q + 4 * kh;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (row < m && c < n) {  // n is a multiple of 8: four columns are in or out together
          if (tall) {
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = g_at(g, dtype, base + (int64_t)(c + u) * N + row);
          } else {
            load4(g, dtype, base + (int64_t)row * N + c, v);
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          x[i][j][4 * q + u] = v[u];
          sq = fma((double)v[u], (double)v[u], sq);
        }
      }
  for (int o = 32; o; o >>= 1) sq += __shfl_xor(sq, o);
  if (lane == 0) sum[wave] = sq;
  __syncthreads();
  const double d = sqrt(((sum[0] + sum[1]) + sum[2]) + sum[3]) + (double)eps;
  const double f = d > 0 ? (double)S / d : 0.0 * d;  // NaN stays NaN
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) x[i][j][r] = (float)((double)x[i][j][r] * f);
  auto row_frag = [&](const f16* a, int pitch, int r0, int ks) {  // 8 consecutive k of row r0 + lr
    return *reinterpret_cast<const bf16x8*>(a + (r0 + lr) * pitch + 16 * ks + 8 * kh);
  };
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  typedef __attribute__((address_space(3))) char lds_char;
  auto col_frag = [&](int c0, int ks) {  // 8 consecutive rows of X's column c0 + lr (transposing reads)
    const int q = lane & 15;
    const f16* at = X + (16 * ks + 8 * kh + (q >> 2)) * kPitchX + c0 + 16 * ((lane >> 4) & 1) + 4 * (q & 3);
    const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)((lds_char*)at));
    const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)((lds_char*)(at + 4 * kPitchX)));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto put4 = [](f16* at, float a, float b, float c, float e) {
    *reinterpret_cast<f16x4*>(at) = f16x4{(f16)a, (f16)b, (f16)c, (f16)e};
  };
  // acc = A A^T over k steps of 16, this wave's 64 x 64 of 128 x 128
  auto square = [&](const f16* a, int pitch, int ksteps, f32x16 (&acc)[2][2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
#pragma unroll 4
    for (int ks = 0; ks < ksteps; ++ks) {
      bf16x8 fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) fa[i] = row_frag(a, pitch, 64 * wm + 32 * i, ks);
#pragma unroll
      for (int j = 0; j < 2; ++j) fb[j] = row_frag(a, pitch, 64 * wn + 32 * j, ks);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma32<true>(fb[j], fa[i], acc[i][j]);
    }
  };
  const int kn = (n + 15) / 16, km = (m + 15) / 16;
  const float scale_p = kSP / (S * S);
  for (int s = 0; s < steps; ++s) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          put4(X + (64 * wm + 32 * i + lr) * kPitchX + 128 * wn + 32 * j + 8 * q + 4 * kh, x[i][j][4 * q],
               x[i][j][4 * q + 1], x[i][j][4 * q + 2], x[i][j][4 * q + 3]);
    __syncthreads();
    f32x16 acc[2][2];
    square(X, kPitchX, kn, acc);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          put4(P + (64 * wm + 32 * i + lr) * kPitchP + 64 * wn + 32 * j + 8 * q + 4 * kh,
               acc[i][j][4 * q] * scale_p, acc[i][j][4 * q + 1] * scale_p, acc[i][j][4 * q + 2] * scale_p,
               acc[i][j][4 * q + 3] * scale_p);
    __syncthreads();
    square(P, kPitchP, km, acc);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int at = (64 * wm + 32 * i + lr) * kPitchP + 64 * wn + 32 * j + 8 * q + 4 * kh;
          const f16x4 pv = *reinterpret_cast<const f16x4*>(P + at);
          float v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) v[u] = fmaf(kB, (float)pv[u], acc[i][j][4 * q + u] * (kC / kSP));
          put4(Q + at, v[0], v[1], v[2], v[3]);
        }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][j] *= kA * kSP;
#pragma unroll 4
    for (int ks = 0; ks < km; ++ks) {
      bf16x8 fa[2], fb[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) fa[i] = row_frag(Q, kPitchP, 64 * wm + 32 * i, ks);
#pragma unroll
      for (int j = 0; j < 4; ++j) fb[j] = col_frag(128 * wn + 32 * j, ks);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = mfma32<true>(fb[j], fa[i], x[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][j] *= 1.f / kSP;
    __syncthreads();  // X, P and Q are read before the next step writes them
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = 64 * wm + 32 * i + lr, c = 128 * wn + 32 * j + 8 * q + 4 * kh;
        if (row >= m || c >= n) continue;
        bf16_t v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = f32_to_bf16(x[i][j][4 * q + u] * (1.f / S));
        if (tall) {
#pragma unroll
          for (int u = 0; u < 4; ++u) out[base + (int64_t)(c + u) * N + row] = v[u];
        } else {
          *reinterpret_cast<uint64_t*>(out + base + (int64_t)row * N + c) =
              (uint64_t)v[0] | ((uint64_t)v[1] << 16) | ((uint64_t)v[2] << 32) | ((uint64_t)v[3] << 48);
        }
      }
}

template <int TS, bool KA, bool KB, bool SYM>
hipError_t launch_tiles(const OrthProduct& p, hipStream_t s) {
  static std::atomic<uint64_t> done;
  constexpr int lds = TS == 256 ? kLdsBytes : 3 * small_stage_bytes<TS>();
  void (*kernel)(OrthProduct);
  if constexpr (TS == 256)
    kernel = moe_orth_tile256_kernel<KA, KB, SYM>;
  else
    kernel = moe_orth_tile_kernel<TS, KA, KB, SYM>;
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), lds, done);
  if (e != hipSuccess) return e;
  const int64_t blocks = (p.n_dp + 7) / 8 * 8 + (int64_t)p.R * p.S;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), lds, s, p);
  if (p.R)
    hipLaunchKernelGGL((moe_orth_fixup_kernel<TS, SYM>), dim3((unsigned)(p.R * (TS / 16))), dim3(256), 0, s, p);
  return hipGetLastError();
}

// Tile size, and which tiles are cut along K (E matrices; ctas CUs).
template <bool KA, bool KB, bool SYM>
hipError_t launch_product(OrthProduct p, int E, int ctas, hipStream_t s) {
  auto tiles = [&](int ts) {
    p.tm = (p.M + ts - 1) / ts;
    p.tn = (p.N + ts - 1) / ts;
    p.per = SYM ? p.tm * (p.tm + 1) / 2 : p.tm * p.tn;
    return (int64_t)E * p.per;
  };
  // half the chip's CUs with 256 x 256 tiles, or smaller ones that reach more CUs; 64 x 64
  // where 128 x 128 do not reach all (8 matrices of 512 x 512 160 us against 235, 2 of
  // 400 x 392 102 against 178; where the chip is filled they have half the reuse)
  int64_t V = tiles(256);
  int ts = 256;
  if (V * 2 < ctas) V = tiles(ts = 128);
  if (ts == 128 && V < ctas) V = tiles(ts = 64);
  // the partial last round, cut along K in pieces of at least 4 stages
  const int64_t rounds = V / ctas;
  int64_t R = V % ctas;
  const int64_t by_k = ((p.K + BK - 1) / BK) / kMinPieceStages;
  int64_t S = R ? ctas / R : 1;
  if (S > by_k) S = by_k;
  if (S > 16) S = 16;
  if (S < 2 || rounds >= kSplitRounds || R * S * ts * ts > kOrthPartialFloats) R = 0, S = 1;
  p.n_dp = V - R;
  p.R = (int)R;
  p.S = (int)S;
  if (ts == 64) return launch_tiles<64, KA, KB, SYM>(p, s);
  return ts == 128 ? launch_tiles<128, KA, KB, SYM>(p, s) : launch_tiles<256, KA, KB, SYM>(p, s);
}

}  // namespace

hipError_t launch_orthogonalize(int E, int M, int N, const OrthPlan& plan, const void* g, int g_dtype,
                                int steps, float eps, void* out, void* ws, hipStream_t st) {
  if (plan.m <= kSmallM && plan.n <= kSmallN) {
    static std::atomic<uint64_t> done[2];
    const bool f32 = g_dtype == MOE_DTYPE_F32;
    auto* kernel = f32 ? moe_orth_small_kernel<MOE_DTYPE_F32> : moe_orth_small_kernel<MOE_DTYPE_BF16>;
    const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), kSmallLds, done[f32]);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3((unsigned)E), dim3(256), kSmallLds, st, g, M, N, steps, eps, plan.scale,
                       static_cast<bf16_t*>(out));
    return hipGetLastError();
  }
  char* w = static_cast<char*>(ws);
  f16* hi[2] = {reinterpret_cast<f16*>(w + plan.off_hi[0]), reinterpret_cast<f16*>(w + plan.off_hi[1])};
  f16* lo = reinterpret_cast<f16*>(w + plan.off_lo);
  f16* P = reinterpret_cast<f16*>(w + plan.off_p);
  f16* Q = reinterpret_cast<f16*>(w + plan.off_q);
  double* part = reinterpret_cast<double*>(w + plan.off_norm);
  int ctas = 0;
  hipError_t e = split_ctas(&ctas);
  if (e != hipSuccess) return e;
  const int64_t mn = (int64_t)M * N;
  const int m = plan.m, n = plan.n;
  const float S = plan.scale;
  const dim3 grid((unsigned)plan.norm_parts, (unsigned)E);
  hipLaunchKernelGGL(moe_orth_norm_kernel, grid, dim3(256), 0, st, g, g_dtype, mn, part);
  const int64_t sb = (mn / 8 + 255) / 256;
  hipLaunchKernelGGL(moe_orth_scale_kernel, dim3((unsigned)(sb < 1024 ? sb : 1024), (unsigned)E), dim3(256), 0, st,
                     g, g_dtype, mn, part, plan.norm_parts, eps, S, hi[0], lo);
  e = hipGetLastError();
  for (int i = 0; i < steps && e == hipSuccess; ++i) {
    const f16* X = hi[i & 1];
    OrthProduct gram{};
    gram.A = gram.B = X;
    gram.sA = gram.sB = mn;
    gram.lda = gram.ldb = N;
    gram.M = gram.N = m;
    gram.K = n;
    gram.sym = 1;
    gram.partial = reinterpret_cast<float*>(w + plan.off_partial);
    gram.d0 = P;
    gram.alpha = kSP / (S * S);
    e = plan.tall ? launch_product<true, true, true>(gram, E, ctas, st)
                  : launch_product<false, false, true>(gram, E, ctas, st);
    OrthProduct poly = gram;
    poly.A = poly.B = P;
    poly.sA = poly.sB = (int64_t)m * m;
    poly.lda = poly.ldb = poly.K = m;
    poly.d0 = Q;
    poly.alpha = kC / kSP;
    poly.c0 = P;
    poly.beta = kB;
    if (e == hipSuccess) e = launch_product<false, false, true>(poly, E, ctas, st);
    OrthProduct step = poly;
    step.sym = 0;
    step.M = M;
    step.N = N;
    step.K = m;
    step.A = plan.tall ? X : Q;
    step.sA = plan.tall ? mn : (int64_t)m * m;
    step.lda = m;
    step.B = plan.tall ? Q : X;
    step.sB = plan.tall ? (int64_t)m * m : mn;
    step.ldb = N;  // tall: N = m
    step.c0 = X;
    step.c1 = lo;
    step.d0 = hi[~i & 1];
    step.d1 = lo;
    step.out = i + 1 == steps ? static_cast<bf16_t*>(out) : nullptr;
    step.alpha = 1.f / kSP;
    step.beta = kA;
    step.gamma = 1.f / S;
    if (e == hipSuccess)
      e = plan.tall ? launch_product<false, false, false>(step, E, ctas, st)
                    : launch_product<false, true, false>(step, E, ctas, st);
  }
  return e;
}

}  // namespace moe
