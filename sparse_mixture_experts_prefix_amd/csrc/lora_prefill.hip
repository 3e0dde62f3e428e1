// The adapters' large products (many rows): out = in W^T (or in W, W read
// K-major) on the 256 x 256 x 64 tiles of gemm_tile.hpp, with the adapters'
// second product, v[t] (in bf16 parts) times expand[a], added to the tile's
// accumulators in registers before they are stored.
#include "gemm_tile.hpp"
#include "lora.hpp"
#include "ops_launch.hpp"
#include "ragged.hpp"

namespace moe {
namespace {

// One dense group of T rows for prefill_tile (field names as GroupedGemm's).
struct LoraGemm {
  static constexpr bool kRagged = true, kFold = false, kLora = true;
  static constexpr const int32_t* row_token = nullptr;
  static constexpr int64_t a_bytes = 0, ld_gu = 0;
  static constexpr uint16_t* gu_out = nullptr;
  static constexpr const void* B_shared = nullptr;
  static constexpr const float *S_shared = nullptr, *S_routed = nullptr;
  static constexpr int N_shared = 0, K_shared = 0, BM = 256, E = 1, stream_out = 0;
  const uint16_t* A;
  int64_t lda;
  const void* B_routed;
  int N_routed, K_routed;
  void* C;
  int64_t ldc;
  int out16;
  int64_t n_tiles_n;
  int ctas;
  float* partial;
  LoraCall call;
  const uint16_t* parts;  // [T][np][r], the upper `used` parts count
  int np, used;
};
__device__ __forceinline__ int group_rows(const LoraGemm& p, int) { return p.call.T; }
__device__ __forceinline__ int group_first(const LoraGemm&, int) { return 0; }

// Infinities and NaN become the largest finite value of their sign: a zero row
// of parts then stays zero, whatever the adapter holds.
__device__ __forceinline__ bf16x8 finite8(bf16x8 v) {
  typedef unsigned short u16x8 __attribute__((ext_vector_type(8)));
  const u16x8 bits = __builtin_bit_cast(u16x8, v);
  const u16x8 mag = __builtin_elementwise_min(bits & (unsigned short)0x7FFF, u16x8(0x7F7F));
  return __builtin_bit_cast(bf16x8, mag | (bits & (unsigned short)0x8000));
}

// acc += parts[rows] . expand[a]^T for every adapter a that the tile's rows
// name.  Per adapter and 64 of its part columns: its rows of `parts` (the other
// rows read as zero) and the tile's columns of expand[a] (rank j for column j of
// every part) go through LDS in the K loop's layouts, the next stage's loads
// under this one's products, and are multiplied onto the tile's sums.  Adapter
// values enter as finite numbers, so they reach no row that does not name the
// adapter; adding only its rows of a product held apart made the 256 sums spill.
// A request's rows are usually a run, so a tile has one or two adapters: a stage
// of 64 each, against K / 64 stages of the projection.
template <bool KMAJ>
__device__ __forceinline__ void lora_expand(const LoraGemm& p, char* lds, int64_t row0, int valid, int n0,
                                            int wm, int wn, bool il, f32x16 (&acc)[4][4]) {
  const LoraCall& c = p.call;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 31, kh = lane >> 5, sub = lane >> 3;
  constexpr int kStage = kABytes + kBBytes;
  int* ids = reinterpret_cast<int*>(lds + 2 * kStage);  // adapter of each tile row
  const int r = c.r, ld = p.np * r, rk = p.used * r, N = c.N;  // a row's part columns, and those used
  __syncthreads();  // every wave has left the K loop's stages
  ids[tid] = tid < valid ? lora_id(c, row0 + tid) : -1;
  __syncthreads();
  // this wave's view of the 256 rows: row 64 q + lane
  int id[4];
  bool left[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    id[q] = ids[64 * q + lane];
    left[q] = id[q] >= 0;
  }
  // the next adapter, in order of its first row (the same in every wave), or -1
  auto next_adapter = [&]() {
    int l = -1;
#pragma unroll
    for (int q = 3; q >= 0; --q) {
      const uint64_t b = __ballot(left[q]);
      if (b) l = __builtin_amdgcn_readlane(id[q], (int)__builtin_ctzll(b));
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) left[q] = left[q] && id[q] != l;
    return l;
  };
  auto rank = [&](int k) { return k < r ? k : k < 2 * r ? k - r : k - 2 * r; };  // of part column k < 3 r
  const __amdgpu_buffer_rsrc_t rsV = make_rsrc(p.parts + row0 * ld, (uint32_t)(valid * ld * 2));
  // part columns k0 .. k0 + 63 of adapter l into stage `buf`
  auto issue = [&](int l, int k0, int buf) {
    const __amdgpu_buffer_rsrc_t rsE = make_rsrc(c.expand + (int64_t)l * N * r, (uint32_t)(N * r * 2));
    char* la = lds + __builtin_amdgcn_readfirstlane(buf * kStage);
    char* lb = la + kABytes;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int ra = (j * 4 + wave) * 8 + sub;  // row of this lane's chunk
      const int k = k0 + 8 * ((lane & 7) ^ swz(ra));
      const bool mine = ids[ra] == l && k < rk;
      lds_dma16(rsV, la + (j * 4 + wave) * 1024, mine ? (uint32_t)((ra * ld + k) * 2) : kOob, 0);
      uint32_t off;
      if constexpr (KMAJ) {
        const int kr = 2 * (wave * 8 + j) + (lane >> 5);  // part column, and 8 columns of the tile
        const int kk = k0 + kr, n = n0 + 8 * kmaj_chunk(kr, lane & 31);
        off = kk < rk && n < N ? (uint32_t)((rank(kk) * N + n) * 2) : kOob;
      } else {
        const int rb = (wave * 8 + j) * 8 + sub;
        const int kb = k0 + 8 * ((lane & 7) ^ swz(rb)), n = n0 + rb;
        off = kb < rk && n < N ? (uint32_t)((n * r + rank(kb)) * 2) : kOob;
      }
      lds_dma16(rsE, lb + (wave * 8 + j) * 1024, off, 0);
    }
  };
  int l = next_adapter(), k0 = 0, buf = 0;
  if (l >= 0) issue(l, 0, 0);
  while (l >= 0) {
    int ln = l, kn = k0 + 64;  // the next stage
    if (kn >= rk) {
      ln = next_adapter();
      kn = 0;
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
    __syncthreads();  // this stage is whole, and every wave has read the one before
    if (ln >= 0) issue(ln, kn, buf ^ 1);
    const char* la = lds + buf * kStage;
    const char* lb = la + kABytes;
    auto read_a = [&](int i, int ks) {
      return *reinterpret_cast<const bf16x8*>(la + a_row_of(wm, i, il) * 128 +
                                              (lr * 8 + ((2 * ks + kh) ^ swz(lr))) * 16);
    };
    auto read_b = [&](int j, int ks) {
      if constexpr (KMAJ) {
        typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
        typedef __attribute__((address_space(3))) char lds_char;
        const int q = lane & 15, k = 16 * ks + 8 * kh + (q >> 2);
        const int cn = b_row_of<false>(wn, j) + 16 * ((lane >> 4) & 1) + 4 * (q & 3);
        const char* at = lb + k * 512 + kmaj_chunk(k, cn >> 3) * 16 + (cn & 7) * 2;
        const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)((lds_char*)at));
        const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)((lds_char*)(at + 4 * 512)));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      } else {
        return *reinterpret_cast<const bf16x8*>(lb + b_row_of<false>(wn, j) * 128 +
                                                (lr * 8 + ((2 * ks + kh) ^ swz(lr))) * 16);
      }
    };
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (k0 + 16 * ks >= rk) break;  // no part columns left in the stage
      bf16x8 fa[4], fb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) fa[i] = read_a(i, ks);
#pragma unroll
      for (int j = 0; j < 4; ++j) fb[j] = finite8(read_b(j, ks));
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mfma32(fa[i], fb[j], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
    l = ln;
    k0 = kn;
    buf ^= 1;
  }
  __syncthreads();  // the last stage is read before the next tile's loads
}

// The output type fixed at compile time (with both epilogues the kernels spilled).
template <bool OUT16>
struct TypedLora : LoraGemm {
  static constexpr int out16 = OUT16;
};

template <bool KT, bool OUT16>
__global__ __launch_bounds__(256) void moe_lora_prefill_kernel(TypedLora<OUT16> p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  prefill_tile<false, false, false, KT>(p, lds);
}

template <bool OUT16>
__global__ __launch_bounds__(256) void moe_lora_kmajor_prefill_kernel(TypedLora<OUT16> p) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  prefill_tile<false, false, true>(p, lds);
}

__global__ __launch_bounds__(256) void moe_lora_fixup_kernel(LoraGemm p) { fixup_tiles<false, false>(p); }

template <bool OUT16>
hipError_t launch_tiles(void (*kernel)(TypedLora<OUT16>), const LoraGemm& g, int64_t blocks,
                        std::atomic<uint64_t>& done, hipStream_t s) {
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(kernel), kLdsBytes, done);
  if (e != hipSuccess) return e;
  TypedLora<OUT16> p;
  static_cast<LoraGemm&>(p) = g;
  hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), kLdsBytes, s, p);
  return hipGetLastError();
}

hipError_t launch_typed(void (*k32)(TypedLora<false>), void (*k16)(TypedLora<true>), const LoraGemm& p, int64_t blocks,
                        std::atomic<uint64_t>& done32, std::atomic<uint64_t>& done16, hipStream_t s) {
  return p.out16 ? launch_tiles<true>(k16, p, blocks, done16, s) : launch_tiles<false>(k32, p, blocks, done32, s);
}

}  // namespace

hipError_t launch_lora_prefill(const LoraCall& c, bool kmajor, const uint16_t* parts, int np, int used,
                               float* partial, hipStream_t s) {
  static std::atomic<uint64_t> done[6];
  LoraGemm p{};
  p.A = c.in;
  p.lda = c.K;
  p.B_routed = c.w;
  p.N_routed = c.N;
  p.K_routed = c.K;
  p.C = c.out;
  p.ldc = c.N;
  p.out16 = c.out16;
  p.n_tiles_n = (c.N + BN - 1) / BN;
  p.call = c;
  p.parts = parts;
  p.np = np;
  p.used = used;
  p.partial = partial;
  hipError_t e = partial ? split_ctas(&p.ctas) : hipSuccess;
  if (e != hipSuccess) return e;
  // the rows are known here, and with them which tiles are cut (as on the device)
  const int64_t mtiles = (c.T + BM - 1) / BM;
  const Split sp = split_of(p, mtiles);
  if (sp.R == 0) p.ctas = 0;
  const int64_t blocks = (sp.n_dp + 7) / 8 * 8 + sp.R * sp.S;
  if (kmajor)
    e = launch_typed(moe_lora_kmajor_prefill_kernel<false>, moe_lora_kmajor_prefill_kernel<true>, p, blocks, done[0],
                     done[3], s);
  else if (c.K % BK)
    e = launch_typed(moe_lora_prefill_kernel<true, false>, moe_lora_prefill_kernel<true, true>, p, blocks, done[1],
                     done[4], s);
  else
    e = launch_typed(moe_lora_prefill_kernel<false, false>, moe_lora_prefill_kernel<false, true>, p, blocks, done[2],
                     done[5], s);
  if (e != hipSuccess || sp.R == 0) return e;
  hipLaunchKernelGGL(moe_lora_fixup_kernel, dim3((unsigned)(sp.R * kFixBlocksPerTile)), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace moe
