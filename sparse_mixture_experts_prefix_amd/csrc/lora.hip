// Low-rank adapters of many requests beside one shared projection
// (moe_lora_forward, moe_lora_backward in moe.h): the adapters' first products,
// and the sequence of launches.
#include "launch.hpp"
#include "lora.hpp"
#include "lora_rows.hpp"
#include "lora_shrink.hpp"
#include "ops_launch.hpp"
#include "ragged.hpp"

namespace moe {
namespace {

// Workgroups (x): the rows' lists (one per adapter, when asked for), then the tiles;
// y: groups of 16 RB ranks; z: slots of a tile's distinct adapters.
template <int RB, bool KMAJ>
__global__ __launch_bounds__(256) void moe_lora_shrink_kernel(LoraCall c, ShrinkOut o, LoraLists rows) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  const int lists = rows.counts ? c.L : 0;
  if ((int)blockIdx.x >= lists)
    lora_shrink_tile<RB, KMAJ, false>(c, o, blockIdx.x - lists, blockIdx.y * RB, blockIdx.z, gridDim.z, 0,
                                      (c.K + 63) / 64, lds);
  else if (blockIdx.y == 0 && blockIdx.z == 0)
    lora_list(c, rows, blockIdx.x, reinterpret_cast<int*>(lds));
}

template <int RB, bool KMAJ>
hipError_t launch_shrink(const LoraCall& c, const ShrinkOut& o, const LoraLists& rows, hipStream_t s) {
  static std::atomic<uint64_t> done;
  const hipError_t e =
      allow_lds(reinterpret_cast<const void*>(moe_lora_shrink_kernel<RB, KMAJ>), shrink_lds_bytes<RB>(), done);
  if (e != hipSuccess) return e;
  const int tiles = (c.T + 15) / 16, groups = (c.r + 16 * RB - 1) / (16 * RB);
  // up to 16 adapters per tile at once while that keeps the grid at a few rounds
  // (slots without an adapter end at once)
  int slots = 1;
  while (slots < 16 && tiles * groups * slots < 1024) slots *= 2;
  const dim3 grid((unsigned)(tiles + (rows.counts ? c.L : 0)), (unsigned)groups, (unsigned)slots);
  hipLaunchKernelGGL((moe_lora_shrink_kernel<RB, KMAJ>), grid, dim3(256), shrink_lds_bytes<RB>(), s, c, o, rows);
  return hipGetLastError();
}

// All ranks in one workgroup (the rows are read once), or fewer where the tiles alone
// would leave CUs idle.
template <bool KMAJ>
hipError_t launch_shrink_rank(const LoraCall& c, const ShrinkOut& o, const LoraLists& rows, hipStream_t s) {
  int rb = c.r <= 16 ? 1 : c.r <= 32 ? 2 : c.r <= 64 ? 4 : 8;
  while (rb > 1 && (c.T + 15) / 16 * ((c.r + 16 * rb - 1) / (16 * rb)) < 256) rb /= 2;
  if (rb == 1) return launch_shrink<1, KMAJ>(c, o, rows, s);
  if (rb == 2) return launch_shrink<2, KMAJ>(c, o, rows, s);
  if (rb == 4) return launch_shrink<4, KMAJ>(c, o, rows, s);
  return launch_shrink<8, KMAJ>(c, o, rows, s);
}

template <class T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

}  // namespace

hipError_t launch_lora_forward(const moe_lora_shape& s, const LoraPlan& p, const moe_lora_tensors& t,
                               void* y, float* xa, void* ws, hipStream_t st) {
  const LoraCall c{static_cast<const bf16_t*>(t.x), static_cast<const bf16_t*>(t.w),
                   static_cast<const bf16_t*>(t.lora_a), static_cast<const bf16_t*>(t.lora_b), t.adapter,
                   t.scale, s.T, s.D, s.N, s.L, s.r, y, s.out_dtype == MOE_DTYPE_BF16};
  if (p.parts)
    return launch_lora_decode(c, false, ShrinkOut{xa, nullptr, 0, nullptr, nullptr}, LoraLists{},
                              at<float>(ws, p.off_v), p.v_parts, at<float>(ws, p.off_partial), p.parts, st);
  uint16_t* parts = at<uint16_t>(ws, p.off_v16);
  const int np = c.out16 ? kParts16 : kParts32;
  const hipError_t e = launch_shrink_rank<false>(c, ShrinkOut{xa, parts, np, nullptr, nullptr}, LoraLists{}, st);
  if (e != hipSuccess) return e;
  return launch_lora_prefill(c, false, parts, np, np, p.split ? at<float>(ws, p.off_partial) : nullptr, st);
}

hipError_t launch_lora_backward(const moe_lora_shape& s, const LoraBwdPlan& p,
                                const moe_lora_tensors& t, const void* dy, const float* xa,
                                const moe_lora_grads& g, void* ws, hipStream_t st) {
  // dx = dy W + u A: the forward's products with W and the adapters read K-major
  const LoraCall c{static_cast<const bf16_t*>(dy), static_cast<const bf16_t*>(t.w),
                   static_cast<const bf16_t*>(t.lora_b), static_cast<const bf16_t*>(t.lora_a), t.adapter,
                   t.scale, s.T, s.N, s.D, s.L, s.r, g.dx, s.out_dtype == MOE_DTYPE_BF16};
  uint16_t* u16 = at<uint16_t>(ws, p.off_u16);
  uint16_t* xa16 = at<uint16_t>(ws, p.off_xa16);
  int32_t* q = at<int32_t>(ws, p.off_rows);
  const LoraLists rows{q, q + s.L, q + 2 * s.L};
  float* partial = at<float>(ws, p.off_partial);
  hipError_t e;
  if (p.parts) {
    e = launch_lora_decode(c, true, ShrinkOut{nullptr, u16, kParts32, xa, xa16}, rows, at<float>(ws, p.off_v), p.v_parts,
                           partial, p.parts, st);
  } else {
    e = launch_shrink_rank<true>(c, ShrinkOut{nullptr, u16, kParts32, xa, xa16}, rows, st);
    if (e == hipSuccess) e = launch_lora_prefill(c, true, u16, kParts32, c.out16 ? kParts16 : kParts32,
                                                   p.split ? partial : nullptr, st);
  }
  if (e != hipSuccess) return e;
  return launch_lora_wgrad(rows, t.x, dy, u16, xa16, t.scale, s.T, s.D, s.N, s.L, s.r, g.da, g.db, st);
}

}  // namespace moe
