// The rows of each adapter, in row order, for the adapters' gradients.
#pragma once
#include "lora.hpp"

namespace moe {
namespace {

// Workgroup l's list: counts its rows and those of the adapters before it (which
// gives the list's place in `sorted`), then writes its row numbers in order:
// four rows per thread and pass, ranked by ballots and the waves' counts.  Two
// reads of the T adapters per list; runs beside the first product's tiles.
// lds: 16 + 1 words.
__device__ __forceinline__ void lora_list(const LoraCall& c, const LoraLists& o, int l, int* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int before = 0;
#pragma unroll 4
  for (int64_t t = threadIdx.x; t < c.T; t += 256) {
    const int id = lora_id(c, t);
    before += id >= 0 && id < l;
  }
  for (int off = 32; off; off >>= 1) before += __shfl_xor(before, off);
  if (lane == 0) lds[wave] = before;
  __syncthreads();
  const int first = lds[0] + lds[1] + lds[2] + lds[3];
  __syncthreads();
  int at = first;
  for (int64_t t0 = 0; t0 < c.T; t0 += 1024) {
    bool mine[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t t = t0 + q * 256 + threadIdx.x;
      mine[q] = t < c.T && lora_id(c, t) == l;
    }
    int rank[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint64_t b = __ballot(mine[q]);
      rank[q] = __popcll(b & ((uint64_t(1) << lane) - 1));
      if (lane == 0) lds[q * 4 + wave] = __popcll(b);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      int base = at;
#pragma unroll
      for (int w = 0; w < 16; ++w) base += w < q * 4 + wave ? lds[w] : 0;
      if (mine[q]) o.sorted[base + rank[q]] = (int)(t0 + q * 256 + threadIdx.x);
    }
#pragma unroll
    for (int w = 0; w < 16; ++w) at += lds[w];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    o.counts[l] = at - first;
    o.offsets[l] = first;
  }
}

}  // namespace
}  // namespace moe
