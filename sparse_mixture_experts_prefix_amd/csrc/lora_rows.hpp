// The rows of each adapter, in row order, for the adapters' gradients.
#pragma once
#include "lora.hpp"

namespace moe {
namespace {

// Workgroup l's list: counts its rows and those of the adapters before it (which
// gives the list's place in `sorted`), then writes its row numbers in order:
// sixteen rows per thread and pass (one memory latency per 4096 rows), ranked by
// ballots and the waves' counts.  Two reads of the T adapters per list; runs
// beside the first product's tiles.  lds: 64 words.
__device__ __forceinline__ void lora_list(const LoraCall& c, const LoraLists& o, int l, int* lds) {
  constexpr int U = 16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int before = 0;
  for (int64_t t0 = threadIdx.x; t0 < c.T; t0 += 256 * U) {
    int id[U];
#pragma unroll
    for (int q = 0; q < U; ++q) id[q] = t0 + 256 * q < c.T ? lora_id(c, t0 + 256 * q) : -1;
#pragma unroll
    for (int q = 0; q < U; ++q) before += id[q] >= 0 && id[q] < l;
  }
  for (int off = 32; off; off >>= 1) before += __shfl_xor(before, off);
  if (lane == 0) lds[wave] = before;
  __syncthreads();
  const int first = lds[0] + lds[1] + lds[2] + lds[3];
  __syncthreads();
  int at = first;
  for (int64_t t0 = 0; t0 < c.T; t0 += 256 * U) {
    bool mine[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int64_t t = t0 + q * 256 + threadIdx.x;
      mine[q] = t < c.T && lora_id(c, t) == l;
    }
    int rank[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const uint64_t b = __ballot(mine[q]);
      rank[q] = __popcll(b & ((uint64_t(1) << lane) - 1));
      if (lane == 0) lds[q * 4 + wave] = __popcll(b);
    }
    __syncthreads();
    // lane i: the count of part i (64 rows each, in row order), and those before it
    const int cnt = lds[lane];
    int incl = cnt;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int y = __shfl_up(incl, off);
      if (lane >= off) incl += y;
    }
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const int base = at + __shfl(incl - cnt, q * 4 + wave);
      if (mine[q]) o.sorted[base + rank[q]] = (int)(t0 + q * 256 + threadIdx.x);
    }
    at += __shfl(incl, 63);
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    o.counts[l] = at - first;
    o.offsets[l] = first;
  }
}

}  // namespace
}  // namespace moe
