// Host-side argument checks and workspace layout of the grouped products, the
// adapters and the orthogonalised update.  No HIP calls, as plan.hpp.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "moe.h"

namespace moe {

// moe_grouped_gemm: shape checks (MOE_OK or an error code).
int check_gemm_shape(const moe_gemm_shape* s);
// ... and those of moe_grouped_gemm_wgrad, whose operands are read by columns.
int check_gemm_wgrad_shape(const moe_gemm_shape* s);

struct GemmPlan {
  int BM;        // rows per tile: 16 and 32 stream the weights, 256 are MFMA-bound
  int split;     // the last round of 256-row tiles may be cut along K
  size_t total;  // workspace bytes (fp32 partial tiles of the cut)
};
int make_gemm_plan(const moe_gemm_shape* s, GemmPlan* p);

constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxRows = 1 << 24;
constexpr int kLoraMaxAdapters = 65536;
constexpr int kLoraMaxTrained = 256;  // adapters of a backward pass (it groups the rows by adapter)
int check_lora_shape(const moe_lora_shape* s);
int check_lora_tensors(const moe_lora_shape* s, const moe_lora_tensors* t);

struct LoraPlan {
  size_t off_xa;     // forward: fp32 [T][r]: A x, when the caller keeps none
  size_t total;
};
int make_lora_plan(const moe_lora_shape* s, LoraPlan* p);

struct LoraBwdPlan {
  size_t off_u;      // fp32 [T][r]: scale B^T dy
  size_t total;
};
int make_lora_backward_plan(const moe_lora_shape* s, LoraBwdPlan* p);

struct OrthPlan {
  int m, n;        // the smaller and the larger side
  int tall;        // M > N: P = X^T X
  size_t off_x[2]; // fp32 [E][M][N]
  size_t off_p, off_q;
  size_t off_norm;
  size_t total;
};
int make_orth_plan(int32_t E, int32_t M, int32_t N, OrthPlan* p);

}  // namespace moe
