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

// Mean rows per group up to which the weight gradient takes its 128 x 128 tiles
// (30 x 2048 x 2880: 120 against 142 us at 23 rows per group; 64 x 2048 x 4096: 470
// against 449 us at 156).
constexpr int kWgradSmallRows = 64;

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

// Whether a call takes the few-row path: its second product reads an adapter's rows
// once per row that names it (2 N r bytes), whoever its neighbours are, where the
// 256-row tiles take a stage of each adapter they hold.  Few rows against tiles, N = D =
// 4096: 250 rows of 30 adapters, rank 64 67 us against 208, rank 128 96 against 371; of 2
// adapters, rank 64 54 against 52, rank 128 77 against 63; 100 rows of 2 adapters, rank 128
// 41 against 53; 512 rows, rank 16, of 30 adapters 62 against 132, of 2 56 against 66;
// past the limits, 1024 rows of 2 adapters, rank 32, 120 against 80.  How many adapters
// the rows name is known on the device alone: L bounds it.
inline bool lora_few_rows(const moe_lora_shape* s) {
  const int64_t T = s->T, Tr = T * s->r;
  if (T <= 64 || (T <= 256 && (s->L > 4 || Tr <= 16384))) return true;
  return s->L > 4 && T <= 1024 && Tr <= 32768 && T * s->N * s->D <= int64_t(1) << 33;
}

struct LoraPlan {
  int parts;           // few rows: parts K is cut into (0: the 256-row tiles)
  int v_parts;         // ... and for the first product
  int split;           // 256-row tiles: the last round may be cut along K
  size_t off_v;        // few rows: fp32 [v_parts][T][r], A x in parts
  size_t off_v16;      // many rows: bf16 [T][3][r], its bf16 parts (two of them for a bf16 y)
  size_t off_partial;  // fp32 [parts][T][N], or partial tiles
  size_t total;
};
int make_lora_plan(const moe_lora_shape* s, LoraPlan* p);

struct LoraBwdPlan {
  int parts, v_parts, split;  // as above, for dx and u
  size_t off_v;        // few rows: fp32 [v_parts][T][r], B^T dy in parts
  size_t off_u16;      // bf16 [T][3][r]: u's parts
  size_t off_xa16;     // bf16 [T][3][r]: xa's
  size_t off_rows;     // int32 [2 L + T]: the adapters' rows (LoraLists)
  size_t off_partial;  // fp32 [parts][T][D], or partial tiles
  size_t total;
};
int make_lora_backward_plan(const moe_lora_shape* s, LoraBwdPlan* p);

constexpr int64_t kOrthPartialFloats = int64_t(256) * 65536;  // 64 MB of partial tiles
struct OrthPlan {
  int m, n;           // the smaller and the larger side
  int tall;           // M > N: P = X^T X
  float scale;        // S: fp16 X holds S X
  int norm_parts;     // blocks per matrix of the sum of squares
  size_t off_hi[2];   // fp16 [E][M][N]: X's upper part, this step's and the next's
  size_t off_lo;      // fp16 [E][M][N]: its lower part
  size_t off_p, off_q;  // fp16 [E][m][m]
  size_t off_norm;    // double [E][norm_parts]
  size_t off_partial; // fp32 partial tiles
  size_t total;
};
int make_orth_plan(int32_t E, int32_t M, int32_t N, OrthPlan* p);

}  // namespace moe
