// Launchers of the grouped products, the adapters and the orthogonalised
// update (host functions defined next to their kernels).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lora.hpp"
#include "ops_plan.hpp"
#include "ragged.hpp"

namespace moe {

hipError_t launch_grouped_gemm(const moe_gemm_shape& s, const GemmPlan& p, const void* x,
                               const int32_t* offsets, const void* w, const float* w_scale, void* y,
                               void* ws, hipStream_t st);
// groups of many rows: mtiles bounds the 256-row tiles that hold rows
hipError_t launch_grouped_prefill(RaggedGemm p, bool fp8, bool kn, int64_t mtiles, hipStream_t s);
hipError_t launch_grouped_wgrad(const moe_gemm_shape& s, const void* dy, const void* x,
                                const int32_t* offsets, float* dw, hipStream_t st);
hipError_t launch_lora_forward(const moe_lora_shape& s, const LoraPlan& p, const moe_lora_tensors& t,
                               void* y, float* xa, void* ws, hipStream_t st);
hipError_t launch_lora_backward(const moe_lora_shape& s, const LoraBwdPlan& p,
                                const moe_lora_tensors& t, const void* dy, const float* xa,
                                const moe_lora_grads& g, void* ws, hipStream_t st);
// out = in w^T + the adapters' second product (kmajor: w and the adapters as the
// backward pass reads them).  Many rows: parts16 [T][np][r] holds the first product's
// bf16 parts, of which the upper `used` count; partial (or NULL: no cut along K) room
// for partial tiles.
hipError_t launch_lora_prefill(const LoraCall& c, bool kmajor, const uint16_t* parts16, int np, int used,
                               float* partial, hipStream_t s);
// At most 64 rows, both products; rows.counts set: the rows' lists too.  Workspace:
// v fp32 [v_parts][T][r], partial fp32 [parts][T][N].
hipError_t launch_lora_decode(const LoraCall& c, bool kmajor, const ShrinkOut& o, const LoraLists& rows,
                              float* v, int v_parts, float* partial, int parts, hipStream_t s);
hipError_t launch_lora_wgrad(const LoraLists& rows, const void* x, const void* dy, const uint16_t* u,
                             const uint16_t* xa, const float* scale, int T, int D, int N, int L, int r,
                             float* da, float* db, hipStream_t s);
hipError_t launch_orthogonalize(int E, int M, int N, const OrthPlan& p, const void* g, int g_dtype,
                                int steps, float eps, void* out, void* ws, hipStream_t st);


}  // namespace moe
