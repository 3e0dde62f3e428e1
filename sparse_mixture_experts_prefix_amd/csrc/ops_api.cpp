// extern "C" entry points of the grouped products, the adapters and the
// orthogonalised update (declared and documented in moe.h).
#include <hip/hip_runtime.h>

#include <cmath>

#include "launch.hpp"
#include "ops_launch.hpp"
#include "plan.hpp"

namespace {

int done(hipError_t e) { return e == hipSuccess ? MOE_OK : moe::record_hip_error(e); }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// a workspace argument of a call that needs `need` bytes
int check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return MOE_OK;
  if (!ws) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned16(ws)) return MOE_ERR_ALIGNMENT;
  return have < need ? MOE_ERR_WORKSPACE : MOE_OK;
}

}  // namespace

extern "C" {

int moe_grouped_gemm_workspace_size(const moe_gemm_shape* shape, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  moe::GemmPlan p;
  const int rc = moe::make_gemm_plan(shape, &p);
  if (rc) return rc;
  *bytes = p.total;
  return MOE_OK;
}

int moe_grouped_gemm(const moe_gemm_shape* shape, const void* x, const int32_t* offsets,
                     const void* w, const float* w_scale, void* y, void* workspace,
                     size_t ws_bytes, void* stream) {
  moe::GemmPlan p;
  int rc = moe::make_gemm_plan(shape, &p);
  if (rc) return rc;
  const bool fp8 = shape->weight_format == MOE_WEIGHTS_FP8_E4M3;
  if (!offsets || !w || (fp8 && !w_scale)) return MOE_ERR_INVALID_ARG;
  if (shape->R > 0 && (!x || !y)) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned16(x) || !moe::aligned16(w) || !moe::aligned16(y) || !aligned4(offsets) ||
      (fp8 && !aligned4(w_scale)))
    return MOE_ERR_ALIGNMENT;
  if (shape->R == 0) return MOE_OK;
  rc = check_workspace(workspace, ws_bytes, p.total);
  if (rc) return rc;
  return done(moe::launch_grouped_gemm(*shape, p, x, offsets, w, w_scale, y, workspace,
                                       static_cast<hipStream_t>(stream)));
}

int moe_grouped_gemm_wgrad(const moe_gemm_shape* shape, const void* dy, const void* x,
                           const int32_t* offsets, float* dw, void* stream) {
  const int rc = moe::check_gemm_wgrad_shape(shape);
  if (rc) return rc;
  if (!offsets || !dw) return MOE_ERR_INVALID_ARG;
  if (shape->R > 0 && (!x || !dy)) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned16(x) || !moe::aligned16(dy) || !moe::aligned16(dw) || !aligned4(offsets))
    return MOE_ERR_ALIGNMENT;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (shape->R == 0)
    return done(moe::launch_fill_f32(dw, (int64_t)shape->G * shape->N * shape->K, s));
  return done(moe::launch_grouped_wgrad(*shape, dy, x, offsets, dw, s));
}

int moe_lora_workspace_size(const moe_lora_shape* shape, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  moe::LoraPlan p;
  const int rc = moe::make_lora_plan(shape, &p);
  if (rc) return rc;
  *bytes = p.total;
  return MOE_OK;
}

int moe_lora_forward(const moe_lora_shape* shape, const moe_lora_tensors* t, void* y, float* xa,
                     void* workspace, size_t ws_bytes, void* stream) {
  moe::LoraPlan p;
  int rc = moe::make_lora_plan(shape, &p);
  if (rc) return rc;
  rc = moe::check_lora_tensors(shape, t);
  if (rc) return rc;
  if (shape->T > 0 && !y) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned16(y) || !moe::aligned16(xa)) return MOE_ERR_ALIGNMENT;
  if (shape->T == 0) return MOE_OK;
  rc = check_workspace(workspace, ws_bytes, p.total);
  if (rc) return rc;
  return done(moe::launch_lora_forward(*shape, p, *t, y, xa, workspace,
                                       static_cast<hipStream_t>(stream)));
}

int moe_lora_backward_workspace_size(const moe_lora_shape* shape, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  moe::LoraBwdPlan p;
  const int rc = moe::make_lora_backward_plan(shape, &p);
  if (rc) return rc;
  *bytes = p.total;
  return MOE_OK;
}

int moe_lora_backward(const moe_lora_shape* shape, const moe_lora_tensors* t, const void* dy,
                      const float* xa, const moe_lora_grads* grads, void* workspace,
                      size_t ws_bytes, void* stream) {
  moe::LoraBwdPlan p;
  int rc = moe::make_lora_backward_plan(shape, &p);
  if (rc) return rc;
  rc = moe::check_lora_tensors(shape, t);
  if (rc) return rc;
  if (!grads || !grads->da || !grads->db) return MOE_ERR_INVALID_ARG;
  if (shape->T > 0 && (!dy || !xa || !grads->dx)) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned16(dy) || !moe::aligned16(xa) || !moe::aligned16(grads->dx) ||
      !moe::aligned16(grads->da) || !moe::aligned16(grads->db))
    return MOE_ERR_ALIGNMENT;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (shape->T == 0) {
    const int64_t lr = (int64_t)shape->L * shape->r;
    hipError_t e = moe::launch_fill_f32(grads->da, lr * shape->D, s);
    if (e == hipSuccess) e = moe::launch_fill_f32(grads->db, lr * shape->N, s);
    return done(e);
  }
  rc = check_workspace(workspace, ws_bytes, p.total);
  if (rc) return rc;
  return done(moe::launch_lora_backward(*shape, p, *t, dy, xa, *grads, workspace, s));
}

int moe_orthogonalize_workspace_size(int32_t E, int32_t M, int32_t N, size_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  moe::OrthPlan p;
  const int rc = moe::make_orth_plan(E, M, N, &p);
  if (rc) return rc;
  *bytes = p.total;
  return MOE_OK;
}

int moe_orthogonalize(int32_t E, int32_t M, int32_t N, const void* g, int32_t g_dtype,
                      int32_t steps, float eps, void* out, void* workspace, size_t ws_bytes,
                      void* stream) {
  moe::OrthPlan p;
  int rc = moe::make_orth_plan(E, M, N, &p);
  if (rc) return rc;
  if ((g_dtype != MOE_DTYPE_F32 && g_dtype != MOE_DTYPE_BF16) || steps < 1 || steps > 16 ||
      !(eps >= 0.f) || !std::isfinite(eps))
    return MOE_ERR_INVALID_ARG;
  if (E == 0) return MOE_OK;
  if (!g || !out) return MOE_ERR_INVALID_ARG;
  if (!moe::aligned16(g) || !moe::aligned16(out)) return MOE_ERR_ALIGNMENT;
  rc = check_workspace(workspace, ws_bytes, p.total);
  if (rc) return rc;
  return done(moe::launch_orthogonalize(E, M, N, p, g, g_dtype, steps, eps, out, workspace,
                                        static_cast<hipStream_t>(stream)));
}

}  // extern "C"
