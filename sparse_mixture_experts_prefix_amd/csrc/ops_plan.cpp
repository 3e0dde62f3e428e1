// Host-side argument checks and workspace layout (no HIP calls).
#include "ops_plan.hpp"

#include "plan.hpp"

namespace moe {

namespace {
constexpr int64_t kLim31 = int64_t(1) << 31;
constexpr int64_t kMaxTiles = int64_t(1) << 23;  // workgroups of a launch (256 threads each)

struct Layout {
  size_t o = 0;
  size_t take(size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) / 256 * 256;
    return at;
  }
};

// a tile's rows (up to 288 of them) are addressed with 32-bit byte offsets
bool width_ok(int64_t w) { return 288 * 4 * w < kLim31; }
// Whether the 256-row tile kernels may cut their last round along K: K long
// enough for two pieces of four 64-wide stages, and fewer than four rounds of
// tiles on the largest chip (see split_of in gemm_tile.hpp).
constexpr size_t kPartialBytes = sizeof(float) * kSplitCtas * kPartialTileFloats;
bool may_split(int64_t mtiles, int64_t N, int64_t K) {
  return (K + 63) / 64 >= 8 && mtiles * ((N + 255) / 256) < 4 * kSplitCtas;
}
bool mult8(int64_t v) { return v > 0 && v % 8 == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
}  // namespace

int check_gemm_shape(const moe_gemm_shape* s) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->R < 0 || s->G <= 0 || !mult8(s->N) || !mult8(s->K)) return MOE_ERR_INVALID_ARG;
  if (s->weight_format != MOE_WEIGHTS_BF16 && s->weight_format != MOE_WEIGHTS_FP8_E4M3)
    return MOE_ERR_INVALID_ARG;
  if (s->weight_layout != MOE_LAYOUT_NK && s->weight_layout != MOE_LAYOUT_KN)
    return MOE_ERR_INVALID_ARG;
  if (s->out_dtype != MOE_DTYPE_F32 && s->out_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (s->G > 256) return MOE_ERR_UNSUPPORTED;
  // E4M3 scales belong to rows of w, which the transposed product sums over
  if (s->weight_format == MOE_WEIGHTS_FP8_E4M3 && s->weight_layout == MOE_LAYOUT_KN)
    return MOE_ERR_UNSUPPORTED;
  if ((int64_t)s->N * s->K * 2 >= kLim31 || !width_ok(s->N) || !width_ok(s->K))
    return MOE_ERR_UNSUPPORTED;
  // row indices, and the workgroups of the smallest tiles of 32 x 64
  if ((int64_t)s->R + 256 * 257 >= kLim31) return MOE_ERR_UNSUPPORTED;
  if (((int64_t)s->R / 32 + 2 * s->G) * (s->N / 64 + 1) >= kMaxTiles) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_gemm_wgrad_shape(const moe_gemm_shape* s) {
  const int rc = check_gemm_shape(s);
  if (rc) return rc;
  if (s->weight_format || s->weight_layout || s->out_dtype) return MOE_ERR_INVALID_ARG;
  const int64_t w = s->N > s->K ? s->N : s->K;
  if ((int64_t)s->R * w * 2 >= kLim31 || (int64_t)s->N * s->K * 4 >= kLim31)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int make_gemm_plan(const moe_gemm_shape* s, GemmPlan* p) {
  const int rc = check_gemm_shape(s);
  if (rc) return rc;
  // tile rows by mean rows per group, as the layer's (choose_block_m): few rows
  // stream the weights.  E4M3 codes move in 16-code chunks in the 256-row tiles.
  const int64_t rows = s->R;
  p->BM = rows <= (int64_t)20 * s->G ? 16 : rows <= (int64_t)48 * s->G ? 32 : 256;
  if (p->BM == 256 && s->weight_format == MOE_WEIGHTS_FP8_E4M3 && s->K % 16) p->BM = 32;
  p->split = p->BM == 256 && may_split((rows + 255) / 256, s->N, s->K);
  p->total = p->split ? kPartialBytes : 0;
  return MOE_OK;
}

int check_lora_shape(const moe_lora_shape* s) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->T < 0 || s->L <= 0 || !mult8(s->D) || !mult8(s->N) || !mult8(s->r))
    return MOE_ERR_INVALID_ARG;
  if (s->out_dtype != MOE_DTYPE_F32 && s->out_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (s->L > kLoraMaxAdapters || s->r > kLoraMaxRank) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)s->N * s->D * 2 >= kLim31 || !width_ok(s->N) || !width_ok(s->D))
    return MOE_ERR_UNSUPPORTED;
  const int64_t w = s->N > s->D ? s->N : s->D;
  if (((int64_t)s->T / 256 + 1) * (w / 64 + 1) >= kMaxTiles || s->T > kLoraMaxRows)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_lora_tensors(const moe_lora_shape* s, const moe_lora_tensors* t) {
  if (!t || !t->w || !t->lora_a || !t->lora_b) return MOE_ERR_INVALID_ARG;
  if (s->T > 0 && (!t->x || !t->adapter)) return MOE_ERR_INVALID_ARG;
  const void* ptrs[] = {t->x, t->w, t->lora_a, t->lora_b};
  for (const void* q : ptrs)
    if (q && !aligned16(q)) return MOE_ERR_ALIGNMENT;
  if (!aligned4(t->adapter) || !aligned4(t->scale)) return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

namespace {
// Parts of K of the few-row path: two workgroups per CU (of 256) less those of the
// first product's longer waits, so that all of them run from the start (512 columns' tiles
// and the first product's 16 workgroups beyond them: 14.8 us against 13.9 us for 16 rows x
// 4096 x 4096), each wave with two or more of the 64-wide K chunks.
int few_row_parts(int64_t T, int64_t N, int64_t K) {
  const int64_t blocks = T > 64 ? (T + 63) / 64 : 1;  // no rows: a plan like one row's
  const int64_t tiles = (N + 63) / 64 * blocks, chunks = (K + 63) / 64;
  int64_t parts = 496 / tiles;
  if (parts > chunks / 8) parts = chunks / 8;
  return parts < 1 ? 1 : (int)parts;
}
// Parts of K of the first product there: two where that adds few workgroups (its
// waits beside the weights' stream are long: 14.7 -> 13.9 us at 16 rows, rank 16; at 64
// rows, rank 64 its 256 workgroups are enough: 28.3 against 28.6 us).
int few_row_v_parts(const moe_lora_shape* s, int64_t K) {
  return K > 1024 && (s->T + 15) / 16 * ((s->r + 15) / 16) <= 2 ? 2 : 1;
}
}  // namespace

int make_lora_plan(const moe_lora_shape* s, LoraPlan* p) {
  const int rc = check_lora_shape(s);
  if (rc) return rc;
  const size_t T = s->T, r = s->r;
  const bool few = lora_few_rows(s);
  p->parts = few ? few_row_parts(s->T, s->N, s->D) : 0;
  p->v_parts = few ? few_row_v_parts(s, s->D) : 0;
  p->split = !few && may_split((s->T + 255) / 256, s->N, s->D);
  Layout l;
  p->off_v = l.take(sizeof(float) * p->v_parts * T * r);
  p->off_v16 = l.take(few ? 0 : sizeof(uint16_t) * T * 3 * r);
  p->off_partial = l.take(few ? sizeof(float) * p->parts * T * s->N : p->split ? kPartialBytes : 0);
  p->total = l.o;
  return MOE_OK;
}

int make_lora_backward_plan(const moe_lora_shape* s, LoraBwdPlan* p) {
  const int rc = check_lora_shape(s);
  if (rc) return rc;
  if (s->L > kLoraMaxTrained) return MOE_ERR_UNSUPPORTED;
  // gathered rows are addressed with 32-bit byte offsets
  const int64_t w = s->N > s->D ? s->N : s->D;
  if (s->T * w * 2 >= kLim31 || (int64_t)s->T * s->r * 6 >= kLim31) return MOE_ERR_UNSUPPORTED;
  const size_t T = s->T, r = s->r;
  const bool few = lora_few_rows(s);
  p->parts = few ? few_row_parts(s->T, s->D, s->N) : 0;
  p->v_parts = few ? few_row_v_parts(s, s->N) : 0;
  p->split = !few && may_split((s->T + 255) / 256, s->D, s->N);
  Layout l;
  p->off_v = l.take(sizeof(float) * p->v_parts * T * r);
  p->off_u16 = l.take(sizeof(uint16_t) * T * 3 * r);
  p->off_xa16 = l.take(sizeof(uint16_t) * T * 3 * r);
  p->off_rows = l.take(sizeof(int32_t) * (2 * s->L + T));
  p->off_partial = l.take(few ? sizeof(float) * p->parts * T * s->D : p->split ? kPartialBytes : 0);
  p->total = l.o;
  return MOE_OK;
}

int make_orth_plan(int32_t E, int32_t M, int32_t N, OrthPlan* p) {
  if (E < 0 || !mult8(M) || !mult8(N)) return MOE_ERR_INVALID_ARG;
  if (E > 256 || M > 32768 || N > 32768) return MOE_ERR_UNSUPPORTED;
  p->m = M < N ? M : N;
  p->n = M < N ? N : M;
  p->tall = M > N;
  if ((int64_t)M * N * 4 >= kLim31 || (int64_t)p->m * p->m * 4 >= kLim31) return MOE_ERR_UNSUPPORTED;
  const int64_t mn = (int64_t)M * N;
  int s = 0;  // S = 2^ceil(log2 sqrt(M N)), at most 2^15
  while (s < 15 && (int64_t(1) << (2 * s)) < mn) ++s;
  p->scale = (float)(1 << s);
  const int64_t blocks = (mn + 16383) / 16384;  // eight passes of 256 threads x 8 values
  p->norm_parts = blocks < 128 ? (int)blocks : 128;
  Layout l;
  const size_t x = 2 * (size_t)E * M * N, mm = 2 * (size_t)E * p->m * p->m;
  p->off_hi[0] = l.take(x);
  p->off_hi[1] = l.take(x);
  p->off_lo = l.take(x);
  p->off_p = l.take(mm);
  p->off_q = l.take(mm);
  p->off_norm = l.take(sizeof(double) * E * p->norm_parts);
  p->off_partial = l.take(E ? sizeof(float) * kOrthPartialFloats : 0);
  p->total = l.o;
  return MOE_OK;
}

}  // namespace moe
