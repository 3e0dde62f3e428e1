// Host-logic driver for the sanitizer test: walks ordinary and extreme shapes
// through the workspace planners and checks that every accepted plan's regions
// are 256-byte aligned, in order and inside the total.
#include <cstdio>
#include <vector>

#include "ops_plan.hpp"

static bool ordered(const std::vector<size_t>& off, size_t total) {
  for (size_t i = 0; i < off.size(); ++i)
    if (off[i] % 256 || off[i] > total || (i && off[i] < off[i - 1])) return false;
  return true;
}

int main() {
  const int big[] = {-8, 0, 1, 8, 64, 100, 264, 2880, 4096, 14336, 32768, 1 << 20, 1 << 24, 2147483640};
  const int rows[] = {-1, 0, 1, 17, 64, 65, 300, 4096, 100000, 1 << 24, 2147483647};
  const int counts[] = {-1, 0, 1, 8, 255, 256, 257, 65536, 65537};
  long accepted = 0;
  for (int n : big)
    for (int k : big)
      for (int r : rows)
        for (int g : counts) {
          for (int f = 0; f < 4; ++f) {
            moe_gemm_shape s{r, g, n, k, f & 1, f >> 1, f & 1};
            moe::GemmPlan p;
            if (moe::make_gemm_plan(&s, &p) != moe::check_gemm_shape(&s)) return 2;
          }
          for (int rank : {8, 40, 128, 136}) {
            moe_lora_shape s{r, k, n, g, rank, 0};
            moe::LoraPlan p;
            moe::LoraBwdPlan b;
            if (moe::make_lora_plan(&s, &p) == 0) {
              ++accepted;
              if (!ordered({p.off_v, p.off_v16, p.off_partial}, p.total)) return 3;
            }
            if (moe::make_lora_backward_plan(&s, &b) == 0 &&
                !ordered({b.off_v, b.off_u16, b.off_xa16, b.off_rows, b.off_partial}, b.total))
              return 4;
          }
          moe::OrthPlan o;
          if (moe::make_orth_plan(g, n, k, &o) == 0) {
            ++accepted;
            if (!ordered({o.off_hi[0], o.off_hi[1], o.off_lo, o.off_p, o.off_q, o.off_norm, o.off_partial},
                         o.total)) return 5;
          }
        }
  std::printf("%ld\n", accepted);
  return accepted > 100 ? 0 : 6;
}
