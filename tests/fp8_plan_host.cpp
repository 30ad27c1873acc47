// The launch rules of csrc/fp8_plan.h as C functions, for the tests.
#include "fp8_plan.h"

extern "C" void norm_rows(int64_t K, int residual, int warps2, int warps4, int* out) {
  const int warps[2] = {warps2, warps4};
  const nvfp4::plan::NormRows p = nvfp4::plan::norm_rows(K, residual != 0, warps);
  out[0] = p.wide;
  out[1] = p.threads;
  out[2] = p.per_sm;
  out[3] = p.slots;
}
