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

extern "C" void gemm_choice(int64_t T, int64_t E, int64_t N, int64_t K, int grouped, int sms, int* out) {
  const nvfp4::plan::Choice c = nvfp4::plan::Product(T, E, N, K, grouped != 0, sms).choose();
  out[0] = c.bn;
  out[1] = c.splits;
}

// counts[bn's index 16, 32, 64, 128, 256][splits - 1] += choices over n random dense shapes:
// M 1 to 8192, N 1 to 50176, K 16 to 49600, each spread over its logarithm
extern "C" void scan_choices(int n, uint64_t seed, int sms, int* counts, int64_t* shapes) {
  auto next = [&] {
    seed = seed * 6364136223846793005ull + 1442695040888963407ull;
    return (double)(seed >> 40) / (double)(1 << 24);
  };
  for (int i = 0; i < n; ++i) {
    const int64_t M = (int64_t)__builtin_exp(next() * __builtin_log(8192.0));
    const int64_t N = (int64_t)__builtin_exp(next() * __builtin_log(50176.0));
    const int64_t K = 16 * (int64_t)__builtin_exp(next() * __builtin_log(3100.0));
    const nvfp4::plan::Choice c = nvfp4::plan::Product(M, 1, N, K, false, sms).choose();
    const int w = c.bn == 16 ? 0 : c.bn == 32 ? 1 : c.bn == 64 ? 2 : c.bn == 128 ? 3 : 4;
    const int at = w * 8 + c.splits - 1;
    // (of each pair the shape with the least work seen so far)
    if (!counts[at] || M * N * K < shapes[3 * at] * shapes[3 * at + 1] * shapes[3 * at + 2]) {
      shapes[3 * at] = M;
      shapes[3 * at + 1] = N;
      shapes[3 * at + 2] = K;
    }
    ++counts[at];
  }
}
