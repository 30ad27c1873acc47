// fp8_plan.h -- host-side choices of the 8-bit kernels' launches: rules on sizes, in
// plain C++ without CUDA, so that they can be run and checked on their own.
#pragma once

#include <cstdint>

namespace nvfp4 {
namespace plan {

// ------------------------------------------------- the norm of many rows

constexpr int kNormSlots = 8;       // most row slots of a CTA
constexpr int kNormSmem = 232448;   // shared memory of an SM for them
constexpr int kNormStatic = 2048;   // left out of each CTA's share: barriers, sums, the CTA's own 1 KB

struct NormRows {
  int wide;     // vectors of 8 columns per thread: 2 or 4
  int threads;  // of a CTA
  int per_sm;   // CTAs of an SM, 0: rows too long for two slots
  int slots;    // row slots of a CTA
};

// warps[0], warps[1]: warps that an SM's registers hold of the kernels with 2 and 4
// vectors per thread.  About 20 warps per SM with a residual and 30 without (fewer
// bytes, more arithmetic per byte; measured from 2 to 6 CTAs at K = 1040 to 16384), and
// two CTAs where the registers hold them.  A CTA has at least two row slots and, where
// that leaves two, at most half of the SM's shared memory: with all of it one CTA took
// as long or longer (4096 x 10240 with a residual: 49.8 us with two slots, 52.3 with
// five; 2048 x 20480 without, whose threads spill to L1: 39.6 against 43.0).  Two CTAs
// planned where one fits, as it was, started the second one with an empty ring: 51.7 us
// on 4096 x 10240, and 40.2 against 37.7 without a residual.
inline NormRows norm_rows(int64_t K, bool residual, const int (&warps)[2]) {
  const int64_t vecs = K / 8;
  NormRows p{vecs <= 2048 ? 2 : 4, 0, 0, 0};
  p.threads = (int)((vecs + p.wide - 1) / p.wide + 31) / 32 * 32;
  const int64_t slot = K * (residual ? 4 : 2);
  const int want = (residual ? 20 : 30) * 32 / p.threads, held = warps[p.wide == 4] * 32 / p.threads;
  int per_sm = want > 2 ? want : 2;
  if (per_sm > held) per_sm = held;
  for (int shares = per_sm > 2 ? per_sm : 2; shares > 0 && p.slots < 2; --shares) {
    p.slots = (int)((kNormSmem / shares - kNormStatic) / slot);
    p.per_sm = per_sm < shares ? per_sm : shares;
  }
  if (p.slots < 2) p.per_sm = p.slots = 0;
  if (p.slots > kNormSlots) p.slots = kNormSlots;
  return p;
}

}  // namespace plan
}  // namespace nvfp4
