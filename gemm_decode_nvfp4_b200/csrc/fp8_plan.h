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

// --------------------------------------------------------- the products

constexpr int kRows = 128;        // MMA M
constexpr int kBlockK = 128;      // k per stage, one scale block, one swizzled row
constexpr int kMaxStages = 8;
constexpr int kMaxBufs = 4;
constexpr int kScaleSlots = 16;

struct Bars {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t sfull[kScaleSlots];   // SWAP: a block's scales are in its slot
  uint64_t sempty[kScaleSlots];  //       its block has been promoted
  uint64_t acc_full[kMaxBufs];
  uint64_t acc_empty[kMaxBufs];
  uint64_t mma_done;
  uint32_t tmem_addr;
  volatile int err;
  int issued[2];  // loads of the tokens' and the weights' tiles, when their producers are done
};

template <bool SWAP_, int BN_, int PW_>
struct Cfg {
  static constexpr bool SWAP = SWAP_;
  static constexpr int BN = BN_, PW = PW_;
  static constexpr int NBUF = 512 / BN < kMaxBufs ? 512 / BN : kMaxBufs;
  static constexpr uint32_t TMEM = NBUF * BN < 32 ? 32 : NBUF * BN;
  static constexpr int COLS = BN / (PW / 4);  // accumulator columns of one thread
  static constexpr int TOK = SWAP ? BN : kRows, WROWS = SWAP ? kRows : BN;
  static constexpr int LD = SWAP ? 16 : 32;  // columns of a tensor-memory load (of 16 at a time) ...
  static constexpr int LDBUF = 2;            // ... and the register buffers for them
  static constexpr int SLOT = TOK + 4;       // floats of a scale slot: token scales, then the weight scale
  static constexpr int STAGE = (kRows + BN) * kBlockK;
  static constexpr int THREADS = (PW + 4) * 32;
  static constexpr int CTAS = BN <= 64 ? 2 : 1;  // per SM
  static constexpr int EPI = SWAP ? 0 : PW * 2176;
  static constexpr int SCALES = SWAP ? kScaleSlots * SLOT * 4 : 0;
  static constexpr int FIXED = EPI + SCALES + (int)sizeof(Bars) + 1024;
};

using S16 = Cfg<true, 16, 4>;
using S32 = Cfg<true, 32, 4>;
using S64 = Cfg<true, 64, 8>;
using S128 = Cfg<true, 128, 16>;
using L256 = Cfg<false, 256, 8>;

constexpr int kSmemMax = 232448;   // dynamic shared memory of a CTA that has the SM to itself
constexpr int kSmemHalf = 115712;  // of one that shares it with another

inline int64_t cdiv(int64_t x, int64_t y) { return (x + y - 1) / y; }

template <class C>
int stages_of(int table) {
  const int n = ((C::CTAS == 2 ? kSmemHalf : kSmemMax) - C::FIXED - table) / C::STAGE;
  return n < kMaxStages ? n : kMaxStages;
}

// CTAs of clusters of c that run at once.  A cluster stays within one GPC, so a
// few SMs are left over; in thousandths of the SMs, as the occupancy of an empty
// kernel with this shared memory has it on one B200 (148 SMs).  (Of this kernel
// the driver reports one CTA per SM whatever its size, but two do run.)
template <class C>
int64_t resident(int c, int sms) {
  constexpr int one[9] = {0, 1000, 1000, 912, 891, 878, 891, 709, 810};
  constexpr int two[9] = {0, 1000, 1000, 942, 959, 945, 912, 875, 891};
  return (int64_t)sms * C::CTAS * (C::CTAS == 2 ? two[c] : one[c]) / 1000;
}

// A tile's width (Cfg::BN) and the CTAs that share its blocks of k.
struct Choice {
  int bn, splits;
};

struct Product {
  int64_t T, E, N, K;  // rows of X, experts (1: dense)
  bool grouped;
  int sms;
  int64_t active, kb;  // experts that may have rows, 0: dense; blocks of k

  Product(int64_t T_, int64_t E_, int64_t N_, int64_t K_, bool grouped_, int sms_)
      : T(T_), E(E_), N(N_), K(K_), grouped(grouped_), sms(sms_), active(grouped_ ? (E_ < T_ ? E_ : T_) : 0),
        kb(cdiv(K_, kBlockK)) {}

  // Token tiles of `tok` rows: of a grouped call an estimate (half a tile per
  // expert is empty), or the most there can be.
  template <class C>
  int64_t tiles(bool most) const {
    const int64_t mt = grouped ? T / C::TOK + (most ? E : (active + 1) / 2) : cdiv(T, C::TOK);
    return mt * cdiv(N, C::WROWS);
  }

  // Estimated microseconds of a configuration with c CTAs sharing each tile's k:
  // waves of CTAs times blocks of k, and the time to read the weights
  // (6.3 TB/s, which nine tenths of the SMs reach); the longer one counts in full,
  // the other one, mostly behind it, a quarter.
  // Measured on one B200 (M 1 to 1024, N 1024 to 17408, K 2048 to 17408): a block
  // of k takes `alone` us with one CTA on an SM and `full` with all SMs (and both
  // CTAs of one) busy, a tile's epilogue `store`, adding the shares of a split
  // 0.8 and 0.025 per token of the tile.  The choices by this rule ran within 7%
  // of the best one of each of 59 shapes there but for one (19%); by tile width alone
  // (M <= 16: 16 tokens, and so on) they were up to 2.7 times slower.  K below 2048
  // and M above 1024 were not measured against the other configurations.
  template <class C>
  double estimate(int c) const {
    constexpr double alone = C::BN == 16 ? 0.19 : C::BN == 32 ? 0.24 : C::BN == 64 ? 0.40 : C::BN == 128 ? 0.38 : 0.40;
    constexpr double full = C::BN == 16 ? 0.29 : C::BN == 32 ? 0.36 : C::BN == 64 ? 0.52 : C::BN == 128 ? 0.45 : 0.51;
    constexpr double store = C::BN == 16 ? 0.5 : C::BN == 32 ? 0.7 : C::BN == 64 ? 1.0 : 1.5;
    const int64_t slots = resident<C>(c, sms), ctas = tiles<C>(false) * c;
    const double per_block = ctas > (C::BN >= 128 ? 100 : sms) ? full : alone;
    const double work = (double)cdiv(ctas, slots) * ((double)cdiv(kb, c) * per_block + store);
    const double bytes = (double)(active ? active : 1) * N * K + (double)T * (K + 2.0 * N);
    const double stream = bytes / 6.3e6 * (ctas < 0.92 * sms ? 0.92 * sms / ctas : 1.0);
    return (work > stream ? work + 0.25 * stream : stream + 0.25 * work) + (c > 1 ? 0.8 + 0.025 * C::BN : 0.0);
  }

  // bytes of shared memory for the table of a grouped call: tiles before, first rows, row ends
  int table() const { return grouped ? 3 * (int)(E + 1) * 4 : 0; }

  template <class C>
  void consider(double& best, Choice& choice) const {
    if (stages_of<C>(table()) < 2) return;
    // (a grouped call's tiles are not known here, so a cluster per tile cannot be)
    const int most = C::SWAP && !grouped ? (int)(kb < 8 ? kb : 8) : 1;
    for (int c = 1; c <= most; ++c) {
      if (c > 1 && tiles<C>(true) * c > 4 * (int64_t)sms) break;  // enough tiles to fill the GPU
      const double t = estimate<C>(c);
      if (t < best) {
        best = t;
        choice = {C::BN, c};
      }
    }
  }

  Choice choose() const {
    double best = 1e300;
    Choice choice{0, 1};
    consider<S16>(best, choice);
    consider<S32>(best, choice);
    consider<S64>(best, choice);
    consider<S128>(best, choice);
    consider<L256>(best, choice);
    return choice;
  }
};

}  // namespace plan
}  // namespace nvfp4
