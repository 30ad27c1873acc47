// Runs drain_ring (csrc/fp8_drain.h) on a model of the product's stage ring and of the
// norm's row ring: barriers with pending arrivals and outstanding bytes, copies that land
// in any order, roles that stop at any point as they do after a wait gave up.
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "fp8_drain.h"

namespace {

struct Barrier {
  int phase = 0, pending = 1;
  long tx = 0;
  bool bad = false;
  void settle() {
    if (pending == 0 && tx == 0) ++phase, pending = 1;
  }
  void arm(long bytes) {
    if (pending != 1) bad = true;  // an arrival more than the phase expects
    --pending;
    tx += bytes;
    settle();
  }
  void land(long bytes) {
    tx -= bytes;
    settle();
  }
};

struct Copy {
  int slot;
  long bytes;
};

struct Ring {
  std::vector<Barrier> bar;
  std::vector<Copy> flight;
  std::mt19937& rng;
  Ring(int slots, std::mt19937& r) : bar(slots), rng(r) {}
  int below(int n) { return (int)(rng() % (unsigned)n); }
  void issue(int slot, long bytes) { flight.push_back({slot, bytes}); }
  void land_one() {
    if (flight.empty()) return;
    const int i = below((int)flight.size());
    bar[flight[i].slot].land(flight[i].bytes);
    flight.erase(flight.begin() + i);
  }
  // a bounded wait for a phase: copies land meanwhile; false: it would run out
  bool wait(int slot, int parity) {
    while ((bar[slot].phase & 1) == parity && !flight.empty()) land_one();
    return (bar[slot].phase & 1) != parity;
  }
  bool clean() const {
    for (const Barrier& b : bar)
      if (b.bad) return false;
    return flight.empty();
  }
};

constexpr long kA = 100, kB = 7;

// The product: producers a and b run up to `slots` loads ahead of the consumer; each
// stops after a number of steps of its own.  gave_up: no role waits any more.
bool product(std::mt19937& rng) {
  const int slots = 2 + (int)(rng() % 7), loads = 1 + (int)(rng() % 40);
  Ring ring(slots, rng);
  int a = 0, b = 0, used = 0;
  const int stop_a = (int)(rng() % (loads + 1)), stop_b = (int)(rng() % (loads + 1));
  const int stop_use = (int)(rng() % (loads + 1));
  for (int step = 0; step < 2000; ++step) {
    switch (rng() % 4) {
      case 0:
        if (a < stop_a && a < used + slots) ring.bar[a % slots].arm(kA + kB), ring.issue(a % slots, kA), ++a;
        break;
      case 1:
        if (b < stop_b && b < used + slots) ring.issue(b % slots, kB), ++b;
        break;
      case 2:
        if (used < stop_use && ring.bar[used % slots].phase > used / slots) ++used;
        break;
      default: ring.land_one();
    }
    if (rng() % 400 == 0) break;
  }
  bool ok = true;
  struct Ops {
    Ring& ring;
    bool& ok;
    void arm_b(int slot) { ring.bar[slot].arm(kB); }
    void load_b(int slot) { ring.issue(slot, kB); }
    void wait(int slot, int parity) { ok = ring.wait(slot, parity) && ok; }
  };
  nvfp4::drain_ring(a, b, slots, Ops{ring, ok});
  return ok && ring.clean();
}

// The norm: one thread fetches row n + slots once row n has been read; from the row whose
// wait gave up on, rows are gone through without waiting and nothing is fetched.
bool norm(std::mt19937& rng) {
  const int slots = 2 + (int)(rng() % 7), rows = 1 + (int)(rng() % 40), fails = (int)(rng() % (rows + 1));
  Ring ring(slots, rng);
  int fetched = 0;
  bool err = false;
  auto fetch = [&] {
    ring.bar[fetched % slots].arm(kA + kB);
    ring.issue(fetched % slots, kA);
    ring.issue(fetched % slots, kB);
    ++fetched;
  };
  while (fetched < slots && fetched < rows) fetch();
  for (int n = 0; n < rows; ++n) {
    if (n == fails) err = true;
    if (!err && !ring.wait(n % slots, (n / slots) & 1)) return false;
    if (n + slots < rows && !err) fetch();
    for (int i = ring.below(3); i > 0; --i) ring.land_one();
  }
  if (!err) return ring.clean();
  bool ok = true;
  nvfp4::drain_ring(fetched, slots, [&](int slot, int parity) { ok = ring.wait(slot, parity) && ok; });
  return ok && ring.clean();
}

}  // namespace

int main() {
  int bad_product = 0, bad_norm = 0;
  for (uint32_t seed = 0; seed < 20000; ++seed) {
    std::mt19937 rng(seed);
    bad_product += !product(rng);
    bad_norm += !norm(rng);
  }
  std::printf("product %d norm %d\n", bad_product, bad_norm);
  return 0;
}
