// fp8_drain.h -- what a CTA of the 8-bit kernels that gave up on a wait still waits
// for before it ends.  A copy left in flight would land in shared memory that the
// next CTA of the SM owns by then.  Plain C++, so that it also runs on the host.
#pragma once

#ifdef __CUDACC__
#define NVFP4_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define NVFP4_HOST_DEVICE inline
#endif

namespace nvfp4 {

// A ring of slots with one barrier each: load n goes to slot n % slots and completes
// the barrier's phase n / slots.  A load has two parts, issued by two producers: `a`,
// whose producer arms the barrier for the bytes of both, and `b`.  issued_a and
// issued_b loads were issued when both producers stopped; each load from `slots` on
// only after the one before it in its slot had been consumed, so all but the last
// `slots` loads have landed.
//   ops.arm_b(slot)         arms the barrier for the bytes of part b alone
//   ops.load_b(slot)        issues a part b that its producer no longer did
//   ops.wait(slot, parity)  waits (bounded) for the phase with this parity
// Every phase that was begun so completes, and with it every copy.
template <class Ops>
NVFP4_HOST_DEVICE void drain_ring(int issued_a, int issued_b, int slots, Ops&& ops) {
  const int end = issued_a > issued_b ? issued_a : issued_b;
  for (int n = end > slots ? end - slots : 0; n < end; ++n) {
    const int slot = n % slots;
    if (n >= issued_a) ops.arm_b(slot);
    if (n >= issued_b) ops.load_b(slot);
    ops.wait(slot, (n / slots) & 1);
  }
}

// The same for loads of one part.
template <class Wait>
NVFP4_HOST_DEVICE void drain_ring(int issued, int slots, Wait&& wait) {
  for (int n = issued > slots ? issued - slots : 0; n < issued; ++n) wait(n % slots, (n / slots) & 1);
}

}  // namespace nvfp4
