// fp8_gemm.cu -- E4M3 matrix product with one fp32 scale per 128, dense and
// grouped by expert, on the sm_100a tensor cores (include/fp8.h):
//   Y[m, n] = bf16( sum_b sx[m, b] sw[n / 128, b] * sum_{k in block b} qx[m, k] qw[n, k] )
//
// The tensor core has no fp32 block scales, so every block of 128 k is one
// accumulation of its own (four tcgen05.mma kind::f8f6f4 of K = 32 into a fresh
// tensor-memory accumulator), which the promotion warps read back and add to
// fp32 registers times sx * sw.  Accumulators are multiply buffered, so the
// next blocks' MMAs run while one is being promoted.
//
// Two operand orders:
//   SWAP  the MMA's 128 rows are weight rows, its BN columns tokens.  One weight
//         scale per block covers the whole tile; a thread owns one weight row
//         and multiplies column j by token j's scale.  For few tokens: a tile
//         streams 128 weight rows whatever M is.
//   !SWAP the rows are tokens, the BN = 256 columns weight rows.  A thread owns
//         128 columns of one token, so its scale is one product per block.  For
//         many tokens.
// Roles per CTA: PW promotion warps; two producer threads (TMA tiles of the tokens
// and of the weights); one MMA warp; SWAP: a warp that copies the block's scales
// into a ring of slots with cp.async (!SWAP: a warp without a role, part of the
// warpgroup whose registers setmaxnreg moves).  Persistent over tiles; the stage
// ring runs on across tiles.  With few tiles a cluster of `splits` CTAs shares a
// tile's blocks of k and adds the partial sums in rank order through distributed
// shared memory.  Every wait is bounded.
//
// What bounds it (one B200): few tokens, the weight stream (one token through
// 17408 x 5120: 17.1 us, 81% of the copy rate); many, the power limit (4096 tokens
// through 17408 x 5120: 350 to 370 us at 1.5 GHz in a loop, 298 us or 2.45 PFLOP/s in
// a short burst) and L2 to SM: bulk copies alone reach 58 bytes per cycle and SM, so a
// 128 x 256 x 128 block's 48 KB take 847 cycles against 512 of MMAs, and a block
// takes 850 to 880.  Pairs of SMs with 256 x 256 tiles, which load a third less,
// ran at 330 us in bursts: the chain commit, promotion, arrival at the other SM, next
// MMA is longer than two accumulators cover.  Short K and middle batches: the stores
// of a tile (1.5 us) and the sums of a split.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "fp8_drain.h"
#include "fp8_plan.h"
#include "nvfp4_device.cuh"
#include "nvfp4_kernels.h"
#include "sm100_ptx.cuh"
#include "tc_host.h"

namespace nvfp4 {

// CTAs whose pipeline wait ran past its limit, and calls with group ends out of order or range.
__device__ unsigned int g_fp8_wait_timeouts = 0;
__device__ unsigned int g_fp8_bad_offsets = 0;

namespace {

using plan::Bars;
using plan::kBlockK;
using plan::kRows;
using plan::kScaleSlots;

constexpr long long kWaitClocks = 4000000000ll;  // 2.0 s at 1.965 GHz, 2.7 s at 1.5 GHz
constexpr uint64_t kDrainNs = 2000000000ull;
constexpr int kGroupTiles = 16;   // token tiles that share a weight tile in the tile order

struct Args {
  const float* sx;
  const float* sw;
  const int* offsets;  // null: dense
  uint16_t* Y;
  int64_t ldy;
  int T, N, K, kb, E, nt;  // rows of X; kb = blocks of k; nt = weight tiles
  int stages, splits, static_weights;
};

// !SWAP: 168 registers a thread (384 threads) do not hold 128 accumulators and
// the loads in flight, and a spill costs a trip to L2 (shared memory leaves no
// L1), so the promotion warps take over registers of the other warpgroup:
// 256 x 224 + 128 x 56 = 384 x 168.
constexpr int kRegsMore = 224, kRegsLess = 56;

// Wait for the phase with the given parity, kWaitClocks at most; then the CTA's
// error is recorded and its other waits fail too.
__device__ __forceinline__ bool wait_or_fail(uint64_t* bar, uint32_t parity, Bars* bars) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (ptx::mbar_try_wait(bar, parity)) return true;
    if (bars->err) return false;
    if (clock64() - t0 > kWaitClocks) {
      bars->err = 1;
      atomicAdd(&g_fp8_wait_timeouts, 1u);
      return false;
    }
  }
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// The warp waits for the phase (all lanes poll; with one lane's tries the products
// took 10 to 15% longer);
// the vote makes the answer the warp's, so that code after it stays convergent.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Bars* bars) {
  const bool ok = __all_sync(0xFFFFFFFFu, wait_or_fail(bar, parity, bars));
  __syncwarp();
  return ok;
}

// four fp32 at the same shared-memory offset as `local` in the cluster's CTA `rank`
__device__ __forceinline__ float4 ld_cluster_v4(const float* local, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(ptx::cluster_addr(local, rank))
               : "memory");
  return v;
}

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// kind::f8f6f4 with E4M3 A and B (format code 0), fp32 accumulator, both K-major
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void cp_async4(float* dst, const float* src, bool in) {
  const int n = in ? 4 : 0;  // 0 bytes read: the word is zero filled
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(ptx::smem_u32(dst)), "l"(src), "r"(n) : "memory");
}

// this thread's arrival on `bar` once its cp.async so far have landed (counted
// in the barrier's expected arrivals)
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(ptx::smem_u32(bar)) : "memory");
}

// Wait for this thread's tensor-memory loads; the registers pass through, so
// nothing that reads them moves above it.
template <int N>
__device__ __forceinline__ void ld_wait(uint32_t (&r)[N]) {
  ptx::tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[16]) { ptx::tmem_ld_16cols(addr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[32]) {
  ptx::tmem_ld_16cols(addr, *reinterpret_cast<uint32_t(*)[16]>(&r[0]));
  ptx::tmem_ld_16cols(addr + 16, *reinterpret_cast<uint32_t(*)[16]>(&r[16]));
}

// Pairs of fp32 in a 64-bit register, for the packed fp32 arithmetic.
__device__ __forceinline__ uint64_t pack_f32(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ float2 unpack_f32(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}

// a += (t0, t1) * s
__device__ __forceinline__ void fma2(uint64_t& a, uint32_t t0, uint32_t t1, uint64_t s) {
  asm("{\n\t.reg .b64 x;\n\tmov.b64 x, {%1, %2};\n\tfma.rn.f32x2 %0, x, %3, %0;\n\t}"
      : "+l"(a)
      : "r"(t0), "r"(t1), "l"(s));
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t v;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
  return v;
}

// The scale sx[m, kb] * sw[n / 128, kb] of one thread's row and columns, block by
// block: four blocks are held, and the next four loaded while they are used.
// (Every lane of a warp has its own row, so a load touches 32 sectors; through a
// warp that copied them into shared memory block by block it took longer than
// the block's MMAs.)
struct ScaleStream {
  const float *x, *w;
  float4 have, nx, nw;
  bool vec;
  __device__ __forceinline__ void fetch(int kb, int kbs) {
    if (vec) {  // rows of whole 16-byte groups
      nx = *reinterpret_cast<const float4*>(x + kb);
      nw = *reinterpret_cast<const float4*>(w + kb);
    } else {
      const int b = min(kb + 1, kbs - 1), c = min(kb + 2, kbs - 1), d = min(kb + 3, kbs - 1);
      nx = make_float4(x[kb], x[b], x[c], x[d]);
      nw = make_float4(w[kb], w[b], w[c], w[d]);
    }
  }
  __device__ __forceinline__ void start(const float* x_, const float* w_, int kbs, bool vec_) {
    x = x_;
    w = w_;
    vec = vec_;
    fetch(0, kbs);
  }
  __device__ __forceinline__ float next(int kb, int kbs) {
    if ((kb & 3) == 0) {
      have = make_float4(nx.x * nw.x, nx.y * nw.y, nx.z * nw.z, nx.w * nw.w);
      if (kb + 4 < kbs) fetch(kb + 4, kbs);
    }
    const float v = have.x;
    have.x = have.y;
    have.y = have.z;
    have.z = have.w;
    return v;
  }
};

// One output tile: its expert's weight rows from w0, tokens [m0, mend).
struct Tile {
  int e, m0, mend, n0;
};

// Tile t of the order: experts in turn; within one, groups of kGroupTiles token
// tiles; within a group, weight tile by weight tile.  Neighbouring CTAs so share
// weight tiles, and a group's tokens stay in L2.  pre (grouped): token tiles
// before each expert; off: its first row (E + 1 each).
template <int TILE, int WROWS>
__device__ __forceinline__ Tile tile_of(int t, const Args& a, const int* pre, const int* off) {
  Tile r;
  int lo = 0, mt, first = 0, mend = a.T;
  if (a.offsets) {
    int hi = a.E;  // the expert e with pre[e] * nt <= t < pre[e + 1] * nt
    const int q = t / a.nt;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= q) lo = mid; else hi = mid;
    }
    t -= pre[lo] * a.nt;
    mt = pre[lo + 1] - pre[lo];
    first = off[lo];
    mend = off[a.E + 1 + lo];
  } else {
    mt = (a.T + TILE - 1) / TILE;
  }
  const int group = t / (kGroupTiles * a.nt);
  const int in = min(kGroupTiles, mt - group * kGroupTiles);
  t -= group * kGroupTiles * a.nt;
  const int n = t / in;
  r.e = lo;
  r.m0 = first + (group * kGroupTiles + t - n * in) * TILE;
  r.mend = mend;
  r.n0 = n * WROWS;
  return r;
}

// Stores COLS columns of the warp's 32 tokens (one per lane) from column n0 on, 32
// columns at a time through 2176 bytes of shared memory, so that lanes store
// neighbouring columns.
template <int COLS>
__device__ __forceinline__ void store_rows(const Args& a, const uint64_t (&acc)[COLS / 2], uint8_t* stg, int m0, int mend,
                                           int n0, int lane) {
  const bool vec = ((reinterpret_cast<uintptr_t>(a.Y) & 15u) == 0) && (a.ldy & 7) == 0;
  // aligned rows: the 16-byte pieces of a row's 64 bytes are rotated by half the
  // row, against bank conflicts
  auto piece = [&](int row, int p) { return stg + row * 64 + 16 * ((p + (row >> 1)) & 3); };
  // rows at any address: 17 words apart
  uint32_t* const words = reinterpret_cast<uint32_t*>(stg);
  const uint16_t* const halves = reinterpret_cast<const uint16_t*>(stg);
#pragma unroll
  for (int c = 0; c < COLS / 32; ++c) {
    const int n = n0 + 32 * c;
    uint32_t o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const __nv_bfloat162 h = __float22bfloat162_rn(unpack_f32(acc[16 * c + i]));
      o[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if (vec && n + 32 <= a.N) {
#pragma unroll
      for (int p = 0; p < 4; ++p)
        *reinterpret_cast<uint4*>(piece(lane, p)) = make_uint4(o[4 * p], o[4 * p + 1], o[4 * p + 2], o[4 * p + 3]);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2), p = lane & 3;
        if (m0 + r < mend)
          *reinterpret_cast<uint4*>(a.Y + (int64_t)(m0 + r) * a.ldy + n + 8 * p) =
              *reinterpret_cast<const uint4*>(piece(r, p));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) words[lane * 17 + i] = o[i];
      __syncwarp();
      if (n + 32 <= a.N) {
        // a row's 16-byte aligned pieces (three, or four of an aligned row), put
        // together from the words around them, then the columns before and behind
        // them, eight in all (column by column in all, one row of 32 at a time:
        // 2000 x 4099 x 2048 in 30.5 us, 19.9 with N = 4096)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * i + (lane >> 2);
          uint16_t* const dst = a.Y + (int64_t)(m0 + r) * a.ldy + n;
          const int head = (int)(-(reinterpret_cast<uintptr_t>(dst) >> 1) & 7), e = head + 8 * (lane & 3);
          if (m0 + r < mend && e + 8 <= 32) {
            const uint32_t* src = words + r * 17 + (e >> 1);
            uint4 v = make_uint4(src[0], src[1], src[2], src[3]);
            if (e & 1)
              v = make_uint4(__funnelshift_r(v.x, v.y, 16), __funnelshift_r(v.y, v.z, 16),
                             __funnelshift_r(v.z, v.w, 16), __funnelshift_r(v.w, src[4], 16));
            *reinterpret_cast<uint4*>(dst + e) = v;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + (lane >> 3), p = lane & 7;
          uint16_t* const dst = a.Y + (int64_t)(m0 + r) * a.ldy + n;
          const int head = (int)(-(reinterpret_cast<uintptr_t>(dst) >> 1) & 7), e = p < head ? p : 24 + p;
          if (m0 + r < mend && head) dst[e] = halves[r * 34 + e];
        }
      } else if (n + lane < a.N) {
        uint16_t* dst = a.Y + (int64_t)m0 * a.ldy + n + lane;
#pragma unroll 8
        for (int r = 0; r < 32; ++r, dst += a.ldy)
          if (m0 + r < mend) *dst = halves[r * 34 + lane];
      }
    }
    __syncwarp();
  }
}

// The loads that a CTA which gave up still has in flight.  (Out of line and at the end
// of the kernel: elsewhere it changed the main loop's registers, 3% of some calls.)
template <class C>
__device__ __noinline__ void drain(Bars* bars, int stages, const CUtensorMap* tmap_w, uint8_t* dst_w) {
  struct Ops {
    Bars* bars;
    const CUtensorMap* tmap_w;
    uint8_t* dst_w;
    __device__ void arm_b(int st) { ptx::mbar_arrive_expect_tx(&bars->full[st], C::WROWS * kBlockK); }
    __device__ void load_b(int st) { ptx::tma_load_2d(dst_w + st * C::STAGE, tmap_w, &bars->full[st], 0, 0); }
    __device__ void wait(int st, int parity) { ptx::mbar_wait(&bars->full[st], parity, kDrainNs); }
  };
  drain_ring(bars->issued[0], bars->issued[1], stages, Ops{bars, tmap_w, dst_w});
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::CTAS)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_x,
                    const Args a) {
  constexpr bool SWAP = C::SWAP;
  constexpr int BN = C::BN, PW = C::PW, NBUF = C::NBUF, COLS = C::COLS;
  constexpr uint32_t kIdesc = idesc_e4m3(kRows, BN);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (((ptx::smem_u32(smem_raw) + 1023u) & ~1023u) - ptx::smem_u32(smem_raw));
  uint8_t* epi = smem + a.stages * C::STAGE;
  float* scales = reinterpret_cast<float*>(epi + C::EPI);
  Bars* bars = reinterpret_cast<Bars*>(epi + C::EPI + C::SCALES);
  int* pre = reinterpret_cast<int*>(bars + 1);  // grouped: [E + 1] token tiles before
  int* off = pre + a.E + 1;                     // then [E + 1] first rows, [E + 1] row ends

  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = a.splits > 1 ? (int)ptx::cluster_ctarank() : 0;
  const int kb0 = (int)((int64_t)a.kb * rank / a.splits), kb1 = (int)((int64_t)a.kb * (rank + 1) / a.splits);
  const int S = a.stages;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(&bars->full[i], 1);
      ptx::mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; SWAP && i < kScaleSlots; ++i) {
      ptx::mbar_init(&bars->sfull[i], 32);
      ptx::mbar_init(&bars->sempty[i], PW);
    }
    for (int i = 0; i < NBUF; ++i) {
      ptx::mbar_init(&bars->acc_full[i], 1);
      ptx::mbar_init(&bars->acc_empty[i], PW);
    }
    ptx::mbar_init(&bars->mma_done, 1);
    bars->err = 0;
    ptx::fence_mbar_init();
  }
  if (warp == PW && lane == 0) {
    ptx::prefetch_tmap(&tmap_w);
    ptx::prefetch_tmap(&tmap_x);
  }
  if (warp == PW + 1) {
    ptx::tmem_alloc(&bars->tmem_addr, C::TMEM);
    ptx::tmem_relinquish();
  }
  if (a.offsets) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 0) {
      // token tiles before each expert, 32 experts at a time; ends are clamped
      // to the rows there are, so a bad one cannot reach outside X or Y
      int before = 0, top = 0;  // tiles, and the largest row end, of the experts so far
      bool bad = false;
      for (int e0 = 0; e0 < a.E; e0 += 32) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < a.E) {
          const int u = a.offsets[e], v = a.offsets[e + 1];
          lo = min(max(u, 0), a.T);
          hi = min(max(v, 0), a.T);
          bad |= u < 0 || v < u || v > a.T;
        }
        // (an expert starts no earlier than the ones before it end: with any
        // offsets the rows of two experts are apart)
        int reach = hi;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xFFFFFFFFu, reach, o);
          if (lane >= o) reach = max(reach, up);
        }
        const int left = __shfl_up_sync(0xFFFFFFFFu, reach, 1);
        lo = max(lo, max(top, lane ? left : 0));
        hi = max(hi, lo);
        top = max(top, __shfl_sync(0xFFFFFFFFu, reach, 31));
        if (e >= a.E) hi = lo;
        const int tiles = (hi - lo + C::TOK - 1) / C::TOK;
        int sum = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xFFFFFFFFu, sum, o);
          if (lane >= o) sum += up;
        }
        if (e < a.E) {
          pre[e + 1] = before + sum;
          off[e] = lo;
          off[a.E + 1 + e] = hi;
        }
        before += __shfl_sync(0xFFFFFFFFu, sum, 31);
      }
      bad = __any_sync(0xFFFFFFFFu, bad);
      if (lane == 0) {
        pre[0] = 0;
        if (bad && blockIdx.x == 0) atomicAdd(&g_fp8_bad_offsets, 1u);
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = bars->tmem_addr;
  // (after the allocation: a dependent's CTA that held tensor memory while this
  // one waited for it would never let either finish)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tiles = a.nt * (a.offsets ? pre[a.E] : (a.T + C::TOK - 1) / C::TOK);
  const int first = blockIdx.x / a.splits, step = gridDim.x / a.splits;

  if (warp >= PW) {
   if constexpr (!SWAP) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLess));
   if (warp == PW || warp == PW + 3) {
    // --------------------------------------------------------------- producers
    // One thread for the tokens' tiles, one for the weights'.  (A wait, the
    // barrier's byte count and two loads of one thread took longer than the
    // block's MMAs.)
    const bool weights = warp == PW + 3;
    if (lane == 0) {
      // With static weights their first stages stream before the preceding work is
      // done.  (Every bounded wait comes after the wait for that work, which may
      // take any time.)
      bool waited = a.offsets != nullptr;
      if (!waited && !(weights && a.static_weights)) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        waited = true;
      }
      const CUtensorMap* map = weights ? &tmap_w : &tmap_x;
      uint8_t* const dst0 = smem + (SWAP == weights ? 0 : kRows * kBlockK);  // operand A is first
      int st = 0, ph = 0, issued = 0;  // ph: parity that `empty` completes next
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        const Tile w = tile_of<C::TOK, C::WROWS>(t, a, pre, off);
        const int row = weights ? w.e * a.N + w.n0 : w.m0;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (issued == S && !waited) asm volatile("griddepcontrol.wait;" ::: "memory");
          if (issued >= S && !wait_or_fail(&bars->empty[st], ph, bars)) {
            ok = false;
            break;
          }
          if (!weights) ptx::mbar_arrive_expect_tx(&bars->full[st], C::STAGE);
          ptx::tma_load_2d(dst0 + st * C::STAGE, map, &bars->full[st], kb * kBlockK, row);
          ++issued;
          if (++st == S) {
            st = 0;
            if (issued > S) ph ^= 1;
          }
        }
      }
      bars->issued[weights] = issued;
    }
    __syncwarp();
   } else if (SWAP && warp == PW + 2) {
    // ------------------------------------------------------------------ scales
    // each block's token scales and weight scale into the next slot
    int slot = 0, ph = 1;
    bool ok = true;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int t = first; t < tiles && ok; t += step) {
      const Tile w = tile_of<C::TOK, C::WROWS>(t, a, pre, off);
      const float* sw = a.sw + (int64_t)(w.e * ((a.N + 127) / 128) + w.n0 / 128) * a.kb;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = warp_wait(&bars->sempty[slot], ph, bars);
        if (!ok) break;
        float* d = scales + slot * C::SLOT;
#pragma unroll
        for (int i = 0; i < (C::TOK + 31) / 32; ++i) {
          const int j = lane + 32 * i, m = w.m0 + j;
          if (C::TOK % 32 == 0 || j < C::TOK)
            cp_async4(d + j, a.sx + (int64_t)min(m, a.T - 1) * a.kb + kb, m < a.T);
        }
        if (lane == 0) cp_async4(d + C::TOK, sw + kb, true);
        cp_async_arrive(&bars->sfull[slot]);
        if (++slot == kScaleSlots) slot = 0, ph ^= 1;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
   } else if (warp == PW + 1) {
    // -------------------------------------------------------------- MMA issuer
    // (the whole warp walks the blocks and one elected lane issues: in a branch
    // of one lane the descriptors would have to be moved to uniform registers
    // before every MMA)
    int st = 0, ph = 0, buf = 0, bph = 1;
    bool ok = true;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int t = first; t < tiles && ok; t += step) {
      for (int kb = kb0; kb < kb1; ++kb) {
        // (parity 1 passes at once on a fresh barrier: every buffer starts free)
        ok = warp_wait(&bars->full[st], ph, bars) && warp_wait(&bars->acc_empty[buf], bph, bars);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint32_t a0 = ptx::smem_u32(smem) + st * C::STAGE, b0 = a0 + kRows * kBlockK;
        const uint64_t da = ptx::sw128_kmajor_desc(a0), db = ptx::sw128_kmajor_desc(b0);
        const uint32_t d = tmem + buf * BN;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 32 bytes on: 2 in the descriptor's 16-byte units
            mma_f8(d, da + 2 * kk, db + 2 * kk, kIdesc, kk != 0);
          ptx::mma_commit(&bars->acc_full[buf]);
          ptx::mma_commit(&bars->empty[st]);
        }
        __syncwarp();
        if (++st == S) st = 0, ph ^= 1;
        if (++buf == NBUF) buf = 0, bph ^= 1;
      }
    }
    // arrives when every MMA above is done, so that tensor memory is never
    // freed under one (also on the error path)
    if (elect_one()) ptx::mma_commit(&bars->mma_done);
    __syncwarp();
    if (lane == 0) ptx::mbar_wait(&bars->mma_done, 0, kDrainNs);
    __syncwarp();
   }
  } else {
    // --------------------------------------------------------------- promotion
    static_assert(SWAP || PW == 8, "registers are split for eight promotion warps");
    if constexpr (!SWAP) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMore));
    const int quarter = warp & 3, part = warp >> 2;
    const int row = 32 * quarter + lane, col0 = part * COLS;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * quarter) << 16) + col0;
    int buf = 0, bph = 0, slot = 0, sph = 0;
    bool ok = true;
    [[maybe_unused]] const bool scale_vec =
        a.kb % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.sx) | reinterpret_cast<uintptr_t>(a.sw)) & 15) == 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the scales and Y
    for (int t = first; t < tiles && ok; t += step) {
      uint64_t acc[COLS / 2];
#pragma unroll
      for (int j = 0; j < COLS / 2; ++j) acc[j] = 0;
      const Tile w = tile_of<C::TOK, C::WROWS>(t, a, pre, off);
      [[maybe_unused]] ScaleStream scale;
      if constexpr (!SWAP) {
        const int m = min(w.m0 + row, a.T - 1);
        const int nb = (a.N + 127) / 128, n = min(w.n0 / 128 + part, nb - 1);
        scale.start(a.sx + (int64_t)m * a.kb, a.sw + (int64_t)(w.e * nb + n) * a.kb, a.kb, scale_vec);
      }
      for (int kb = kb0; kb < kb1; ++kb) {
        uint64_t srow = 0, sw2 = 0;
        const float* sc = nullptr;
        if constexpr (SWAP) {
          ok = warp_wait(&bars->sfull[slot], sph, bars) && warp_wait(&bars->acc_full[buf], bph, bars);
          sc = scales + slot * C::SLOT;
          sw2 = pack_f32(sc[C::TOK], sc[C::TOK]);
        } else {
          const float v = scale.next(kb, a.kb);
          srow = pack_f32(v, v);
          ok = warp_wait(&bars->acc_full[buf], bph, bars);
        }
        if (!ok) break;
        ptx::tc_fence_after();
        constexpr int LD = COLS < C::LD ? COLS : C::LD, NLD = COLS / LD, NR = NLD < C::LDBUF ? NLD : C::LDBUF;
        uint32_t r[NR][LD];
        tmem_ld(lane_addr + buf * BN, r[0]);
#pragma unroll
        for (int c = 0; c < NLD; ++c) {
          ld_wait(r[c % NR]);
          if (c + 1 == NLD) {  // all of it read: the MMAs may have the accumulator back
            ptx::tc_fence_before();
            if (elect_one()) ptx::mbar_arrive(&bars->acc_empty[buf]);
          }
          if (c + 1 < NLD) tmem_ld(lane_addr + buf * BN + LD * (c + 1), r[(c + 1) % NR]);
#pragma unroll
          for (int j = 0; j < LD / 2; ++j) {
            const uint64_t s =
                SWAP ? mul2(*reinterpret_cast<const uint64_t*>(sc + col0 + LD * c + 2 * j), sw2) : srow;
            fma2(acc[LD / 2 * c + j], r[c % NR][2 * j], r[c % NR][2 * j + 1], s);
          }
        }
        if (++buf == NBUF) buf = 0, bph ^= 1;
        if constexpr (SWAP) {
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&bars->sempty[slot]);
          if (++slot == kScaleSlots) slot = 0, sph ^= 1;
        }
      }
      if (!ok) break;
      if constexpr (SWAP) {
        if (a.splits > 1) {
          // partial sums to the (now idle) stage memory, [token][weight row]
          float* part_sum = reinterpret_cast<float*>(smem);
#pragma unroll
          for (int j = 0; j < COLS / 2; ++j) {
            const float2 v = unpack_f32(acc[j]);
            part_sum[(col0 + 2 * j) * kRows + row] = v.x;
            part_sum[(col0 + 2 * j + 1) * kRows + row] = v.y;
          }
        } else if (w.n0 + row < a.N) {
#pragma unroll
          for (int j = 0; j < COLS; ++j) {
            const int m = w.m0 + col0 + j;
            if (m < w.mend) {
              const __nv_bfloat16 o = __float2bfloat16_rn(j & 1 ? unpack_f32(acc[j / 2]).y : unpack_f32(acc[j / 2]).x);
              a.Y[(int64_t)m * a.ldy + w.n0 + row] = *reinterpret_cast<const uint16_t*>(&o);
            }
          }
        }
      } else {
        store_rows<COLS>(a, acc, epi + warp * 2176, w.m0 + 32 * quarter, w.mend,
                         w.n0 + col0, lane);
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == PW + 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM);
  }
  if constexpr (SWAP) {
    if (a.splits > 1) {
      // every CTA of the cluster has its partial sums in shared memory (one tile
      // per cluster); each adds and stores its share of the tile, in rank order
      ptx::cluster_sync();
      if (!bars->err && first < tiles) {
        const Tile w = tile_of<C::TOK, C::WROWS>(first, a, pre, off);
        const float* part_sum = reinterpret_cast<const float*>(smem);
        // four weight rows of one token at a time; all shares are asked for before
        // the first is added
        const int live = min(BN, w.mend - w.m0) * (kRows / 4);
        const bool vec = ((reinterpret_cast<uintptr_t>(a.Y) & 7u) == 0) && (a.ldy & 3) == 0;
        for (int i = threadIdx.x + rank * C::THREADS; i < live; i += C::THREADS * a.splits) {
          float4 v[8];
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (r < a.splits) v[r] = ld_cluster_v4(part_sum + 4 * i, r);
          float4 sum = v[0];
#pragma unroll
          for (int r = 1; r < 8; ++r)
            if (r < a.splits) {
              sum.x += v[r].x;
              sum.y += v[r].y;
              sum.z += v[r].z;
              sum.w += v[r].w;
            }
          const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x, sum.y), hi = __floats2bfloat162_rn(sum.z, sum.w);
          const uint2 o = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
          const int m = w.m0 + i / (kRows / 4), n = w.n0 + 4 * (i % (kRows / 4));
          uint16_t* dst = a.Y + (int64_t)m * a.ldy + n;
          if (vec && n + 4 <= a.N) {
            *reinterpret_cast<uint2*>(dst) = o;
          } else {
            if (n < a.N) dst[0] = (uint16_t)o.x;
            if (n + 1 < a.N) dst[1] = (uint16_t)(o.x >> 16);
            if (n + 2 < a.N) dst[2] = (uint16_t)o.y;
            if (n + 3 < a.N) dst[3] = (uint16_t)(o.y >> 16);
          }
        }
      }
      ptx::cluster_sync();
    }
  }
  // (every role has stopped: no load is issued and no wait gives up any more)
  if (threadIdx.x == 0 && bars->err) drain<C>(bars, S, &tmap_w, smem + (SWAP ? 0 : kRows * kBlockK));
}

struct Launch {
  const uint8_t* x;
  const uint8_t* w;
  Args a;
  plan::Product p;
  cudaStream_t stream;

  template <class C>
  cudaError_t run(int splits) const {
    static tc::SmemOptIn opt;
    Args b = a;
    b.splits = splits;
    b.nt = (int)plan::cdiv(a.N, C::WROWS);
    b.stages = plan::stages_of<C>(p.table());
    CUtensorMap mw, mx;
    if (!tc::make_tmap_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, (uint64_t)a.K, (uint64_t)a.E * a.N, (uint64_t)a.K,
                          kBlockK, C::WROWS, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !tc::make_tmap_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, (uint64_t)a.K, (uint64_t)a.T, (uint64_t)a.K, kBlockK,
                          C::TOK, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
    const int smem = C::FIXED + p.table() + b.stages * C::STAGE;
    const void* fn = (const void*)fp8_gemm_kernel<C>;
    cudaError_t e = opt.ensure(fn, smem);
    if (e != cudaSuccess) return e;
    const int64_t n = p.tiles<C>(true), slots = (int64_t)p.sms * C::CTAS;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(splits > 1 ? n * splits : n < slots ? n : slots));
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)splits, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    void* args[] = {&mw, &mx, &b};
    return cudaLaunchKernelExC(&cfg, fn, args);
  }
};

}  // namespace

cudaError_t launch_fp8_gemm(const uint8_t* x, const float* sx, const uint8_t* w, const float* sw, const int* offsets,
                            uint16_t* Y, int64_t ldy, int64_t T, int64_t E, int64_t N, int64_t K, bool static_weights,
                            int sms, cudaStream_t stream) {
  Args a{};
  a.sx = sx;
  a.sw = sw;
  a.offsets = offsets;
  a.Y = Y;
  a.ldy = ldy;
  a.T = (int)T;
  a.N = (int)N;
  a.K = (int)K;
  a.E = (int)E;
  a.kb = (int)plan::cdiv(K, kBlockK);
  a.static_weights = static_weights;
  const Launch l{x, w, a, plan::Product(T, E, N, K, offsets != nullptr, sms), stream};
  const plan::Choice c = l.p.choose();
  switch (c.bn) {
    case 16: return l.run<plan::S16>(c.splits);
    case 32: return l.run<plan::S32>(c.splits);
    case 64: return l.run<plan::S64>(c.splits);
    case 128: return l.run<plan::S128>(c.splits);
    case 256: return l.run<plan::L256>(c.splits);
  }
  return cudaErrorInvalidConfiguration;
}

cudaError_t read_and_clear_fp8_errors(unsigned int* timeouts, unsigned int* bad_offsets) {
  const unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(timeouts, g_fp8_wait_timeouts, sizeof(zero));
  if (e == cudaSuccess && *timeouts) e = cudaMemcpyToSymbol(g_fp8_wait_timeouts, &zero, sizeof(zero));
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(bad_offsets, g_fp8_bad_offsets, sizeof(zero));
  if (e == cudaSuccess && *bad_offsets) e = cudaMemcpyToSymbol(g_fp8_bad_offsets, &zero, sizeof(zero));
  return e;
}

}  // namespace nvfp4
