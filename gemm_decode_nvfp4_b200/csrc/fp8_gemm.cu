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
// Roles per CTA: PW promotion warps, one producer warp (lane 0 issues the TMA
// tiles; all lanes copy the block's scales with cp.async into a ring of their
// own), one MMA warp.  Persistent over tiles; the stage ring runs on across
// tiles.  With few tiles a cluster of `splits` CTAs shares a tile's blocks of k
// and adds the partial sums in rank order through distributed shared memory.
// Every wait is bounded.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "nvfp4_device.cuh"
#include "nvfp4_kernels.h"
#include "sm100_ptx.cuh"
#include "tc_host.h"

namespace nvfp4 {

// CTAs whose pipeline wait ran past its limit, and group ends out of order or range.
__device__ unsigned int g_fp8_wait_timeouts = 0;
__device__ unsigned int g_fp8_bad_offsets = 0;

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr int kRows = 128;        // MMA M
constexpr int kBlockK = 128;      // k per stage, one scale block, one swizzled row
constexpr int kMaxStages = 8;
constexpr int kMaxBufs = 4;
constexpr int kScaleSlots = 12;   // >= stages + accumulator buffers
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

struct Bars {
  uint64_t full[kMaxStages];
  uint64_t empty[kMaxStages];
  uint64_t sfull[kScaleSlots];
  uint64_t acc_full[kMaxBufs];
  uint64_t acc_empty[kMaxBufs];
  uint64_t mma_done;
  uint32_t tmem_addr;
  volatile int err;
};

template <bool SWAP_, int BN_, int PW_>
struct Cfg {
  static constexpr bool SWAP = SWAP_;
  static constexpr int BN = BN_, PW = PW_;
  static constexpr int NBUF = 512 / BN < kMaxBufs ? 512 / BN : kMaxBufs;
  static constexpr uint32_t TMEM = NBUF * BN < 32 ? 32 : NBUF * BN;
  static constexpr int COLS = BN / (PW / 4);  // accumulator columns of one thread
  static constexpr int TOK = SWAP ? BN : kRows, WROWS = SWAP ? kRows : BN;
  static constexpr int SW = WROWS / 128;      // weight scales per block
  static constexpr int SLOT = TOK + 4;        // floats of a scale slot: token scales, then weight scales
  static constexpr int STAGE = (kRows + BN) * kBlockK;
  static constexpr int THREADS = (PW + 2) * 32;
  static constexpr int CTAS = BN <= 64 ? 2 : 1;  // per SM
  static constexpr int EPI = SWAP ? 0 : PW * 2048;
  static constexpr int FIXED = EPI + kScaleSlots * SLOT * 4 + (int)sizeof(Bars) + 1024;
};

__device__ __forceinline__ bool wait_or_fail(uint64_t* bar, uint32_t parity, Bars* bars) {
  if (bars->err) return false;
  if (ptx::mbar_wait(bar, parity, kWaitLimitNs)) return true;
  if (!bars->err) {
    bars->err = 1;
    atomicAdd(&g_fp8_wait_timeouts, 1u);
  }
  return false;
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
__device__ __forceinline__ void ld_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// a += t * s on pairs of fp32
__device__ __forceinline__ void fma2(float2& a, uint32_t t0, uint32_t t1, float2 s) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%0, %1};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "+f"(a.x), "+f"(a.y)
      : "r"(t0), "r"(t1), "f"(s.x), "f"(s.y));
}

// One output tile: its expert's weight rows from w0, tokens [m0, mend).
struct Tile {
  int e, m0, mend, n0;
};

// Tile t of the order: experts in turn; within one, groups of kGroupTiles token
// tiles; within a group, weight tile by weight tile.  Neighbouring CTAs so share
// weight tiles, and a group's tokens stay in L2.  pre (grouped): token tiles
// before each expert; off: its first row (E + 1 each).
template <int TOK, int WROWS>
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
    mt = (a.T + TOK - 1) / TOK;
  }
  const int group = t / (kGroupTiles * a.nt);
  const int in = min(kGroupTiles, mt - group * kGroupTiles);
  t -= group * kGroupTiles * a.nt;
  const int n = t / in;
  r.e = lo;
  r.m0 = first + (group * kGroupTiles + t - n * in) * TOK;
  r.mend = mend;
  r.n0 = n * WROWS;
  return r;
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
  Bars* bars = reinterpret_cast<Bars*>(scales + kScaleSlots * C::SLOT);
  int* pre = reinterpret_cast<int*>(bars + 1);  // grouped: [E + 1] token tiles before
  int* off = pre + a.E + 1;                     // then [E + 1] first rows, [E + 1] row ends

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = a.splits > 1 ? (int)ptx::cluster_ctarank() : 0;
  const int kb0 = (int)((int64_t)a.kb * rank / a.splits), kb1 = (int)((int64_t)a.kb * (rank + 1) / a.splits);
  const int S = a.stages;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(&bars->full[i], 1);
      ptx::mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < kScaleSlots; ++i) ptx::mbar_init(&bars->sfull[i], 32);
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
      if (lane == 0) pre[0] = 0;
      if (bad && blockIdx.x == 0) atomicAdd(&g_fp8_bad_offsets, 1u);
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

  if (warp == PW) {
    // ---------------------------------------------------------------- producer
    int st = 0, ph = 0, slot = 0;  // ph: parity that `empty` completes next
    bool fresh = true;             // the ring's first pass: every stage is free
    bool waited = a.offsets != nullptr;
    int issued = 0;
    for (int t = first; t < tiles; t += step) {
      const Tile w = tile_of<C::TOK, C::WROWS>(t, a, pre, off);
      const int wrow = w.e * a.N + w.n0;
      const int wsrow = w.e * ((a.N + 127) / 128) + w.n0 / 128;
      auto issue_w = [&](int s, int kb) {
        ptx::tma_load_2d(smem + s * C::STAGE + (SWAP ? 0 : kRows * kBlockK), &tmap_w, &bars->full[s], kb * kBlockK,
                         wrow);
      };
      int ahead = 0;  // stages whose weights are already on the way
      if (!waited) {
        ahead = a.static_weights ? min(S, kb1 - kb0) : 0;
        if (lane == 0)
          for (int i = 0; i < ahead; ++i) {
            ptx::mbar_arrive_expect_tx(&bars->full[i], C::STAGE);
            issue_w(i, kb0 + i);
          }
        asm volatile("griddepcontrol.wait;" ::: "memory");
        waited = true;
      }
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!fresh && !__all_sync(0xFFFFFFFFu, wait_or_fail(&bars->empty[st], ph, bars))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          if (kb - kb0 >= ahead) {
            ptx::mbar_arrive_expect_tx(&bars->full[st], C::STAGE);
            issue_w(st, kb);
          }
          ptx::tma_load_2d(smem + st * C::STAGE + (SWAP ? kRows * kBlockK : 0), &tmap_x, &bars->full[st],
                           kb * kBlockK, w.m0);
        }
        // A slot is written again only after its block was promoted: this stage
        // is free, so the MMAs of block g - stages are done, which could start
        // once block g - stages - NBUF was promoted; there are more slots than that.
        float* d = scales + slot * C::SLOT;
#pragma unroll
        for (int i = 0; i < (C::TOK + 31) / 32; ++i) {
          const int j = lane + 32 * i, m = w.m0 + j;
          if (C::TOK % 32 == 0 || j < C::TOK)
            cp_async4(d + j, a.sx + (int64_t)min(m, a.T - 1) * a.kb + kb, m < a.T);
        }
        if (lane < C::SW)
          cp_async4(d + C::TOK + lane,
                    a.sw + (int64_t)min(wsrow + lane, a.E * ((a.N + 127) / 128) - 1) * a.kb + kb,
                    w.n0 + 128 * lane < a.N);
        cp_async_arrive(&bars->sfull[slot]);
        ++issued;
        if (++slot == kScaleSlots) slot = 0;
        if (++st == S) {
          st = 0;
          if (fresh) fresh = false; else ph ^= 1;
        }
      }
      if (!ok) break;
    }
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (bars->err && lane == 0) {
      // let the tiles already asked for land before the CTA exits
      for (int g = max(issued - S, 0); g < issued; ++g) ptx::mbar_wait(&bars->full[g % S], (g / S) & 1, kWaitLimitNs);
    }
  } else if (warp == PW + 1) {
    // -------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      int st = 0, ph = 0, buf = 0, bph = 1;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        for (int kb = kb0; kb < kb1; ++kb) {
          // (parity 1 passes at once on a fresh barrier: every buffer starts free)
          if (!wait_or_fail(&bars->acc_empty[buf], bph, bars) || !wait_or_fail(&bars->full[st], ph, bars)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t a0 = ptx::smem_u32(smem + st * C::STAGE), b0 = a0 + kRows * kBlockK;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f8(tmem + buf * BN, ptx::sw128_kmajor_desc(a0 + 32 * kk), ptx::sw128_kmajor_desc(b0 + 32 * kk), kIdesc,
                   kk != 0);
          ptx::mma_commit(&bars->empty[st]);
          ptx::mma_commit(&bars->acc_full[buf]);
          if (++st == S) st = 0, ph ^= 1;
          if (++buf == NBUF) buf = 0, bph ^= 1;
        }
      }
      // arrives when every MMA above is done, so that tensor memory is never
      // freed under one (also on the error path)
      ptx::mma_commit(&bars->mma_done);
      ptx::mbar_wait(&bars->mma_done, 0, kWaitLimitNs);
    }
  } else {
    // --------------------------------------------------------------- promotion
    const int quarter = warp & 3, part = warp >> 2;
    const int row = 32 * quarter + lane, col0 = part * COLS;
    const uint32_t lane_addr = tmem + ((uint32_t)(32 * quarter) << 16) + col0;
    int buf = 0, bph = 0, slot = 0, sph = 0;
    bool ok = true;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // Y
    for (int t = first; t < tiles && ok; t += step) {
      float2 acc[COLS / 2];
#pragma unroll
      for (int j = 0; j < COLS / 2; ++j) acc[j] = make_float2(0.0f, 0.0f);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!__all_sync(0xFFFFFFFFu,
                        wait_or_fail(&bars->sfull[slot], sph, bars) && wait_or_fail(&bars->acc_full[buf], bph, bars))) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const float* sc = scales + slot * C::SLOT;
        const float sw = sc[C::TOK + (SWAP ? 0 : col0 / 128)];
        const float srow = SWAP ? 0.0f : sc[row] * sw;
        uint32_t r[2][16];
        ptx::tmem_ld_16cols(lane_addr + buf * BN, r[0]);
#pragma unroll
        for (int c = 0; c < COLS / 16; ++c) {
          ld_wait16(r[c & 1]);
          if (c + 1 < COLS / 16) ptx::tmem_ld_16cols(lane_addr + buf * BN + 16 * (c + 1), r[(c + 1) & 1]);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float2 s;
            if (SWAP) {
              s = *reinterpret_cast<const float2*>(sc + col0 + 16 * c + 2 * j);
              s.x *= sw;
              s.y *= sw;
            } else {
              s = make_float2(srow, srow);
            }
            fma2(acc[8 * c + j], r[c & 1][2 * j], r[c & 1][2 * j + 1], s);
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&bars->acc_empty[buf]);
        if (++buf == NBUF) buf = 0, bph ^= 1;
        if (++slot == kScaleSlots) slot = 0, sph ^= 1;
      }
      if (!ok) break;
      const Tile w = tile_of<C::TOK, C::WROWS>(t, a, pre, off);
      if constexpr (SWAP) {
        if (a.splits > 1) {
          // partial sums to the (now idle) stage memory, [token][weight row]
          float* part_sum = reinterpret_cast<float*>(smem);
#pragma unroll
          for (int j = 0; j < COLS / 2; ++j) {
            part_sum[(col0 + 2 * j) * kRows + row] = acc[j].x;
            part_sum[(col0 + 2 * j + 1) * kRows + row] = acc[j].y;
          }
        } else if (w.n0 + row < a.N) {
#pragma unroll
          for (int j = 0; j < COLS; ++j) {
            const int m = w.m0 + col0 + j;
            if (m < w.mend) {
              const __nv_bfloat16 o = __float2bfloat16_rn(j & 1 ? acc[j / 2].y : acc[j / 2].x);
              a.Y[(int64_t)m * a.ldy + w.n0 + row] = *reinterpret_cast<const uint16_t*>(&o);
            }
          }
        }
      } else {
        // through shared memory, 32 columns (64 bytes) of the warp's 32 tokens at
        // a time, so that four lanes store one token's 64 bytes; the 16-byte
        // pieces are rotated by the row against bank conflicts
        uint8_t* stg = epi + warp * 2048;
        const bool vec = ((reinterpret_cast<uintptr_t>(a.Y) & 15u) == 0) && (a.ldy & 7) == 0;
#pragma unroll
        for (int c = 0; c < COLS / 32; ++c) {
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 h = __float22bfloat162_rn(acc[16 * c + 4 * p + i]);
              o[i] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(stg + lane * 64 + ((p + (lane >> 1)) & 3) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int rr = 8 * i + (lane >> 2), p = lane & 3;
            const uint4 v = *reinterpret_cast<const uint4*>(stg + rr * 64 + ((p + (rr >> 1)) & 3) * 16);
            const int m = w.m0 + 32 * quarter + rr, n = w.n0 + col0 + 32 * c + 8 * p;
            if (m < w.mend && n < a.N) {
              uint16_t* dst = a.Y + (int64_t)m * a.ldy + n;
              if (vec && n + 8 <= a.N) {
                *reinterpret_cast<uint4*>(dst) = v;
              } else {
                const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  if (n + k < a.N) dst[k] = (uint16_t)(w4[k >> 1] >> (16 * (k & 1)));
              }
            }
          }
          __syncwarp();
        }
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
        const int live = min(BN, w.mend - w.m0) * kRows;
        for (int i = threadIdx.x + rank * C::THREADS; i < live; i += C::THREADS * a.splits) {
          float v = 0.0f;
          for (int r = 0; r < a.splits; ++r) v += ptx::ld_cluster_f32(part_sum + i, r);
          const int m = w.m0 + i / kRows, n = w.n0 + i % kRows;
          if (n < a.N) {
            const __nv_bfloat16 o = __float2bfloat16_rn(v);
            a.Y[(int64_t)m * a.ldy + n] = *reinterpret_cast<const uint16_t*>(&o);
          }
        }
      }
      ptx::cluster_sync();
    }
  }
}

constexpr int kSmemMax = 232448;  // dynamic shared memory of a CTA that has the SM to itself
constexpr int kSmemHalf = 115712; // of one that shares it with another

template <class C>
cudaError_t run(const uint8_t* x, const uint8_t* w, Args a, int sms, int64_t tiles, cudaStream_t stream) {
  static tc::SmemOptIn opt;
  const int table = a.offsets ? 3 * (a.E + 1) * 4 : 0;
  const int room = (C::CTAS == 2 ? kSmemHalf : kSmemMax) - C::FIXED - table;
  a.stages = room / C::STAGE < kMaxStages ? room / C::STAGE : kMaxStages;
  if (a.stages < 2) return cudaErrorInvalidConfiguration;
  static_assert(kMaxStages + C::NBUF <= kScaleSlots, "scale slots outlive stages and accumulators");
  CUtensorMap mw, mx;
  if (!tc::make_tmap_2d(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, (uint64_t)a.K, (uint64_t)a.E * a.N, (uint64_t)a.K,
                        kBlockK, C::WROWS, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !tc::make_tmap_2d(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, (uint64_t)a.K, (uint64_t)a.T, (uint64_t)a.K, kBlockK,
                        C::TOK, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const int smem = C::FIXED + table + a.stages * C::STAGE;
  const void* fn = (const void*)fp8_gemm_kernel<C>;
  cudaError_t e = opt.ensure(fn, smem);
  if (e != cudaSuccess) return e;
  const int64_t slots = (int64_t)sms * C::CTAS;
  const int64_t grid = a.splits > 1 ? tiles * a.splits : (tiles < slots ? tiles : slots);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)a.splits, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 2 : 1;
  void* args[] = {&mw, &mx, &a};
  return cudaLaunchKernelExC(&cfg, fn, args);
}

int64_t cdiv(int64_t x, int64_t y) { return (x + y - 1) / y; }

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
  a.kb = (int)cdiv(K, kBlockK);
  a.splits = 1;
  a.static_weights = static_weights;
  const int64_t rows = offsets ? cdiv(T, E) : T;  // per expert, on average
  if (rows > 128 && cdiv(rows, 128) * cdiv(N, 256) * E >= 120) {
    a.nt = (int)cdiv(N, 256);
    const int64_t most = a.nt * (offsets ? T / 128 + E : cdiv(T, 128));
    return run<Cfg<false, 256, 8>>(x, w, a, sms, most, stream);
  }
  const int bn = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
  const int per_sm = bn <= 64 ? 2 : 1;
  a.nt = (int)cdiv(N, 128);
  const int64_t tiles = a.nt * (offsets ? T / bn + E : cdiv(T, bn));
  if (!offsets) {
    // fewest waves times blocks of k per CTA
    int64_t best = 0;
    for (int c = 1; c <= 8 && c <= a.kb; ++c) {
      const int64_t cost = cdiv(tiles * c, (int64_t)sms * per_sm) * (cdiv(a.kb, c) + 2) + (c > 1 ? 2 : 0);
      if (c == 1 || cost < best) {
        best = cost;
        a.splits = c;
      }
    }
  }
  switch (bn) {
    case 16: return run<Cfg<true, 16, 4>>(x, w, a, sms, tiles, stream);
    case 32: return run<Cfg<true, 32, 4>>(x, w, a, sms, tiles, stream);
    case 64: return run<Cfg<true, 64, 4>>(x, w, a, sms, tiles, stream);
    default: return run<Cfg<true, 128, 8>>(x, w, a, sms, tiles, stream);
  }
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
