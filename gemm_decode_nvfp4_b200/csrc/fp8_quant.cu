// fp8_quant.cu -- the kernels that write E4M3 values with one fp32 scale per
// 128: the RMS norm with the residual's addition, the activation quantizer
// (plain, or of silu(gate) * up) and the weight quantizer (include/fp8.h).
//
// One rule everywhere, over a block of 128 columns of one row (activations) or
// of 128 rows (weights):
//   s = max(max|v| / 448, 2^-126),  q = E4M3_rne_satfinite(v * (1 / s))
// with IEEE fp32 divisions.  The lower limit keeps 1 / s finite.
// fmaxf drops NaN, so a NaN element stays a NaN code of its own and leaves the
// rest of its block alone; an infinity makes its block's scale infinite.
//
// All three stream HBM once (norm rows of more than 32768 columns twice).  A thread
// owns 16-byte vectors of 8 columns, so a block of 128 columns is neighbouring lanes:
// 8 of two vectors in the activation quantizer, 16 of one in the norm of few rows, 8 or
// 4 of two or four in that of many; K is a multiple of 16, so no lane straddles the
// end of a row.
#include "fp8_drain.h"
#include "fp8_plan.h"
#include "nvfp4_device.cuh"
#include "nvfp4_kernels.h"
#include "sm100_ptx.cuh"
#include "tc_host.h"

namespace nvfp4 {

// CTAs of the RMS norm whose wait for a row ran past its limit.
__device__ unsigned int g_fp8_norm_timeouts = 0;

namespace {

constexpr float kScaleMin = 1.17549435e-38f;  // 2^-126
constexpr uint64_t kNormWaitNs = 2000000000ull;

// 16-byte load of what is read once, past L1.  Not a read-only load (ld.global.nc,
// __ldg): those are for data that nothing writes while the kernel runs, and these
// kernels' CTAs start while the kernels before them may still be writing what they
// read after their wait.
__device__ __forceinline__ uint4 ld_once_v4(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo_to_float(w[i]);
    f[2 * i + 1] = bf16hi_to_float(w[i]);
  }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

__device__ __forceinline__ float absmax(const float (&f)[8]) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(f[i]));
  return a;
}

// maximum over the 16 lanes that share a block of 128 columns
__device__ __forceinline__ float max16(float a) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  return a;
}

__device__ __forceinline__ float scale_of(float amax) { return fmaxf(__fdiv_rn(amax, 448.0f), kScaleMin); }

// (lo, hi) -> two E4M3 bytes, lo in the low one
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t out;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(out) : "f"(hi), "f"(lo));
  return out;
}

__device__ __forceinline__ uint2 quantize8(const float (&f)[8], float r) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = e4m3x2(__fmul_rn(f[2 * i], r), __fmul_rn(f[2 * i + 1], r));
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

struct NormArgs {
  const uint16_t* x;
  const uint16_t* w;
  const uint16_t* res;  // null: none
  uint16_t* res_out;
  uint16_t* y;  // null: none
  uint8_t* q;   // null: none
  float* s;
  int64_t ldx, ldr, ldro, ldy;
  int64_t M;
  int K, kb;
  float eps;
};

// x (+ residual) of one vector: what the norm is taken of.  The sum is used as
// its BF16 value, the one that the residual stream carries on.
__device__ __forceinline__ void load_h(const NormArgs& a, int64_t row, int c, float (&f)[8]) {
  unpack8(*reinterpret_cast<const uint4*>(a.x + row * a.ldx + c), f);
  if (a.res) {
    float r[8];
    unpack8(*reinterpret_cast<const uint4*>(a.res + row * a.ldr + c), r);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __fadd_rn(f[i], r[i]);
    unpack8(pack8(f), f);
  }
}

__device__ __forceinline__ void norm_out(const NormArgs& a, int64_t row, int c, bool in, float (&f)[8], uint4 wv,
                                         float rstd) {
  float w[8];
  unpack8(wv, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(__fmul_rn(f[i], rstd), w[i]);
  if (a.y && in) *reinterpret_cast<uint4*>(a.y + row * a.ldy + c) = pack8(f);
  if (a.q) {
    const float s = scale_of(max16(absmax(f)));
    if (in) {
      *reinterpret_cast<uint2*>(a.q + row * a.K + c) = quantize8(f, __frcp_rn(s));
      if ((c & 127) == 0) a.s[row * a.kb + (c >> 7)] = s;
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// RMS norm: `threads` (a multiple of 32) threads per row, VPT vectors each, the
// row kept in registers between the sum of squares and the output.  threads
// == 32 takes 4 rows per CTA and needs no barrier.
template <int VPT>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormArgs a, int threads) {
  __shared__ float red[32];
  const int t = threadIdx.x % threads;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x / threads) + threadIdx.x / threads;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= a.M) return;  // whole warps: one row's threads stay together
  float f[VPT][8];
  uint4 wv[VPT];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t + i * threads) * 8;
    if (c < a.K) {
      load_h(a, row, c, f[i]);
      wv[i] = *reinterpret_cast<const uint4*>(a.w + c);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] = 0.0f;
      wv[i] = make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(f[i][j], f[i][j], sum);
  if (a.res_out) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t + i * threads) * 8;
      if (c < a.K) *reinterpret_cast<uint4*>(a.res_out + row * a.ldro + c) = pack8(f[i]);
    }
  }
  sum = warp_sum(sum);
  if (threads > 32) {
    if ((t & 31) == 0) red[t >> 5] = sum;
    __syncthreads();
    sum = warp_sum((t & 31) < (threads >> 5) ? red[t & 31] : 0.0f);
  }
  const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)a.K), a.eps));
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t + i * threads) * 8;
    norm_out(a, row, c, c < a.K, f[i], wv[i], rstd);
  }
}

// Many rows: each CTA takes rows blockIdx.x, + gridDim.x, ... and bulk copies
// bring them into a ring of row slots (x, then the residual) ahead of time, so
// that reads go on while a row is summed, scaled and stored.  A thread has VPT
// neighbouring vectors, so a block of 128 columns is 16 / VPT lanes.  8192 rows of
// 5120 with a residual (295 MB): 49.6 us, 92% of the copy rate; a CTA per row, its
// loads waiting for its place on the SM, 73.6 us.  Without the residual the
// arithmetic per byte bounds it (8192 x 5120: 36.4 us, 54%).
template <int VPT>
__global__ void __launch_bounds__(1024) rmsnorm_rows_kernel(const NormArgs a, int slots) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t full[plan::kNormSlots];
  __shared__ float red[2][32];
  __shared__ volatile int err;
  __shared__ int left_out;  // rows not fetched since a wait gave up (thread 0's)
  const int t = threadIdx.x, threads = blockDim.x;
  const uint32_t row_bytes = (uint32_t)a.K * 2, slot_bytes = a.res ? 2 * row_bytes : row_bytes;
  if (t == 0) {
    for (int i = 0; i < slots; ++i) ptx::mbar_init(&full[i], 1);
    err = 0;
    left_out = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  auto fetch = [&](int64_t row, int slot) {
    uint8_t* d = smem + (size_t)slot * slot_bytes;
    ptx::mbar_arrive_expect_tx(&full[slot], slot_bytes);
    ptx::bulk_load(d, a.x + row * a.ldx, row_bytes, &full[slot]);
    if (a.res) ptx::bulk_load(d + row_bytes, a.res + row * a.ldr, row_bytes, &full[slot]);
  };
  if (t == 0)
    for (int i = 0; i < slots; ++i) {
      const int64_t row = blockIdx.x + (int64_t)i * gridDim.x;
      if (row < a.M) fetch(row, i);
    }
  uint4 wv[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (t * VPT + i) * 8;
    wv[i] = c < a.K ? *reinterpret_cast<const uint4*>(a.w + c) : make_uint4(0, 0, 0, 0);
  }
  int slot = 0, ph = 0, odd = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    // (after a wait that gave up, the CTA goes through its rows without waiting or
    // fetching, so that all its threads meet at the same barriers)
    bool landed = !err;
    if (landed && !ptx::mbar_wait(&full[slot], ph, kNormWaitNs)) {
      landed = false;
      err = 1;
      if (t == 0) atomicAdd(&g_fp8_norm_timeouts, 1u);
    }
    const uint8_t* d = smem + (size_t)slot * slot_bytes;
    float f[VPT][8], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (t * VPT + i) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] = 0.0f;
      if (c < a.K) {
        unpack8(*reinterpret_cast<const uint4*>(d + c * 2), f[i]);
        if (a.res) {
          float r[8];
          unpack8(*reinterpret_cast<const uint4*>(d + row_bytes + c * 2), r);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[i][j] = __fadd_rn(f[i][j], r[j]);
          const uint4 h = pack8(f[i]);
          *reinterpret_cast<uint4*>(a.res_out + row * a.ldro + c) = h;
          unpack8(h, f[i]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(f[i][j], f[i][j], sum);
    }
    sum = warp_sum(sum);
    if ((t & 31) == 0) red[odd][t >> 5] = sum;
    __syncthreads();  // (the next row uses the other half of red)
    const int64_t next = row + (int64_t)slots * gridDim.x;
    if (t == 0 && next < a.M) {  // every thread has read its part of the slot
      if (landed) {
        ptx::fence_proxy_async_smem();
        fetch(next, slot);
      } else {
        ++left_out;
      }
    }
    sum = warp_sum((t & 31) < (threads >> 5) ? red[odd][t & 31] : 0.0f);
    const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)a.K), a.eps));
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float w[8];
      unpack8(wv[i], w);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[i][j] = __fmul_rn(__fmul_rn(f[i][j], rstd), w[j]);
      m = fmaxf(m, absmax(f[i]));
    }
    if (a.q) {  // the block's other columns are with the next 16 / VPT - 1 lanes
#pragma unroll
      for (int o = 8 / VPT; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    }
    const float s = scale_of(m), r = __frcp_rn(s);
    const int c0 = t * VPT * 8;
    if (c0 < a.K) {
#pragma unroll
      for (int i = 0; i < VPT; i += 2) {  // K is a multiple of 16: pairs of vectors are in or out together
        const int c = c0 + i * 8;
        if (c < a.K) {
          if (a.y) {
            *reinterpret_cast<uint4*>(a.y + row * a.ldy + c) = pack8(f[i]);
            *reinterpret_cast<uint4*>(a.y + row * a.ldy + c + 8) = pack8(f[i + 1]);
          }
          if (a.q) {
            const uint2 lo = quantize8(f[i], r), hi = quantize8(f[i + 1], r);
            *reinterpret_cast<uint4*>(a.q + row * a.K + c) = make_uint4(lo.x, lo.y, hi.x, hi.y);
          }
        }
      }
      if (a.q && (c0 & 127) == 0) a.s[row * a.kb + (c0 >> 7)] = s;
    }
    odd ^= 1;
    if (++slot == slots) slot = 0, ph ^= 1;
  }
  if (t == 0 && err) {
    const int rows = (int)((a.M - blockIdx.x + gridDim.x - 1) / gridDim.x);
    drain_ring(rows - left_out, slots, [&](int i, int parity) { ptx::mbar_wait(&full[i], parity, kNormWaitNs); });
  }
}

// Rows too long for registers: 1024 threads walk the row twice, the second time
// (out of L2) over residual_out where there is one.
__global__ void __launch_bounds__(1024) rmsnorm_long_kernel(const NormArgs a) {
  __shared__ float red[32];
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float sum = 0.0f;
  for (int c = t * 8; c < a.K; c += 8192) {
    float f[8];
    load_h(a, row, c, f);
    if (a.res_out) *reinterpret_cast<uint4*>(a.res_out + row * a.ldro + c) = pack8(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(f[j], f[j], sum);
  }
  sum = warp_sum(sum);
  if ((t & 31) == 0) red[t >> 5] = sum;
  __syncthreads();
  sum = warp_sum(red[t & 31]);
  const float rstd = __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)a.K), a.eps));
  NormArgs b = a;
  if (a.res_out) {  // written above by this same thread
    b.x = a.res_out;
    b.ldx = a.ldro;
    b.res = nullptr;
  }
  for (int c0 = 0; c0 < a.K; c0 += 8192) {  // whole warps: the block maxima shuffle
    const int c = c0 + t * 8;
    const bool in = c < a.K;
    float f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    uint4 wv = make_uint4(0, 0, 0, 0);
    if (in) {
      load_h(b, row, c, f);
      wv = *reinterpret_cast<const uint4*>(a.w + c);
    }
    norm_out(a, row, c, in, f, wv, rstd);
  }
}

struct QuantArgs {
  const uint16_t* x;
  uint8_t* q;
  float* s;
  int64_t ldx;
  uint32_t blocks;  // M * kb
  int K, kb;
};

// silu(g) * u in fp32: silu(g) = g / (1 + exp(-g)) with the divisor times 2^-8,
//   g * (2^-8 / (2^-8 + 2^(-g log2(e) - 8))),
// so that it stays within the approximate reciprocal's range (2^126) down to g = -92,
// as far as silu is a normal number.  silu is off by less than 2^-17 of itself at
// g = -91 (the exponent's rounding 2^-18, log2(e)'s 2^-19, the subnormal quotient's
// 2^-18.7, the approximations' 2^-22 and 2^-23), where the E4M3 code is rounded to 2^-4
// and the scale follows one value.  1024 x 17408: 16.5 us, as with __expf and
// __fdividef, which give zero below -87.3; with t = exp(-|g| / 2) taken twice, 17.5 to
// 19.3; with expf and a true division (8 columns per lane, __expf then 20.2), 28.8.
__device__ __forceinline__ float silu_mul(float g, float u) {
  constexpr float kLog2E = 1.44269504f, k = 0.00390625f;
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(g, -kLog2E, -8.0f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + k));
  return __fmul_rn(__fmul_rn(g, __fmul_rn(r, k)), u);
}

// Activation quantizer: 8 lanes of 16 columns per block of 128, two (gated: four)
// 16-byte loads of a lane in flight at six CTAs per SM.  4096 x 5120: 12.1 us, 81%
// of the copy rate; gated 1024 x 17408: 16.5 us, 84%.  (16 lanes of 8 columns at
// eight CTAs: 14.6 and 20.2 us; two or four blocks of a lane in flight with as many
// fewer warps: 14.9 to 18.9 us.)
template <bool GATED>
__global__ void __launch_bounds__(256, 6) quantize_rows_kernel(const QuantArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane8 = threadIdx.x & 7;
  const uint64_t stride = (uint64_t)gridDim.x * 32;
  // (whole warps stay in the loop: all four blocks of a warp take part in the shuffles)
  for (uint64_t b = (uint64_t)blockIdx.x * 32 + (threadIdx.x >> 5) * 4; b < a.blocks; b += stride) {
    const uint32_t blk = (uint32_t)b + ((threadIdx.x >> 3) & 3);
    const uint32_t row = blk / (uint32_t)a.kb;
    const int c = (int)(blk - row * (uint32_t)a.kb) * 128 + lane8 * 16;
    const bool in = blk < a.blocks && c < a.K;  // K is a multiple of 16: all 16 columns or none
    float f[2][8] = {};
    if (in) {
      const uint16_t* p = a.x + (int64_t)row * a.ldx + c;
      const uint4 v0 = ld_once_v4(p), v1 = ld_once_v4(p + 8);
      unpack8(v0, f[0]);
      unpack8(v1, f[1]);
      if (GATED) {
        const uint4 u0 = ld_once_v4(p + a.K), u1 = ld_once_v4(p + a.K + 8);
        float uf[8];
        unpack8(u0, uf);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[0][i] = silu_mul(f[0][i], uf[i]);
        unpack8(u1, uf);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[1][i] = silu_mul(f[1][i], uf[i]);
      }
    }
    float m = fmaxf(absmax(f[0]), absmax(f[1]));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float s = scale_of(m);
    if (in) {
      const float r = __frcp_rn(s);
      const uint2 lo = quantize8(f[0], r), hi = quantize8(f[1], r);
      *reinterpret_cast<uint4*>(a.q + (int64_t)row * a.K + c) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      if (lane8 == 0) a.s[blk] = s;
    }
  }
}

// Weight quantizer: one CTA of 256 threads per 128 x 128 block, held in
// registers between the maximum and the codes.
__global__ void __launch_bounds__(256, 4) quantize_blocks_kernel(const uint16_t* w, int64_t ldw, int64_t N,
                                                              int K, int kb, uint8_t* __restrict__ q,
                                                              float* __restrict__ s) {
  __shared__ float red[8];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t nb = blockIdx.x / kb;
  const int b = (int)(blockIdx.x - nb * kb);
  const int c = b * 128 + (threadIdx.x & 15) * 8;
  const int64_t row0 = nb * 128 + (threadIdx.x >> 4);
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = row0 + 16 * i;
    v[i] = n < N && c < K ? ld_once_v4(w + n * ldw + c) : make_uint4(0, 0, 0, 0);
  }
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float f[8];
    unpack8(v[i], f);
    m = fmaxf(m, absmax(f));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  m = red[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) m = fmaxf(m, red[i]);
  const float sc = scale_of(m), r = __frcp_rn(sc);
  if (threadIdx.x == 0) s[blockIdx.x] = sc;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t n = row0 + 16 * i;
    if (n < N && c < K) {
      float f[8];
      unpack8(v[i], f);
      *reinterpret_cast<uint2*>(q + n * K + c) = quantize8(f, r);
    }
  }
}

// Warps of a kernel that an SM's 65536 registers hold (a thread has them in eights).
int warps_held(const void* fn) {
  cudaFuncAttributes attr;
  if (cudaFuncGetAttributes(&attr, fn) != cudaSuccess) return 32;  // 64 a thread, the launch bound's most
  return 65536 / 32 / ((attr.numRegs + 7) / 8 * 8);
}

}  // namespace

cudaError_t launch_fp8_rmsnorm(const uint16_t* x, int64_t ldx, const uint16_t* weight, const uint16_t* residual,
                               int64_t ldr, uint16_t* residual_out, int64_t ldro, uint16_t* y, int64_t ldy, uint8_t* q,
                               float* s, int64_t M, int64_t K, float eps, int sms, cudaStream_t stream) {
  NormArgs a{x, weight, residual, residual_out, y, q, s, ldx, ldr, ldro, ldy, M, (int)K, (int)((K + 127) / 128), eps};
  const int64_t vecs = K / 8;
  if (vecs > 1024 * 4) {
    void* args[] = {&a};
    return tc::launch_pdl((const void*)rmsnorm_long_kernel, dim3((unsigned)M), dim3(1024), 0, stream, args);
  }
  // one warp per row while four vectors a lane hold it, else up to four vectors a thread
  int vpt = vecs <= 32 ? 1 : vecs <= 64 ? 2 : 4, threads = 32;
  if (vecs > 128) {
    vpt = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : 4;
    threads = (int)(((vecs + vpt - 1) / vpt + 31) / 32 * 32);
  }
  if (threads > 32 && M > 2 * (int64_t)sms) {
    static const int warps[2] = {warps_held((const void*)rmsnorm_rows_kernel<2>),
                                 warps_held((const void*)rmsnorm_rows_kernel<4>)};
    const plan::NormRows p = plan::norm_rows(K, residual != nullptr, warps);
    if (p.per_sm > 0) {
      static tc::SmemOptIn opt[2];
      const void* fn = p.wide == 2 ? (const void*)rmsnorm_rows_kernel<2> : (const void*)rmsnorm_rows_kernel<4>;
      const int smem = p.slots * (int)K * (residual ? 4 : 2);
      cudaError_t e = opt[p.wide == 4].ensure(fn, smem);
      if (e != cudaSuccess) return e;
      const int64_t grid = (int64_t)sms * p.per_sm;
      int slots = p.slots;
      void* args[] = {&a, &slots};
      return tc::launch_pdl(fn, dim3((unsigned)(M < grid ? M : grid)), dim3(p.threads), smem, stream, args);
    }
  }
  const int rows = threads == 32 ? 4 : 1;
  void* args[] = {&a, &threads};
  const void* fn = vpt == 1 ? (const void*)rmsnorm_kernel<1> : vpt == 2 ? (const void*)rmsnorm_kernel<2>
                                                                       : (const void*)rmsnorm_kernel<4>;
  return tc::launch_pdl(fn, dim3((unsigned)((M + rows - 1) / rows)), dim3(threads * rows), 0, stream, args);
}

cudaError_t launch_fp8_quantize(const uint16_t* x, int64_t ldx, int64_t M, int64_t K, bool gated, uint8_t* q, float* s,
                                int sms, cudaStream_t stream) {
  const int64_t kb = (K + 127) / 128;
  QuantArgs a{x, q, s, ldx, (uint32_t)(M * kb), (int)K, (int)kb};
  const int64_t want = (M * kb + 31) / 32, most = (int64_t)sms * 6;
  void* args[] = {&a};
  return tc::launch_pdl(gated ? (const void*)quantize_rows_kernel<true> : (const void*)quantize_rows_kernel<false>,
                        dim3((unsigned)(want < most ? want : most)), dim3(256), 0, stream, args);
}

cudaError_t launch_fp8_quantize_weights(const uint16_t* w, int64_t ldw, int64_t N, int64_t K, uint8_t* q, float* s,
                                        cudaStream_t stream) {
  int kb = (int)((K + 127) / 128), k = (int)K;
  const int64_t blocks = (N + 127) / 128 * kb;
  void* args[] = {&w, &ldw, &N, &k, &kb, &q, &s};
  return tc::launch_pdl((const void*)quantize_blocks_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, args);
}

cudaError_t read_and_clear_fp8_norm_timeouts(unsigned int* count) {
  const unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(count, g_fp8_norm_timeouts, sizeof(zero));
  if (e == cudaSuccess && *count) e = cudaMemcpyToSymbol(g_fp8_norm_timeouts, &zero, sizeof(zero));
  return e;
}

}  // namespace nvfp4
