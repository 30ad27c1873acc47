// fp8_abi.cu -- the extern "C" entry points of include/fp8.h: host-side argument
// validation and dispatch.  Nothing here allocates device memory or synchronizes.
#include <cmath>

#include "fp8.h"
#include "nvfp4_kernels.h"

namespace {

using nvfp4::report_error;

constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 512;
constexpr int64_t kMaxTiles = (int64_t)1 << 30;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// The bytes of a tensor, from its first to its last element.
struct Range {
  const void* p;
  size_t n;
};
Range bf16_rows(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  return {p, p ? (size_t)((rows - 1) * ld + cols) * 2 : 0};
}
bool overlaps(Range a, Range b) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  return a.n && b.n && pa < pb + b.n && pb < pa + a.n;
}
// Whether an output overlaps an input or another output.
template <size_t NO, size_t NI>
bool any_overlap(const Range (&out)[NO], const Range (&in)[NI]) {
  for (size_t i = 0; i < NO; ++i) {
    for (size_t j = 0; j < NI; ++j)
      if (overlaps(out[i], in[j])) return true;
    for (size_t j = 0; j < i; ++j)
      if (overlaps(out[i], out[j])) return true;
  }
  return false;
}

nvfp4_status check_shape(const char* rows_name, int64_t rows, int64_t K) {
  if (K <= 0 || K % 16 != 0 || K > ((int64_t)1 << 24))
    return report_error(NVFP4_ERR_SHAPE, "K=%lld must be a positive multiple of 16, at most 2^24", (long long)K);
  if (rows < 0 || rows > kMaxRows)
    return report_error(NVFP4_ERR_SHAPE, "%s=%lld must be in 0..2^31-512", rows_name, (long long)rows);
  return NVFP4_OK;
}

nvfp4_status launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? NVFP4_OK : nvfp4::report_cuda_error(e, what);
}

}  // namespace

extern "C" {

nvfp4_status fp8_rmsnorm(const uint16_t* x, int64_t ldx, const uint16_t* weight, const uint16_t* residual, int64_t ldr,
                         uint16_t* residual_out, int64_t ldro, uint16_t* y, int64_t ldy, uint8_t* q, float* s,
                         int64_t M, int64_t K, float eps, nvfp4_stream_t stream) {
  nvfp4_status st = check_shape("M", M, K);
  if (st != NVFP4_OK) return st;
  if (!(eps >= 0.0f) || !std::isfinite(eps))
    return report_error(NVFP4_ERR_INVALID_ARG, "eps=%g must be finite and not negative", (double)eps);
  if (M == 0) return NVFP4_OK;  // (tensors without elements have null pointers)
  if ((residual != nullptr) != (residual_out != nullptr))
    return report_error(NVFP4_ERR_INVALID_ARG, "residual and residual_out go together");
  if ((q != nullptr) != (s != nullptr)) return report_error(NVFP4_ERR_INVALID_ARG, "q and s go together");
  if (!y && !q) return report_error(NVFP4_ERR_INVALID_ARG, "no output: give y, or q and s");
  if (!x || !weight) return report_error(NVFP4_ERR_INVALID_ARG, "null pointer");
  if (ldx < K || (residual && (ldr < K || ldro < K)) || (y && ldy < K))
    return report_error(NVFP4_ERR_INVALID_ARG, "a leading dimension is smaller than K=%lld", (long long)K);
  if (!aligned(x, 16) || ldx % 8 || !aligned(weight, 16) || (residual && (!aligned(residual, 16) || ldr % 8)) ||
      (residual && (!aligned(residual_out, 16) || ldro % 8)) || (y && (!aligned(y, 16) || ldy % 8)) ||
      (q && !aligned(q, 16)))
    return report_error(NVFP4_ERR_ALIGNMENT,
                        "BF16 tensors and q must be 16-byte aligned, leading dimensions multiples of 8");
  if (s && !aligned(s, 4)) return report_error(NVFP4_ERR_ALIGNMENT, "s must be 4-byte aligned");
  const Range rx = bf16_rows(x, M, K, ldx), rw = {weight, (size_t)K * 2}, rr = bf16_rows(residual, M, K, ldr);
  const Range ro = bf16_rows(residual_out, M, K, ldro), ry = bf16_rows(y, M, K, ldy);
  const Range rq = {q, q ? (size_t)(M * K) : 0}, rs = {s, s ? (size_t)(M * cdiv(K, 128)) * 4 : 0};
  const bool in_place = residual && residual == residual_out && ldr == ldro;
  if (any_overlap({ro, ry, rq, rs}, {rx, rw, in_place ? Range{nullptr, 0} : rr}))
    return report_error(NVFP4_ERR_INVALID_ARG,
                        "outputs must not overlap inputs or each other (residual_out may be residual itself)");
  int sms = 0;
  st = nvfp4::require_device(&sms);
  if (st != NVFP4_OK) return st;
  return launched(nvfp4::launch_fp8_rmsnorm(x, ldx, weight, residual, ldr, residual_out, ldro, y, ldy, q, s, M, K, eps, sms,
                                            (cudaStream_t)stream),
                  "rmsnorm launch");
}

nvfp4_status fp8_quantize(const uint16_t* X, int64_t ldx, int64_t M, int64_t K, uint8_t* q, float* s, uint32_t flags,
                          nvfp4_stream_t stream) {
  if (flags & ~FP8_FLAG_GATED) return report_error(NVFP4_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
  nvfp4_status st = check_shape("M", M, K);
  if (st != NVFP4_OK) return st;
  const int64_t cols = (flags & FP8_FLAG_GATED) ? 2 * K : K;
  if (M * cdiv(K, 128) > ((int64_t)1 << 31))
    return report_error(NVFP4_ERR_SHAPE, "M=%lld x K=%lld has more than 2^31 blocks", (long long)M, (long long)K);
  if (M == 0) return NVFP4_OK;
  if (!X || !q || !s) return report_error(NVFP4_ERR_INVALID_ARG, "null pointer");
  if (ldx < cols) return report_error(NVFP4_ERR_INVALID_ARG, "ldx=%lld < %lld columns", (long long)ldx, (long long)cols);
  if (!aligned(X, 16) || ldx % 8 || !aligned(q, 16) || !aligned(s, 4))
    return report_error(NVFP4_ERR_ALIGNMENT, "X and q must be 16-byte aligned, ldx a multiple of 8, s 4-byte aligned");
  if (any_overlap({{q, (size_t)(M * K)}, {s, (size_t)(M * cdiv(K, 128)) * 4}}, {bf16_rows(X, M, cols, ldx)}))
    return report_error(NVFP4_ERR_INVALID_ARG, "X, q and s must not overlap");
  int sms = 0;
  st = nvfp4::require_device(&sms);
  if (st != NVFP4_OK) return st;
  return launched(nvfp4::launch_fp8_quantize(X, ldx, M, K, (flags & FP8_FLAG_GATED) != 0, q, s, sms,
                                             (cudaStream_t)stream),
                  "fp8 quantize launch");
}

nvfp4_status fp8_quantize_weights(const uint16_t* W, int64_t ldw, int64_t N, int64_t K, uint8_t* q, float* s,
                                  nvfp4_stream_t stream) {
  nvfp4_status st = check_shape("N", N, K);
  if (st != NVFP4_OK) return st;
  if (N == 0) return NVFP4_OK;
  const int64_t blocks = cdiv(N, 128) * cdiv(K, 128);
  if (blocks > (int64_t)INT32_MAX)
    return report_error(NVFP4_ERR_SHAPE, "N=%lld x K=%lld has too many 128 x 128 blocks", (long long)N, (long long)K);
  if (!W || !q || !s) return report_error(NVFP4_ERR_INVALID_ARG, "null pointer");
  if (ldw < K) return report_error(NVFP4_ERR_INVALID_ARG, "ldw=%lld < K=%lld", (long long)ldw, (long long)K);
  if (!aligned(W, 16) || ldw % 8 || !aligned(q, 16) || !aligned(s, 4))
    return report_error(NVFP4_ERR_ALIGNMENT, "W and q must be 16-byte aligned, ldw a multiple of 8, s 4-byte aligned");
  if (any_overlap({{q, (size_t)(N * K)}, {s, (size_t)blocks * 4}}, {bf16_rows(W, N, K, ldw)}))
    return report_error(NVFP4_ERR_INVALID_ARG, "W, q and s must not overlap");
  int sms = 0;
  st = nvfp4::require_device(&sms);
  if (st != NVFP4_OK) return st;
  return launched(nvfp4::launch_fp8_quantize_weights(W, ldw, N, K, q, s, (cudaStream_t)stream),
                  "fp8 weight quantize launch");
}

}  // extern "C"

namespace {

// Both products; offsets == null: dense, E == 1.
nvfp4_status product(const uint8_t* x, const float* sx, const uint8_t* w, const float* sw, const int32_t* offsets,
                     bool grouped, uint16_t* Y, int64_t ldy, int64_t M, int64_t E, int64_t N, int64_t K, uint32_t flags,
                     nvfp4_stream_t stream) {
  const char* rows = grouped ? "T" : "M";
  if (flags & ~NVFP4_FLAG_STATIC_WEIGHTS) return report_error(NVFP4_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
  nvfp4_status st = check_shape(rows, M, K);
  if (st == NVFP4_OK) st = check_shape("N", N, K);
  if (st != NVFP4_OK) return st;
  if (E < 1 || E > FP8_MAX_EXPERTS)
    return report_error(NVFP4_ERR_SHAPE, "E=%lld must be in 1..%d", (long long)E, FP8_MAX_EXPERTS);
  if (E * N > kMaxRows) return report_error(NVFP4_ERR_SHAPE, "E=%lld x N=%lld is too large", (long long)E, (long long)N);
  if (M == 0 || N == 0) return NVFP4_OK;
  const int64_t nb = cdiv(N, 128), kb = cdiv(K, 128);
  // output tiles, of at least 16 x 128, and their shares of K are numbered with 32-bit integers
  if (nb * (cdiv(M, 16) + E) > kMaxTiles)
    return report_error(NVFP4_ERR_SHAPE, "%s=%lld x N=%lld has too many tiles", rows, (long long)M, (long long)N);
  if (!x || !sx || !w || !sw || !Y || (grouped && !offsets)) return report_error(NVFP4_ERR_INVALID_ARG, "null pointer");
  if (ldy < N) return report_error(NVFP4_ERR_INVALID_ARG, "ldy=%lld < N=%lld", (long long)ldy, (long long)N);
  if (!aligned(x, 16) || !aligned(w, 16))
    return report_error(NVFP4_ERR_ALIGNMENT, "x and w must be 16-byte aligned");
  if (!aligned(sx, 4) || !aligned(sw, 4) || !aligned(offsets, 4) || !aligned(Y, 2))
    return report_error(NVFP4_ERR_ALIGNMENT, "scales and offsets must be 4-byte aligned, Y 2-byte aligned");
  if (any_overlap({bf16_rows(Y, M, N, ldy)},
                  {{x, (size_t)(M * K)}, {sx, (size_t)(M * kb) * 4}, {w, (size_t)(E * N * K)},
                   {sw, (size_t)(E * nb * kb) * 4}, {offsets, offsets ? (size_t)(E + 1) * 4 : 0}}))
    return report_error(NVFP4_ERR_INVALID_ARG, "Y must not overlap an input");
  int sms = 0;
  st = nvfp4::require_device(&sms);
  if (st != NVFP4_OK) return st;
  return launched(nvfp4::launch_fp8_gemm(x, sx, w, sw, offsets, Y, ldy, M, E, N, K,
                                         (flags & NVFP4_FLAG_STATIC_WEIGHTS) != 0, sms, (cudaStream_t)stream),
                  grouped ? "grouped fp8 gemm launch" : "fp8 gemm launch");
}

}  // namespace

extern "C" {

nvfp4_status fp8_gemm(const uint8_t* x, const float* sx, const uint8_t* w, const float* sw, uint16_t* Y, int64_t ldy,
                      int64_t M, int64_t N, int64_t K, uint32_t flags, nvfp4_stream_t stream) {
  return product(x, sx, w, sw, nullptr, false, Y, ldy, M, 1, N, K, flags, stream);
}

nvfp4_status fp8_gemm_grouped(const uint8_t* x, const float* sx, const uint8_t* w, const float* sw,
                              const int32_t* offsets, uint16_t* Y, int64_t ldy, int64_t T, int64_t E, int64_t N,
                              int64_t K, uint32_t flags, nvfp4_stream_t stream) {
  return product(x, sx, w, sw, offsets, true, Y, ldy, T, E, N, K, flags, stream);
}

}  // extern "C"
