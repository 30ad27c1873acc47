/*
 * fp8.h -- 8-bit (FP8 E4M3) linear layer with one fp32 scale per 128, for
 * NVIDIA B200 (sm_100a), beside the 4-bit entry points of nvfp4.h (same
 * library, status codes and conventions: device pointers owned by the caller,
 * asynchronous on `stream`, host-side validation, nothing allocated, no
 * synchronization).
 *
 * The pages name block-FP8 weights only as the format that another engine falls
 * back to (model card "Qwen3.8-27B-NVFP4", vLLM paragraph) and give no kernels.
 * Here an 8-bit layer is four kinds of call: the RMS norm or a quantizer writes
 * 8-bit activations, and the product, dense or grouped by expert, multiplies
 * them by 8-bit weights.
 *
 * Layouts (row-major, no padding inside a row; kb = ceil(K / 128); the last
 * block of a row or column may be short):
 *   activations  q E4M3 [M, K],  s fp32 [M, kb]: one scale per row and 128 columns
 *   weights      q E4M3 [N, K],  s fp32 [ceil(N / 128), kb]: one per 128 x 128 block
 *   a value is e4m3(q) * s
 * Quantization rule of a block with values v (fp32, round to nearest even):
 *   s = max(max |v| / 448, 2^-126);  q = E4M3_rne_satfinite(v * (1 / s))
 * A NaN value gives a NaN code and leaves the rest of its block alone; a block
 * with an infinity gets the scale infinity, and its products are NaN.
 *
 * K is a positive multiple of 16, at most 2^24; M, N at most 2^31 - 512.
 * BF16 tensors that are read, residual_out and the norm's y need 16-byte
 * alignment and leading dimensions that are multiples of 8; q 16-byte
 * alignment; scales and offsets 4-byte; the products' Y 2-byte alignment and
 * any ldy >= N.  Outputs must not overlap inputs or each other (compared as
 * the address ranges from a tensor's first to its last element), residual_out
 * excepted.
 */
#ifndef FP8_H_
#define FP8_H_

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* fp8_quantize: X is [M, 2K], gate columns then up columns, and silu(gate) * up
 * is quantized, computed in fp32 with silu within 2^-15 of itself (for silu a
 * normal fp32 number, gates above -91). */
#define FP8_FLAG_GATED 2u

/* Most experts of one fp8_gemm_grouped call. */
#define FP8_MAX_EXPERTS 4096

/*
 * RMS norm, with the residual's addition and an 8-bit output:
 *   h = residual ? bf16_rne(x + residual) : x        (written to residual_out)
 *   v = h / sqrt(mean(h^2) + eps) * weight           (fp32; the sum of squares in fp32)
 *   y = bf16_rne(v) if y is given;  (q, s) = v quantized per row and 128
 *   columns if q and s are given (from v, not from its BF16 value)
 * x, residual, residual_out, y: BF16 [M, K] with leading dimensions ldx, ldr,
 * ldro, ldy; weight: BF16 [K].  residual and residual_out go together (both or
 * neither); residual_out may be residual itself (same address, ldro == ldr).
 * q and s go together; at least one of y and (q, s) is given.  eps is finite
 * and not negative.  M == 0 is a no-op.
 */
NVFP4_API nvfp4_status fp8_rmsnorm(const uint16_t* x, int64_t ldx, const uint16_t* weight, const uint16_t* residual,
                                   int64_t ldr, uint16_t* residual_out, int64_t ldro, uint16_t* y, int64_t ldy,
                                   uint8_t* q, float* s, int64_t M, int64_t K, float eps, nvfp4_stream_t stream);

/*
 * Activations X (BF16 [M, K], leading dimension ldx; [M, 2K] with
 * FP8_FLAG_GATED) into q [M, K] and s [M, kb].  M == 0 is a no-op.
 */
NVFP4_API nvfp4_status fp8_quantize(const uint16_t* X, int64_t ldx, int64_t M, int64_t K, uint8_t* q, float* s,
                                    uint32_t flags, nvfp4_stream_t stream);

/* Weights W (BF16 [N, K], leading dimension ldw) into q [N, K] and
 * s [ceil(N / 128), kb].  N == 0 is a no-op. */
NVFP4_API nvfp4_status fp8_quantize_weights(const uint16_t* W, int64_t ldw, int64_t N, int64_t K, uint8_t* q, float* s,
                                            nvfp4_stream_t stream);

/*
 * Y[m, n] = bf16_rne( sum_b sx[m, b] sw[n / 128, b] sum_{k in block b} x[m, k] w[n, k] ),
 * each block's sum on the tensor cores (fp32), the sum over blocks in fp32.
 * A block's sx * sw is formed first, in fp32, and should be a normal number there:
 * below 2^-126 it has fewer bits (its share of the sum is off by up to 2^-150
 * times the block's sum), from 2^128 on it is infinite and the output infinite or
 * NaN, also where the block's sum is zero.
 * x, sx: activations [M, K]; w, sw: weights [N, K]; Y: BF16 [M, N], leading
 * dimension ldy.  Deterministic.  flags: NVFP4_FLAG_STATIC_WEIGHTS (w; sw is
 * read after the preceding work either way).  M == 0 or N == 0 is a no-op.
 */
NVFP4_API nvfp4_status fp8_gemm(const uint8_t* x, const float* sx, const uint8_t* w, const float* sw, uint16_t* Y,
                                int64_t ldy, int64_t M, int64_t N, int64_t K, uint32_t flags, nvfp4_stream_t stream);

/*
 * The same product grouped by expert: rows offsets[e] .. offsets[e + 1] - 1 of
 * X [T, K] and Y [T, N] belong to expert e of the stacked weights w [E, N, K],
 * sw [E, ceil(N / 128), kb].  offsets: device int32 [E + 1], not decreasing,
 * within 0 .. T (e.g. written by a router earlier on the stream); experts may
 * have no rows.  Rows of Y outside offsets[0] .. offsets[E] - 1 keep what they
 * hold.  Offsets that decrease or leave 0 .. T are clamped (each to 0 .. T, and
 * an expert starts no earlier than any before it ends, so no row is read or
 * written outside X and Y, and none twice); the call is counted for
 * nvfp4_check_device_errors (NVFP4_ERR_INVALID_ARG).  flags:
 * NVFP4_FLAG_STATIC_WEIGHTS (changes nothing here: the experts are known only
 * after the preceding work).  1 <= E <= FP8_MAX_EXPERTS, E * N < 2^31.
 * T == 0 or N == 0 is a no-op.
 */
NVFP4_API nvfp4_status fp8_gemm_grouped(const uint8_t* x, const float* sx, const uint8_t* w, const float* sw,
                                        const int32_t* offsets, uint16_t* Y, int64_t ldy, int64_t T, int64_t E,
                                        int64_t N, int64_t K, uint32_t flags, nvfp4_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8_H_ */
