/*
 * fp8bs_g128.h - the entry points of libfp8bs.so whose scales cover 128 values:
 * E4M3 products with one fp32 scale per row and 128 K of the activations and
 * one per 128x128 block of the weight, for one matrix or for ragged groups of
 * rows, the quantizers that feed them, and the backward products of an expert
 * layer.  The 32-value forms are in fp8bs.h; status codes, pointer ownership,
 * streams and errors are those of fp8bs.h, and so is the E4M3 format.
 *
 * Conventions of this header
 *   - ceil128(n) = (n + 127) / 128.  A dimension that is not a multiple of 128
 *     has a partial last block, which is scaled by itself.
 *   - Columns and K must be multiples of 16, and so must N (else
 *     FP8BS_ESHAPE); rows and group sizes are arbitrary.  A product's K and both
 *     N and K of a weight gradient are at most 2^22, every other dimension at
 *     most 2^30, and a call whose grid would not fit one launch is refused
 *     (FP8BS_ESHAPE; that takes 2^24 tiles or blocks, of 32 x 32 at least, or
 *     close to 2^31 regions of 4 rows x 512 columns).
 *   - Matrix pointers are 16-byte aligned, scale and offset pointers 4-byte
 *     aligned (else FP8BS_EALIGN).
 *   - The quantizer's rule for a group of values with absolute maximum amax:
 *       s = amax / 448 (fp32, round to nearest);  s == 0: codes 0x00;
 *       else q = E4M3(x / s), the quotient in fp32, ties to even, clamped to
 *       +-448, sign kept.
 *     Inputs must be finite: a group that holds an infinity or a NaN has no
 *     defined codes (the other groups' are not affected).
 *   - Results are batch invariant: an output row depends on its own inputs
 *     only, never on the other rows, on how many there are or on which kernel
 *     ran.  K is accumulated in ascending order of its 128-deep blocks.
 */
#ifndef FP8BS_G128_H
#define FP8BS_G128_H

#include "fp8bs.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * fp8bs_quantize_tg128 - bf16 -> E4M3 with one scale per row and 128 columns.
 *   x [rows, cols] bf16, q [rows, cols] E4M3 out,
 *   scales [rows, ceil128(cols)] fp32 out.
 *   rows == 0 or cols == 0: no-op.
 */
fp8bs_status fp8bs_quantize_tg128(const void* x_bf16, int64_t rows, int64_t cols, void* q_e4m3, float* scales,
                                  void* stream);

/*
 * fp8bs_quantize_b128 - G matrices bf16 -> E4M3 with one scale per 128x128
 *   block, and, if qt is given, the transposed codes as well: with a weight
 *   [N, K] the codes q serve the forward product and qt the product of the
 *   input gradient, bit for bit the same values.
 *   x  [G, rows, cols] bf16
 *   q  [G, rows, cols] E4M3 out, scales [G, ceil128(rows), ceil128(cols)] fp32 out
 *   qt [G, cols, rows] E4M3 out, scales_t [G, ceil128(cols), ceil128(rows)] fp32
 *      out; both NULL, or both given, and then rows % 16 == 0 (else FP8BS_ESHAPE)
 *   1 <= G (else FP8BS_EINVAL); G * ceil128(rows) <= 2^30.
 */
fp8bs_status fp8bs_quantize_b128(const void* x_bf16, int64_t G, int64_t rows, int64_t cols, void* q_e4m3,
                                 float* scales, void* qt_e4m3, float* scales_t, void* stream);

/*
 * fp8bs_gemm_tg128_nt - C[i,j] = sum_kb sa[i,kb] * sbt[j/128,kb] * P,
 *   P = sum_{k in kb} A[i,k] Bt[j,k] over the 128-deep K-block kb.
 *   P is formed by one matrix instruction, multiplied by the fp32 product
 *   sa*sbt (one rounding) and added into one fp32 accumulator by a fused
 *   multiply-add, K-blocks ascending; C is rounded once to bf16 (nearest,
 *   ties to even) and an exact zero is stored as +0.
 *   The instruction forms P from 16 groups of 8 consecutive K.  A product's
 *   exponent sum is that of its two codes' exponents (a subnormal code's and a
 *   zero's is -6, see fp8bs_gemm_e8m0_nt); with S the largest one of a group, each of
 *   the group's products is cut toward zero to a multiple of 2^(S-13).  A product
 *   is a multiple of 2^(-6) times 2^(its exponent sum), so those whose exponent sum
 *   is within 7 of S lose nothing, and P is within the sum over the groups of
 *   8 * 2^(S-13) of its exact value, beside at most 2^(T-23) more per group (T the
 *   K-block's largest exponent sum) and the rounding to fp32.  These losses are
 *   relative to the products: where products cancel they can exceed the bf16
 *   rounding of C.  (fp8bs_gemm_tg_nt, with scales of 32 values, forms its partial
 *   sums without them.)  They do not build up along K, since the accumulator across
 *   K-blocks is fp32 arithmetic.
 *   a  [M, K] E4M3,  sa  [M, ceil128(K)] fp32
 *   bt [N, K] E4M3,  sbt [ceil128(N), ceil128(K)] fp32
 *   c  [M, N] bf16 out
 *   M == 0 or N == 0: no-op.  K == 0: C is filled with +0.
 *   The product of the input gradient, dX[M, K] = dY[M, N] W[N, K], is this
 *   call on dY quantized by rows and on the transposed codes of W.
 */
fp8bs_status fp8bs_gemm_tg128_nt(const void* a, const float* sa, const void* bt, const float* sbt, void* c_bf16,
                                 int64_t M, int64_t N, int64_t K, void* stream);

/*
 * fp8bs_grouped_gemm_tg128_nt - the same for G consecutive row ranges of A,
 *   range g = rows [offsets[g], offsets[g+1]) with the weight bt[g], bit for
 *   bit fp8bs_gemm_tg128_nt of those rows.
 *   a  [M_total, K] E4M3, sa [M_total, ceil128(K)] fp32
 *   bt [G, N, K] E4M3, sbt [G, ceil128(N), ceil128(K)] fp32
 *   offsets [G+1] int32 on the device, ascending, entries in [0, M_total], any
 *      values (no alignment); they are read when the kernel runs, so a captured
 *      graph follows them.  Not checked on the host.  Entries are clamped into
 *      [0, M_total] and a range that runs backwards is empty, so a bad table
 *      gives wrong rows, never an access out of bounds.
 *   c  [M_total, N] bf16 out; rows outside every range are left as they were.
 *   1 <= G <= FP8BS_MAX_GROUPS (else FP8BS_EINVAL).
 */
fp8bs_status fp8bs_grouped_gemm_tg128_nt(const void* a, const float* sa, const void* bt, const float* sbt,
                                         const int32_t* offsets_dev, int32_t G, void* c_bf16, int64_t M_total,
                                         int64_t N, int64_t K, void* stream);

/*
 * fp8bs_grouped_wgrad - the weight gradients of a grouped product,
 *     dW_g[n,k] = sum_{m in range g} dY[m,n] X[m,k]
 *   from bf16 operands (exact products, fp32 accumulation, rows ascending).
 *   dy [M_total, N] bf16, x [M_total, K] bf16
 *   offsets [G+1] int32 on the device, as for fp8bs_grouped_gemm_tg128_nt
 *   dw [G, N, K] fp32: overwritten (an empty range gives zeros), or, if
 *      accumulate != 0, added to (one fp32 addition per element; an empty range
 *      leaves dw[g] as it was).
 *   1 <= G <= FP8BS_MAX_GROUPS (else FP8BS_EINVAL); M_total == 0 is every
 *   range empty; N == 0 or K == 0: no-op.  N and K multiples of 16.
 */
fp8bs_status fp8bs_grouped_wgrad(const void* dy_bf16, const void* x_bf16, const int32_t* offsets_dev, int32_t G,
                                 float* dw, int32_t accumulate, int64_t M_total, int64_t N, int64_t K, void* stream);

/*
 * fp8bs_swiglu_quantize_tg128 - y = silu(gate) * up and its quantizer, between
 *   the two products of an expert: per row of gu = [gate | up]
 *     y_i = g_i * sigma(g_i) * u_i, sigma(g) = 1 / (1 + exp(-g))      (fp32)
 *     q, scales = the row quantizer's rule on the fp32 y (not on a bf16 y)
 *   gu [rows, 2d] bf16 (d gates, then d ups), q [rows, d] E4M3 out,
 *   scales [rows, ceil128(d)] fp32 out, y [rows, d] bf16 out (rounded to
 *   nearest) or NULL.  d % 16 == 0 and d <= 2^29 (else FP8BS_ESHAPE).
 */
fp8bs_status fp8bs_swiglu_quantize_tg128(const void* gu_bf16, int64_t rows, int64_t d, void* q_e4m3, float* scales,
                                         void* y_bf16, void* stream);

/*
 * fp8bs_swiglu_backward_quantize_tg128 - its gradient, with the quantizer that
 *   the input gradient's product needs:
 *     dg_i = dy_i * u_i * sigma(g_i) * (1 + g_i * (1 - sigma(g_i)))   (fp32)
 *     du_i = dy_i * g_i * sigma(g_i)
 *     dgu  = [dg | du] rounded to bf16 (for the weight gradient)
 *     q, scales = the row quantizer's rule on the fp32 row [dg | du]
 *   gu [rows, 2d] bf16, dy [rows, d] bf16, dgu [rows, 2d] bf16 out,
 *   q [rows, 2d] E4M3 out, scales [rows, ceil128(2d)] fp32 out,
 *   y [rows, d] bf16 out, the forward value again (for the second product's
 *   weight gradient), or NULL.  d as above.
 */
fp8bs_status fp8bs_swiglu_backward_quantize_tg128(const void* gu_bf16, const void* dy_bf16, int64_t rows, int64_t d,
                                                  void* dgu_bf16, void* q_e4m3, float* scales, void* y_bf16,
                                                  void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BS_G128_H */
