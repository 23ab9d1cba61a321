/*
 * qgemv_f8.h -- C ABI of the 8-bit floating point operators: matrix products
 * with a scale for each block of 128, 8-bit activation checkpoints with the
 * products of the backward pass, and expert routing with the balance loss.
 * The conventions of qgemv.h hold (caller-owned device memory, the caller's
 * stream, no synchronization, arguments validated before anything is
 * enqueued); qg_status is defined there.
 *
 * f8 values.  A code is an OCP e4m3 byte (largest value 448, no infinity,
 * 0x7f / 0xff are NaN); a scale is a power of two 2^e held as the byte
 * e + 127 (0..254).  A block's scale is the smallest 2^e, e >= -127, with
 * |v| <= 448 * 2^e for every finite v of the block, and 2^0 where all of
 * them are zero; a code is v / 2^e rounded to nearest, ties to even, and at
 * most 240 under 2^120, the largest scale (256 would be 2^128), so finite
 * values stay finite.  A power of two costs a floating code no precision and
 * keeps values exact in bf16, down to multiples of 2^-133, bf16's smallest
 * step: only a block whose largest magnitude is below 448 * 2^-124 holds
 * values between those, which dequantize exactly in fp32 and enter products to
 * within 2^-133.
 *   Weights N x K: one scale per 128 x 128 block.
 *   Activations M x K: one scale per 128 elements of a row; infinities and
 *   NaNs become the NaN code and do not enter the block's scale, so they
 *   reach only the outputs of their own row.
 *
 * Packed weights (one N x K matrix, any N, K >= 1; rb = ceil(N / 128),
 * cb = ceil(K / 128), rt = ceil(N / 16), ls = cb rounded up to 4):
 *   codes   at byte 0: tiles of 16 rows x 128 columns, 2048 bytes each, tile
 *           (t, c) at byte 2048 (t cb + c).  Inside a tile the code of row r,
 *           column k is at byte 256 (k / 16) + 16 r + k % 16: the order in
 *           which a wave's lanes hold a matrix-core operand, so a wave reads
 *           whole kilobytes.
 *   scales  at byte S0 = 2048 rt cb: byte (n / 128) ls + k / 128.
 *   total   S0 + rb ls, rounded up to a multiple of 256; padding is zero.
 * Packed activations (M x K): codes [M][128 cb] row-major at byte 0 (columns
 * K.. zero), scales at byte S0 = 128 M cb rounded up to 256: byte m ls + c
 * (the padding of a scale row is unspecified); total rounded up to 256.
 *
 * Element types of inputs and outputs: QG_F32, QG_F16, QG_BF16.
 *
 * Accuracy of the products.  Both sides are widened to bf16, exactly, and
 * multiplied with fp32 sums, whose roundings are all that is lost: at most
 * (K / 8 + 16) 2^-24 sum |w x|, about 1e-7 of the result on ordinary data.
 * 16-bit outputs are rounded once from these sums.
 * Results are bitwise reproducible: no atomics.
 */
#ifndef QGEMV_F8_H
#define QGEMV_F8_H

#include <stddef.h>
#include <stdint.h>

#include "qgemv.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { QG_F32 = 0, QG_F16 = 1, QG_BF16 = 2 };

/* ------------------------------------------------------------ host side */

/* Bytes of one packed N x K weight matrix, and of packed M x K activations;
 * 0 if a size is < 1, K > 2^20 or a row count > 2^30. */
size_t qpacked_bytes_f8(int64_t N, int64_t K);
size_t qact_bytes_f8(int64_t M, int64_t K);

/* Quantize and pack fp32 weights w[N][K] (host) into `packed` (host, at least
 * qpacked_bytes_f8 bytes).  QG_ERR_RANGE (after writing every block) if a
 * weight is not finite; its code is NaN. */
qg_status qquantize_f8(const float *w, int64_t N, int64_t K, void *packed, size_t packed_bytes);

/* ----------------------------------------------------------- device side
 * Packed buffers are 256-byte aligned, workspaces 16-byte, other pointers to
 * the size of their elements.  1 <= N, M <= 2^30,
 * 1 <= K <= 2^20 (and N <= 2^20 where N is the summed side). */

/* Packed weights -> out[N][K], fp32 (out_fp16 = 0) or fp16 rounded to nearest
 * even (1). */
qg_status qdequant_f8(const void *Wp, int64_t N, int64_t K, int out_fp16, void *out, void *stream);

/* The packed N x K matrix Wp as the packed K x N matrix WpT (exact: codes and
 * scales only move), the operand of dx = f8(dy) W.  The buffers must not
 * overlap. */
qg_status qtranspose_f8(const void *Wp, int64_t N, int64_t K, void *WpT, void *stream);

/* x[M][K] (type x_type, rows ldx >= K elements apart) -> packed activations:
 * the operand of the products below and, kept until the backward pass, an
 * activation checkpoint of 8 bits a value. */
qg_status qact_quantize_f8(const void *x, int x_type, int64_t ldx, int64_t M, int64_t K, void *xq, void *stream);

/* Packed activations -> out[M][K] (contiguous, rounded to nearest even where
 * the type is narrower; exact in fp32 and bf16 above their subnormals). */
qg_status qact_dequant_f8(const void *xq, int64_t M, int64_t K, int out_type, void *out, void *stream);

/* One-launch product for 1 <= M <= 8 tokens: x[M][K] (type x_type,
 * contiguous) is quantized inside the launch, as qact_quantize_f8 does, and
 *   y[m][n] = sum_k f8(x)[m][k] W[n][k],   y: fp32 [M][N].
 * K <= 16384.  Every value equals qgemm_f8's on the packed activations up to
 * the order of the fp32 sums. */
qg_status qgemv_f8(const void *Wp, const void *x, int x_type, float *y, int M, int64_t N, int64_t K, void *stream);

/* Y[m][n] = sum_k X[m][k] W[n][k] on packed activations, any M >= 1.
 * Y: y_type [M][N], contiguous. */
qg_status qgemm_f8(const void *Wp, const void *xq, void *Y, int y_type, int64_t M, int64_t N, int64_t K, void *stream);

/* Weight gradient from an 8-bit checkpoint: dW[n][k] = sum_m dY[m][n] X[m][k]
 * (+ dW[n][k] with accumulate), dY: bf16 [M][N] contiguous, X packed M x K,
 * dW: fp32 [N][K].  The checkpoint's values are exact in bf16: the only
 * roundings are those of the fp32 sums.  workspace: device memory of
 * qgemm_f8_wgrad_workspace(M, N, K) bytes (0: may be NULL), 16-byte aligned,
 * used by this call only. */
size_t qgemm_f8_wgrad_workspace(int64_t M, int64_t N, int64_t K);
qg_status qgemm_f8_wgrad(const void *dY, const void *xq, float *dW, int accumulate, int64_t M, int64_t N, int64_t K,
                         void *workspace, void *stream);

/* ------------------------------------------------------------- experts */

/* Top-k softmax routing of T tokens over E experts.
 *   logits: type [T][E], rows ldl >= E elements apart; 1 <= E <= 512,
 *   1 <= k <= min(E, 16), 1 <= T <= 2^24; token_mask: uint8 [T] or NULL,
 *   0 = the token is not routed (padding).
 * An expert is open to a token if its logit is above -infinity; a token that
 * is not masked and has an open expert is live.  With p = softmax(logits) of
 * a live token (0 elsewhere):
 *   idx[t][j]     the j-th largest logit's expert (ties: the lowest index);
 *                 -1 where there is none (fewer than k open experts, or the
 *                 token is not live)
 *   weight[t][j]  p of that expert, with renormalize divided by the sum of
 *                 the token's chosen p; 0 at idx -1
 *   counts[e]     slots routed to e (slot t k + j); counts[E] = live tokens n
 *   offsets[e], order[r]   the slots sorted by expert, ascending inside an
 *                 expert: those of e are order[offsets[e] .. offsets[e+1]);
 *                 slots without an expert come last, from offsets[E]
 *   loss          E * sum_e (counts[e] / (k n)) * (sum_t p[t][e] / n), the
 *                 balance loss (1 when both are even; 0 if n is 0)
 * A NaN logit ranks below every number and is closed, but makes its token's
 * p NaN; +infinity does so too.  workspace: qmoe_route_workspace(T, E) bytes
 * of device memory, 16-byte aligned, used by this call only. */
size_t qmoe_route_workspace(int64_t T, int64_t E);
qg_status qmoe_route(const void *logits, int type, int64_t ldl, const uint8_t *token_mask, int64_t T, int64_t E,
                     int k, int renormalize, int32_t *idx, float *weight, int32_t *counts, int32_t *offsets,
                     int32_t *order, float *loss, void *workspace, void *stream);

/* Gradient of weight and loss with respect to the logits (counts and the
 * choice of experts are constants): grad_weight fp32 [T][k] or NULL (0),
 * grad_loss fp32 [1] on the device or NULL (0); logits, token_mask, idx,
 * weight and counts as of the forward call.  dlogits: type [T][E],
 * contiguous; 0 for closed experts and tokens that are not live. */
qg_status qmoe_route_backward(const void *logits, int type, int64_t ldl, const uint8_t *token_mask, int64_t T,
                              int64_t E, int k, int renormalize, const int32_t *idx, const float *weight,
                              const int32_t *counts, const float *grad_weight, const float *grad_loss,
                              void *dlogits, void *stream);

/* Products of the slots with their experts' matrices, in one launch: for each
 * r in offsets[e] .. offsets[e+1] - 1, with s = order[r],
 *   Y[s][n] = sum_k X[s / k_slots][k] W_e[n][k],
 * and Y[s] = 0 for the slots from offsets[P] on.  pool: P packed N x K
 * matrices, qpacked_bytes_f8(N, K) apart, 1 <= P <= 512; xq: packed T x K
 * activations, 1 <= k_slots <= 16, T k_slots <= 2^30, T ceil(K / 128) <=
 * 2^25 - 2 (X's codes within 4 GiB); order int32 [T k_slots], offsets int32
 * [P + 1] (device, as qmoe_route writes them); Y: y_type [T k_slots][N].  With k_slots = 1, X has
 * a row for each slot (the second product of an expert).  An entry of order
 * outside 0 .. T k_slots - 1 is skipped, offsets are held to 0 .. T k_slots. */
qg_status qmoe_gemm_f8(const void *pool, int64_t P, const void *xq, int64_t T, int k_slots, const int32_t *order,
                       const int32_t *offsets, void *Y, int y_type, int64_t N, int64_t K, void *stream);

/* Weight gradients of the experts: dW[e][n][k] = sum over the slots s of e of
 * dY[s][n] X[s / k_slots][k] (+ dW with accumulate; without it an expert that
 * has no slots gets zeros).  dY: bf16 [T k_slots][N], dW: fp32 [P][N][K]. */
qg_status qmoe_gemm_f8_wgrad(const void *dY, const void *xq, int64_t T, int k_slots, const int32_t *order,
                             const int32_t *offsets, int64_t P, float *dW, int accumulate, int64_t N, int64_t K,
                             void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QGEMV_F8_H */
