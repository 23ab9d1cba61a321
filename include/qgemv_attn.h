/*
 * qgemv_attn.h -- C ABI of what stands between a layer's qkv projection and
 * its output projection: norms of the query and key heads with the rotation
 * of positions (forward and backward), a paged key-value cache that is
 * quantised as it is written, and attention of new tokens over it.
 * The conventions of qgemv.h hold (caller-owned device memory, the caller's
 * stream, no synchronization, arguments validated before anything is
 * enqueued); qg_status is defined there, the element types QG_F32, QG_F16 and
 * QG_BF16 and the f8 values in qgemv_f8.h.
 *
 * Head tensors.  [T][heads][D], the heads of a token contiguous, tokens `ld`
 * elements apart: the q, k and v parts of one projection's output are such
 * tensors.  1 <= T <= 2^30, 1 to 1024 heads in all.
 *
 * Norm and rotation of a head vector x[D], D a multiple of 8 from 8 to 256:
 *   n = x / sqrt(mean(x^2) + eps) * gain          (n = x without a gain)
 *   y = n with its first `rot` elements turned in pairs, rot a multiple of 8
 *       from 0 to D: pair i is (n[i], n[i + rot / 2]), interleaved (n[2 i],
 *       n[2 i + 1]); (a, b) becomes (a c - b s, b c + a s), c and s the cosine
 *       and sine of position * freq[i].
 * positions: int32 [axes][T], 1 <= axes <= 4 (time, height, width, ...);
 * pair i takes axis 0 if i < sections[0], axis 1 for the next sections[1]
 * pairs and so on, the sections summing up to rot / 2.  Any int32 is a
 * position: the angle's whole turns are taken out exactly to 2^-53 of a turn
 * (up to 2^51 turns), whatever their number.
 * freq: fp32 [rot / 2]; gains: type gain_type [D].
 * Everything is computed in fp32 and rounded once (the squares of a row sum up
 * to less than 2^128).  The gradient of a row needs nothing of the forward pass
 * but its inputs.
 *
 * Cache.  `pages` pages of qkv_page_bytes(page, heads, dim, type) bytes, each
 * holding `page` tokens of every key head, page 16, 32, ... 1024 (a power of
 * two), dim 64, 128, 192 or 256, type QG_F8, QG_F16 or QG_BF16:
 *   codes   at byte 0: [head][keys, values][token][dim];
 *   scales  (QG_F8) behind them: bytes [head][keys, values][token];
 *   total   rounded up to a multiple of 256 (the padding is never touched).
 * QG_F8 holds a token's key vector of a head, and its value vector, as dim
 * e4m3 codes and one power of two, by the rule of f8 blocks in qgemv_f8.h.
 * Token t of page p is slot p * page + t; pages * page <= 2^31 - 1.
 *
 * Sums, norms and softmax statistics are fp32 or wider; results are bitwise
 * reproducible: no atomics.
 */
#ifndef QGEMV_ATTN_H
#define QGEMV_ATTN_H

#include <stddef.h>
#include <stdint.h>

#include "qgemv.h"
#include "qgemv_f8.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { QG_F8 = 3 };

/* Bytes of one cache page; 0 if a size or the type is out of range (1 to 1024
 * heads). */
size_t qkv_page_bytes(int page, int heads, int dim, int type);

/* Norm and rotation of q[T][q_heads][D] and k[T][k_heads][D] (type x_type,
 * tokens ldq, ldk elements apart; k NULL with k_heads 0) into yq and yk (type
 * y_type, tokens ldyq, ldyk apart).  q_gain, k_gain: both or none; sections:
 * host memory, NULL for one axis; freq may be NULL if rot is 0, positions too. */
qg_status qhead_norm_rope(const void *q, int64_t ldq, int q_heads, const void *k, int64_t ldk, int k_heads, int x_type,
                          const void *q_gain, const void *k_gain, int gain_type, float eps, const int32_t *positions,
                          int axes, const int32_t *sections, const float *freq, int rot, int interleaved, int64_t T,
                          int D, void *yq, int64_t ldyq, void *yk, int64_t ldyk, int y_type, void *stream);

/* Its gradient: from gyq and gyk (type y_type, tokens ldgq, ldgk apart) and the
 * inputs of the forward call, gq and gk (type x_type, tokens lddq, lddk apart)
 * and, with gains, the fp32 sums over tokens and heads g_gain[2][D] (row 0
 * for q_gain, row 1 for k_gain; zeros without k).  workspace: as many bytes
 * as the size function says (0: may be NULL), 16-byte aligned, used by this
 * call only. */
size_t qhead_norm_rope_backward_workspace(int64_t T, int q_heads, int k_heads, int D, int gains);
qg_status qhead_norm_rope_backward(const void *gyq, int64_t ldgq, const void *gyk, int64_t ldgk, int y_type,
                                   const void *q, int64_t ldq, int q_heads, const void *k, int64_t ldk, int k_heads,
                                   int x_type, const void *q_gain, const void *k_gain, int gain_type, float eps,
                                   const int32_t *positions, int axes, const int32_t *sections, const float *freq,
                                   int rot, int interleaved, int64_t T, int D, void *gq, int64_t lddq, void *gk,
                                   int64_t lddk, float *g_gain, void *workspace, void *stream);

/* k and v[T][heads][dim] (type x_type, tokens ldk, ldv apart) into the slots
 * of the cache: token t into slots[t] (int32 [T], device).  A slot outside
 * 0 .. pages * page - 1 writes nothing (-1: padding).  If two tokens have the
 * same slot, that slot's values are unspecified, all others are not. */
qg_status qkv_write(const void *k, int64_t ldk, const void *v, int64_t ldv, int x_type, const int32_t *slots,
                    int64_t T, void *cache, int64_t pages, int page, int heads, int dim, int cache_type, void *stream);

/* The values of slots[t] as k and v[T][heads][dim] (contiguous, y_type); zeros
 * for slots outside the cache. */
qg_status qkv_read(const void *cache, int64_t pages, int page, int heads, int dim, int cache_type,
                   const int32_t *slots, int64_t T, void *k, void *v, int y_type, void *stream);

/* The serving form of both in one launch: norm and rotation of q into yq, of
 * k into the cache together with v as it is.  Keys that go into an 8-bit cache
 * are computed in 64 bits, so their codes are those of the exact values. */
qg_status qkv_norm_rope_write(const void *q, int64_t ldq, int q_heads, const void *k, int64_t ldk, const void *v,
                              int64_t ldv, int x_type, const void *q_gain, const void *k_gain, int gain_type,
                              float eps, const int32_t *positions, int axes, const int32_t *sections,
                              const float *freq, int rot, int interleaved, int64_t T, const int32_t *slots, void *yq,
                              int64_t ldyq, int y_type, void *cache, int64_t pages, int page, int heads, int dim,
                              int cache_type, void *stream);

/* Attention of the last M tokens of each of B sequences over their cache:
 *   q: [B][M][q_heads][dim], type q_type (QG_F16 or QG_BF16; the cache's type
 *   where that has 16 bits), tokens ldq elements apart; 1 <= M <= 16,
 *   q_heads a multiple of kv_heads, at most 1024: query heads
 *   j q_heads / kv_heads .. share key head j; 1 <= B <= 65536, B M q_heads <=
 *   2^23.
 *   table: int32 [B][width], the pages of a sequence in order, width * page <=
 *   2^30 and B times that <= 2^36; lens: int32 [B], its tokens, the M new ones
 *   among them (already written).
 * Token i of the M new ones stands at place p = lens[b] - M + i and sees the
 * places max(0, p - window + 1) .. p (window 0: all up to p):
 *   s = scale * q.k,  softcap > 0: s = softcap * tanh(s / softcap)  (scale /
 *   softcap finite; right to a few 2^-24 of the score however large the cap),
 *   out = sum softmax(s) v          [B][M][q_heads][dim], q_type, contiguous.
 * A query that sees no token gets zeros.  lens are held to 0 .. width * page;
 * a table entry outside 0 .. pages - 1 holds no tokens.  What lies in places
 * that a query does not see, NaN or infinity, does not reach it; a value that
 * is not finite makes its element of every query that sees it not finite,
 * infinity or NaN.  Products are exact with fp32 sums (8-bit keys beside bf16
 * queries down to multiples of 2^-133); the softmax's weights enter the second
 * product as two 16-bit parts (2^-16 of a weight is lost); one rounding to
 * q_type.  Weights reach 2^4 and are divided by their sum at the end: the values
 * that a query sees may sum up, in magnitude, to 2^123.  An 8-bit value's scale
 * enters its weight, in multiples of 2^-133: values of 2^-100 keep 2^-23 of the
 * largest.
 * workspace: qattn_decode_workspace bytes (0: may be NULL; at most 33 MiB,
 * however many sequences there are), 16-byte aligned, used by this call only. */
size_t qattn_decode_workspace(int64_t B, int M, int q_heads, int kv_heads, int dim, int cache_type, int page,
                              int64_t width);
qg_status qattn_decode(const void *cache, int64_t pages, int page, int kv_heads, int dim, int cache_type,
                       const void *q, int q_type, int64_t ldq, int64_t B, int M, int q_heads, const int32_t *table,
                       int64_t width, const int32_t *lens, float scale, int64_t window, float softcap, void *out,
                       void *workspace, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* QGEMV_ATTN_H */
