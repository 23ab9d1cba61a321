// C-ABI entry points of qgemv_attn.h: host-side validation, then launches on
// the caller's stream.  Nothing here allocates device memory or synchronizes.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "qgemv_attn.h"
#include "qgemv_attn_internal.h"

namespace qg {
namespace {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline qg_status status(hipError_t e) { return e == hipSuccess ? QG_OK : QG_ERR_LAUNCH; }
inline hipStream_t on(void *stream) { return static_cast<hipStream_t>(stream); }
inline bool tokens_ok(int64_t T) { return T >= 1 && T <= kAttnMaxTokens; }

// Tokens of `heads` heads of D elements, ld apart.
inline bool rows_ok(int64_t ld, int heads, int D, int64_t T)
{
    return ld >= (int64_t)heads * D && ld <= INT64_MAX / 8 / T;
}

// The queries and the table of an attention call.
inline bool batch_ok(int64_t B, int M, int q_heads, int kv_heads, int page, int64_t width)
{
    return B >= 1 && B <= kAttnMaxBatch && M >= 1 && M <= kAttnMaxNew && kv_heads >= 1 && q_heads >= kv_heads &&
           q_heads <= kAttnMaxHeads && q_heads % kv_heads == 0 && B * M * q_heads <= kAttnMaxRows && width >= 1 &&
           width <= kAttnMaxPlaces / page && B * width * page <= kAttnMaxTable;
}

qg_status check_cache(const void *cache, int64_t pages, int page, int heads, int dim, int type)
{
    if (!cache)
        return QG_ERR_NULL;
    if (!page_ok(page) || !cache_dim_ok(dim) || !cache_type_ok(type) || heads < 1 || heads > kAttnMaxHeads ||
        pages < 1 || pages > INT32_MAX / page)
        return QG_ERR_SHAPE;
    return aligned(cache, 256) ? QG_OK : QG_ERR_ALIGN;
}

// What the calls with norms and rotation have in common; fills `a`.
qg_status check_heads(HeadArgs &a, const void *q, int64_t ldq, int q_heads, const void *k, int64_t ldk, int k_heads,
                      int x_type, const void *q_gain, const void *k_gain, int gain_type, float eps,
                      const int32_t *positions, int axes, const int32_t *sections, const float *freq, int rot,
                      int interleaved, int64_t T, int D)
{
    if (!q || (k_heads != 0 && !k) || (rot > 0 && (!positions || !freq)) || (axes > 1 && !sections) ||
        (q_gain == nullptr) != (k_gain == nullptr))
        return QG_ERR_NULL;
    if (!tokens_ok(T) || q_heads < 1 || k_heads < 0 || q_heads > kAttnMaxHeads || k_heads > kAttnMaxHeads - q_heads ||
        D < 8 || D > 256 || D % 8 || rot < 0 || rot > D || rot % 8 || axes < 1 || axes > kMaxAxes || !type_ok(x_type) ||
        !(eps >= 0.0f) || std::isinf(eps) || (q_gain && !type_ok(gain_type)) || !rows_ok(ldq, q_heads, D, T) ||
        (k_heads && !rows_ok(ldk, k_heads, D, T)))
        return QG_ERR_SHAPE;
    a = HeadArgs{};
    int end = 0;
    for (int i = 0; i < axes; ++i) {
        const int n = sections ? sections[i] : rot / 2;
        if (n < 0 || n > rot / 2 - end)
            return QG_ERR_SHAPE;
        a.sections[i] = end += n;
    }
    if (end != rot / 2)
        return QG_ERR_SHAPE;
    if (!aligned(q, type_bytes(x_type)) || !aligned(k, type_bytes(x_type)) ||
        (q_gain && (!aligned(q_gain, type_bytes(gain_type)) || !aligned(k_gain, type_bytes(gain_type)))) ||
        !aligned(positions, 4) || !aligned(freq, 4))
        return QG_ERR_ALIGN;
    a.x[0] = q, a.x[1] = k;
    a.ldx[0] = ldq, a.ldx[1] = ldk;
    a.heads[0] = q_heads, a.heads[1] = k_heads;
    a.gain[0] = q_gain, a.gain[1] = k_gain;
    a.gain_type = gain_type;
    a.eps = eps;
    a.positions = positions;
    a.freq = freq;
    a.axes = axes;
    a.half = rot / 2;
    a.interleaved = interleaved != 0;
    a.T = T;
    a.D = D;
    return QG_OK;
}

}  // namespace
}  // namespace qg

using namespace qg;

extern "C" {

size_t qkv_page_bytes(int page, int heads, int dim, int type)
{
    if (!page_ok(page) || !cache_dim_ok(dim) || !cache_type_ok(type) || heads < 1 || heads > kAttnMaxHeads)
        return 0;
    return (size_t)kv_cache(nullptr, 1, page, heads, dim, type).page_bytes;
}

qg_status qhead_norm_rope(const void *q, int64_t ldq, int q_heads, const void *k, int64_t ldk, int k_heads, int x_type,
                          const void *q_gain, const void *k_gain, int gain_type, float eps, const int32_t *positions,
                          int axes, const int32_t *sections, const float *freq, int rot, int interleaved, int64_t T,
                          int D, void *yq, int64_t ldyq, void *yk, int64_t ldyk, int y_type, void *stream)
{
    HeadArgs a;
    const qg_status st = check_heads(a, q, ldq, q_heads, k, ldk, k_heads, x_type, q_gain, k_gain, gain_type, eps,
                                     positions, axes, sections, freq, rot, interleaved, T, D);
    if (st != QG_OK)
        return st;
    if (!yq || (k_heads && !yk))
        return QG_ERR_NULL;
    if (!type_ok(y_type) || !rows_ok(ldyq, q_heads, D, T) || (k_heads && !rows_ok(ldyk, k_heads, D, T)))
        return QG_ERR_SHAPE;
    if (!aligned(yq, type_bytes(y_type)) || !aligned(yk, type_bytes(y_type)))
        return QG_ERR_ALIGN;
    a.y[0] = yq, a.y[1] = yk;
    a.ldy[0] = ldyq, a.ldy[1] = ldyk;
    a.y_type = y_type;
    return status(launch_head_norm_rope(a, x_type, on(stream)));
}

size_t qhead_norm_rope_backward_workspace(int64_t T, int q_heads, int k_heads, int D, int gains)
{
    if (!gains || !tokens_ok(T) || q_heads < 1 || k_heads < 0 || q_heads > kAttnMaxHeads ||
        k_heads > kAttnMaxHeads - q_heads || D < 8 || D > 256 || D % 8)
        return 0;
    return head_backward_workspace(T, q_heads, k_heads, D);
}

qg_status qhead_norm_rope_backward(const void *gyq, int64_t ldgq, const void *gyk, int64_t ldgk, int y_type,
                                   const void *q, int64_t ldq, int q_heads, const void *k, int64_t ldk, int k_heads,
                                   int x_type, const void *q_gain, const void *k_gain, int gain_type, float eps,
                                   const int32_t *positions, int axes, const int32_t *sections, const float *freq,
                                   int rot, int interleaved, int64_t T, int D, void *gq, int64_t lddq, void *gk,
                                   int64_t lddk, float *g_gain, void *workspace, void *stream)
{
    HeadGradArgs g{};
    const qg_status st = check_heads(g.h, q, ldq, q_heads, k, ldk, k_heads, x_type, q_gain, k_gain, gain_type, eps,
                                     positions, axes, sections, freq, rot, interleaved, T, D);
    if (st != QG_OK)
        return st;
    if (!gyq || !gq || (k_heads && (!gyk || !gk)) || (q_gain && (!g_gain || !workspace)))
        return QG_ERR_NULL;
    if (!type_ok(y_type) || !rows_ok(ldgq, q_heads, D, T) || !rows_ok(lddq, q_heads, D, T) ||
        (k_heads && (!rows_ok(ldgk, k_heads, D, T) || !rows_ok(lddk, k_heads, D, T))))
        return QG_ERR_SHAPE;
    if (!aligned(gyq, type_bytes(y_type)) || !aligned(gyk, type_bytes(y_type)) || !aligned(gq, type_bytes(x_type)) ||
        !aligned(gk, type_bytes(x_type)) || !aligned(g_gain, 4) || !aligned(workspace, 16))
        return QG_ERR_ALIGN;
    g.h.y[0] = const_cast<void *>(gyq), g.h.y[1] = const_cast<void *>(gyk);
    g.h.ldy[0] = ldgq, g.h.ldy[1] = ldgk;
    g.h.y_type = y_type;
    g.g[0] = gq, g.g[1] = gk;
    g.ldg[0] = lddq, g.ldg[1] = lddk;
    g.g_gain = g_gain;
    g.workspace = static_cast<float *>(workspace);
    return status(launch_head_norm_rope_backward(g, x_type, on(stream)));
}

qg_status qkv_write(const void *k, int64_t ldk, const void *v, int64_t ldv, int x_type, const int32_t *slots,
                    int64_t T, void *cache, int64_t pages, int page, int heads, int dim, int cache_type, void *stream)
{
    if (!k || !v || !slots)
        return QG_ERR_NULL;
    const qg_status st = check_cache(cache, pages, page, heads, dim, cache_type);
    if (st != QG_OK)
        return st;
    if (!type_ok(x_type) || !tokens_ok(T) || !qg::rows_ok(ldk, heads, dim, T) || !qg::rows_ok(ldv, heads, dim, T))
        return QG_ERR_SHAPE;
    if (!aligned(k, type_bytes(x_type)) || !aligned(v, type_bytes(x_type)) || !aligned(slots, 4))
        return QG_ERR_ALIGN;
    const KvArgs a{k, v, ldk, ldv, nullptr, nullptr, slots, T, kv_cache(cache, pages, page, heads, dim, cache_type)};
    return status(launch_kv_write(a, x_type, on(stream)));
}

qg_status qkv_read(const void *cache, int64_t pages, int page, int heads, int dim, int cache_type,
                   const int32_t *slots, int64_t T, void *k, void *v, int y_type, void *stream)
{
    if (!k || !v || !slots)
        return QG_ERR_NULL;
    const qg_status st = check_cache(cache, pages, page, heads, dim, cache_type);
    if (st != QG_OK)
        return st;
    if (!type_ok(y_type) || !tokens_ok(T))
        return QG_ERR_SHAPE;
    if (!aligned(k, type_bytes(y_type)) || !aligned(v, type_bytes(y_type)) || !aligned(slots, 4))
        return QG_ERR_ALIGN;
    const KvArgs a{nullptr, nullptr, 0, 0, k, v, slots, T,
                   kv_cache(const_cast<void *>(cache), pages, page, heads, dim, cache_type)};
    return status(launch_kv_read(a, y_type, on(stream)));
}

qg_status qkv_norm_rope_write(const void *q, int64_t ldq, int q_heads, const void *k, int64_t ldk, const void *v,
                              int64_t ldv, int x_type, const void *q_gain, const void *k_gain, int gain_type,
                              float eps, const int32_t *positions, int axes, const int32_t *sections,
                              const float *freq, int rot, int interleaved, int64_t T, const int32_t *slots, void *yq,
                              int64_t ldyq, int y_type, void *cache, int64_t pages, int page, int heads, int dim,
                              int cache_type, void *stream)
{
    if (!v || !slots || !yq)
        return QG_ERR_NULL;
    qg_status st = check_cache(cache, pages, page, heads, dim, cache_type);
    if (st != QG_OK)
        return st;
    HeadArgs a;
    st = check_heads(a, q, ldq, q_heads, k, ldk, heads, x_type, q_gain, k_gain, gain_type, eps, positions, axes,
                     sections, freq, rot, interleaved, T, dim);
    if (st != QG_OK)
        return st;
    if (!type_ok(y_type) || !qg::rows_ok(ldv, heads, dim, T) || !qg::rows_ok(ldyq, q_heads, dim, T))
        return QG_ERR_SHAPE;
    if (!aligned(v, type_bytes(x_type)) || !aligned(slots, 4) || !aligned(yq, type_bytes(y_type)))
        return QG_ERR_ALIGN;
    a.x[2] = v;
    a.ldx[2] = ldv;
    a.heads[2] = heads;
    a.y[0] = yq;
    a.ldy[0] = ldyq;
    a.y_type = y_type;
    a.slots = slots;
    a.cache = kv_cache(cache, pages, page, heads, dim, cache_type);
    return status(launch_head_norm_rope_write(a, x_type, on(stream)));
}

size_t qattn_decode_workspace(int64_t B, int M, int q_heads, int kv_heads, int dim, int cache_type, int page,
                              int64_t width)
{
    if (!page_ok(page) || !cache_dim_ok(dim) || !cache_type_ok(cache_type) ||
        !batch_ok(B, M, q_heads, kv_heads, page, width))
        return 0;
    return attend_workspace(B, M, q_heads, kv_heads, dim, cache_type, page, width);
}

qg_status qattn_decode(const void *cache, int64_t pages, int page, int kv_heads, int dim, int cache_type,
                       const void *q, int q_type, int64_t ldq, int64_t B, int M, int q_heads, const int32_t *table,
                       int64_t width, const int32_t *lens, float scale, int64_t window, float softcap, void *out,
                       void *workspace, void *stream)
{
    if (!q || !table || !lens || !out)
        return QG_ERR_NULL;
    const qg_status st = check_cache(cache, pages, page, kv_heads, dim, cache_type);
    if (st != QG_OK)
        return st;
    if ((q_type != QG_F16 && q_type != QG_BF16) || (cache_type != QG_F8 && cache_type != q_type) ||
        !batch_ok(B, M, q_heads, kv_heads, page, width) || !qg::rows_ok(ldq, q_heads, dim, B * M) || window < 0 ||
        window > INT32_MAX || !std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.0f ||
        (softcap > 0.0f && !std::isfinite(scale / softcap)))
        return QG_ERR_SHAPE;
    if (!workspace && attend_workspace(B, M, q_heads, kv_heads, dim, cache_type, page, width) > 0)
        return QG_ERR_NULL;
    if (!aligned(q, 2) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(out, 2) || !aligned(workspace, 16))
        return QG_ERR_ALIGN;
    const AttendArgs a{kv_cache(const_cast<void *>(cache), pages, page, kv_heads, dim, cache_type),
                       q, ldq, (int)B, M, q_heads, q_heads / kv_heads, table, (int)width, lens, scale,
                       window >= kAttnMaxPlaces ? 0 : (int)window,
                       softcap, out, workspace};
    return status(launch_attend(a, q_type, on(stream)));
}

}  // extern "C"
