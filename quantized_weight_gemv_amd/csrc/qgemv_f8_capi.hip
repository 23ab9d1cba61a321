// C-ABI entry points of qgemv_f8.h: host-side validation, then launches on
// the caller's stream.  Nothing here allocates device memory or synchronizes.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "qgemv_f8.h"
#include "qgemv_f8_internal.h"

namespace qg {
namespace {

// Rows of X of an expert call are gathered with 32-bit offsets.
constexpr int64_t kF8MaxMoeBlocks = ((int64_t)1 << 25) - 2;

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline qg_status status(hipError_t e) { return e == hipSuccess ? QG_OK : QG_ERR_LAUNCH; }

inline bool rows_ok(int64_t n) { return n >= 1 && n <= kF8MaxRows; }
inline bool k_ok(int64_t k) { return k >= 1 && k <= kF8MaxK; }

inline hipStream_t on(void *stream) { return static_cast<hipStream_t>(stream); }

// Slots of an expert call.
qg_status check_slots(int64_t P, int64_t T, int k_slots, const int32_t *order, const int32_t *offsets)
{
    if (!order || !offsets)
        return QG_ERR_NULL;
    if (P < 1 || P > kMaxExperts || !rows_ok(T) || k_slots < 1 || k_slots > kMaxTopK || T * k_slots > kF8MaxRows)
        return QG_ERR_SHAPE;
    if (!aligned(order, 4) || !aligned(offsets, 4))
        return QG_ERR_ALIGN;
    return QG_OK;
}

qg_status check_route(const void *logits, int type, int64_t ldl, int64_t T, int64_t E, int k, const void *idx,
                      const void *weight, const void *counts)
{
    if (!logits || !idx || !weight || !counts)
        return QG_ERR_NULL;
    if (!type_ok(type) || T < 1 || T > kRouteMaxTokens || E < 1 || E > kMaxExperts || ldl < E || ldl > INT64_MAX / 4 / T ||
        k < 1 || k > E || k > kMaxTopK)
        return QG_ERR_SHAPE;
    if (!aligned(logits, type_bytes(type)) || !aligned(idx, 4) || !aligned(weight, 4) || !aligned(counts, 4))
        return QG_ERR_ALIGN;
    return QG_OK;
}

// Few rows: the streaming kernels, bound by W's way to every compute unit, or
// the tiled ones, whose time is one tile's as long as tiles are few.  Measured
// (us, streaming / tiled, bf16 out; fp32 out the same within a microsecond),
// K 4096: M 32: N 8192 11 / 20, 12288 16 / 20, 22016 29 / 21, 28672 35 / 23;
// M 64: 4096 9 / 18, 8192 19 / 20, 12288 28 / 20, 28672 62 / 24.  K 1024: M 32:
// 12288 5.2 / 7.7, 22016 8.1 / 7.9, 28672 9.6 / 7.9; M 64: 8192 6.8 / 7.5, 12288
// 8.9 / 7.7.  M 16: 28672 x 4096 28 / 23, the largest difference of up to 16
// rows.  fp32 outputs of up to 32 rows always stream: their bits are then the
// same in any split of the rows of W.
bool few_rows(int64_t M, int64_t N, int y_type, int cus)
{
    const int64_t tiles = ceil_div(N, 128);
    return M <= 16 || (M <= 32 && (y_type == QG_F32 || tiles < cus / 2)) || (M <= 64 && tiles < cus / 4);
}

// The same for experts, by their average slots.  Measured (us, streaming /
// tiled), 64 experts of 2048 x 2048, bf16 out: 8 slots each 60 / 66, 16 86 /
// 64, 24 108 / 67; fp32: 58 / 67, 83 / 69, 107 / 70.  128 experts of 640 x 2560,
// bf16: 8 47 / 49, 16 66 / 50; fp32: 45 / 50, 65 / 51.
bool few_slots(int64_t slots, int64_t P) { return slots <= 8 * P; }

}  // namespace
}  // namespace qg

using namespace qg;

extern "C" {

qg_status qdequant_f8(const void *Wp, int64_t N, int64_t K, int out_fp16, void *out, void *stream)
{
    if (!Wp || !out)
        return QG_ERR_NULL;
    if (!rows_ok(N) || !k_ok(K))
        return QG_ERR_SHAPE;
    if (!aligned(Wp, 256) || !aligned(out, out_fp16 ? 2 : 4))
        return QG_ERR_ALIGN;
    return status(launch_f8_dequant(static_cast<const uint8_t *>(Wp), N, K, out_fp16 != 0, out, on(stream)));
}

qg_status qtranspose_f8(const void *Wp, int64_t N, int64_t K, void *WpT, void *stream)
{
    if (!Wp || !WpT)
        return QG_ERR_NULL;
    if (!k_ok(N) || !k_ok(K))
        return QG_ERR_SHAPE;
    if (!aligned(Wp, 256) || !aligned(WpT, 256))
        return QG_ERR_ALIGN;
    return status(launch_f8_transpose(static_cast<const uint8_t *>(Wp), N, K, static_cast<uint8_t *>(WpT),
                                      on(stream)));
}

qg_status qact_quantize_f8(const void *x, int x_type, int64_t ldx, int64_t M, int64_t K, void *xq, void *stream)
{
    if (!x || !xq)
        return QG_ERR_NULL;
    if (!type_ok(x_type) || !rows_ok(M) || !k_ok(K) || ldx < K || ldx > INT64_MAX / 4 / M)
        return QG_ERR_SHAPE;
    if (!aligned(x, type_bytes(x_type)) || !aligned(xq, 256))
        return QG_ERR_ALIGN;
    return status(launch_act_quantize(x, x_type, ldx, M, K, static_cast<uint8_t *>(xq), on(stream)));
}

qg_status qact_dequant_f8(const void *xq, int64_t M, int64_t K, int out_type, void *out, void *stream)
{
    if (!xq || !out)
        return QG_ERR_NULL;
    if (!type_ok(out_type) || !rows_ok(M) || !k_ok(K))
        return QG_ERR_SHAPE;
    if (!aligned(xq, 256) || !aligned(out, type_bytes(out_type)))
        return QG_ERR_ALIGN;
    return status(launch_act_dequant(static_cast<const uint8_t *>(xq), M, K, out_type, out, on(stream)));
}

qg_status qgemv_f8(const void *Wp, const void *x, int x_type, float *y, int M, int64_t N, int64_t K, void *stream)
{
    if (!Wp || !x || !y)
        return QG_ERR_NULL;
    if (!type_ok(x_type) || M < 1 || M > 8 || !rows_ok(N) || !k_ok(K) || K > kF8MaxGemvK)
        return QG_ERR_SHAPE;
    if (!aligned(Wp, 256) || !aligned(x, type_bytes(x_type)) || !aligned(y, 4))
        return QG_ERR_ALIGN;
    const int cus = device_cus();
    if (cus <= 0)
        return QG_ERR_DEVICE;
    const F8Rows r{M, M, nullptr, nullptr, 0, 1, 0};
    return status(launch_f8_skinny(static_cast<const uint8_t *>(Wp), nullptr, x, x_type, y, QG_F32, r, N, K, cus,
                                   on(stream)));
}

qg_status qgemm_f8(const void *Wp, const void *xq, void *Y, int y_type, int64_t M, int64_t N, int64_t K, void *stream)
{
    if (!Wp || !xq || !Y)
        return QG_ERR_NULL;
    if (!type_ok(y_type) || !rows_ok(M) || !rows_ok(N) || !k_ok(K))
        return QG_ERR_SHAPE;
    if (!aligned(Wp, 256) || !aligned(xq, 256) || !aligned(Y, type_bytes(y_type)))
        return QG_ERR_ALIGN;
    const int cus = device_cus();
    if (cus <= 0)
        return QG_ERR_DEVICE;
    const F8Rows r{M, M, nullptr, nullptr, 0, 1, 0};
    const auto *W = static_cast<const uint8_t *>(Wp);
    const auto *X = static_cast<const uint8_t *>(xq);
    if (few_rows(M, N, y_type, cus))
        return status(launch_f8_skinny(W, X, nullptr, 0, Y, y_type, r, N, K, cus, on(stream)));
    return status(launch_f8_gemm(W, X, Y, y_type, r, N, K, cus, on(stream)));
}

size_t qgemm_f8_wgrad_workspace(int64_t M, int64_t N, int64_t K)
{
    return rows_ok(M) && k_ok(N) && k_ok(K) ? f8_wgrad_workspace(M, N, K) : 0;
}

qg_status qgemm_f8_wgrad(const void *dY, const void *xq, float *dW, int accumulate, int64_t M, int64_t N, int64_t K,
                         void *workspace, void *stream)
{
    if (!dY || !xq || !dW)
        return QG_ERR_NULL;
    if (!rows_ok(M) || !k_ok(N) || !k_ok(K))
        return QG_ERR_SHAPE;
    if (!workspace && f8_wgrad_workspace(M, N, K) > 0)
        return QG_ERR_NULL;
    if (!aligned(dY, 2) || !aligned(xq, 256) || !aligned(dW, 4) || !aligned(workspace, 16))
        return QG_ERR_ALIGN;
    const F8Rows r{M, M, nullptr, nullptr, 0, 1, 0};
    return status(launch_f8_wgrad(static_cast<const uint16_t *>(dY), static_cast<const uint8_t *>(xq), dW,
                                  accumulate != 0, r, N, K, static_cast<float *>(workspace), on(stream)));
}

size_t qmoe_route_workspace(int64_t T, int64_t E)
{
    return T >= 1 && T <= kRouteMaxTokens && E >= 1 && E <= kMaxExperts ? route_workspace(T, E) : 0;
}

qg_status qmoe_route(const void *logits, int type, int64_t ldl, const uint8_t *token_mask, int64_t T, int64_t E,
                     int k, int renormalize, int32_t *idx, float *weight, int32_t *counts, int32_t *offsets,
                     int32_t *order, float *loss, void *workspace, void *stream)
{
    const qg_status st = check_route(logits, type, ldl, T, E, k, idx, weight, counts);
    if (st != QG_OK)
        return st;
    if (!offsets || !order || !loss || (!workspace && route_workspace(T, E) > 0))
        return QG_ERR_NULL;
    if (!aligned(offsets, 4) || !aligned(order, 4) || !aligned(loss, 4) || !aligned(workspace, 16))
        return QG_ERR_ALIGN;
    const RouteArgs a{logits, type, ldl, token_mask, T, (int)E, k, renormalize != 0, idx, weight, counts, offsets,
                      order, loss, workspace, false};
    return status(launch_route(a, on(stream)));
}

qg_status qmoe_route_backward(const void *logits, int type, int64_t ldl, const uint8_t *token_mask, int64_t T,
                              int64_t E, int k, int renormalize, const int32_t *idx, const float *weight,
                              const int32_t *counts, const float *grad_weight, const float *grad_loss,
                              void *dlogits, void *stream)
{
    const qg_status st = check_route(logits, type, ldl, T, E, k, idx, weight, counts);
    if (st != QG_OK)
        return st;
    if (!dlogits)
        return QG_ERR_NULL;
    if (!aligned(grad_weight, 4) || !aligned(grad_loss, 4) || !aligned(dlogits, type_bytes(type)))
        return QG_ERR_ALIGN;
    const int cus = device_cus();
    if (cus <= 0)
        return QG_ERR_DEVICE;
    const RouteGradArgs a{logits, type, ldl, token_mask, T, (int)E, k, renormalize != 0, idx, weight, counts,
                          grad_weight, grad_loss, dlogits, false, false};
    return status(launch_route_backward(a, cus, on(stream)));
}

qg_status qmoe_gemm_f8(const void *pool, int64_t P, const void *xq, int64_t T, int k_slots, const int32_t *order,
                       const int32_t *offsets, void *Y, int y_type, int64_t N, int64_t K, void *stream)
{
    if (!pool || !xq || !Y)
        return QG_ERR_NULL;
    const qg_status st = check_slots(P, T, k_slots, order, offsets);
    if (st != QG_OK)
        return st;
    if (!type_ok(y_type) || !rows_ok(N) || !k_ok(K) || T * ceil_div(K, 128) > kF8MaxMoeBlocks)
        return QG_ERR_SHAPE;
    if (!aligned(pool, 256) || !aligned(xq, 256) || !aligned(Y, type_bytes(y_type)))
        return QG_ERR_ALIGN;
    const int cus = device_cus();
    if (cus <= 0)
        return QG_ERR_DEVICE;
    const F8Rows r{T * k_slots, T, order, offsets, (int)P, k_slots, f8_weights(N, K).bytes};
    const auto *W = static_cast<const uint8_t *>(pool);
    const auto *X = static_cast<const uint8_t *>(xq);
    if (few_slots(r.rows, P))
        return status(launch_f8_skinny(W, X, nullptr, 0, Y, y_type, r, N, K, cus, on(stream)));
    return status(launch_f8_gemm(W, X, Y, y_type, r, N, K, cus, on(stream)));
}

qg_status qmoe_gemm_f8_wgrad(const void *dY, const void *xq, int64_t T, int k_slots, const int32_t *order,
                             const int32_t *offsets, int64_t P, float *dW, int accumulate, int64_t N, int64_t K,
                             void *stream)
{
    if (!dY || !xq || !dW)
        return QG_ERR_NULL;
    const qg_status st = check_slots(P, T, k_slots, order, offsets);
    if (st != QG_OK)
        return st;
    if (!k_ok(N) || !k_ok(K))
        return QG_ERR_SHAPE;
    if (!aligned(dY, 2) || !aligned(xq, 256) || !aligned(dW, 4))
        return QG_ERR_ALIGN;
    const F8Rows r{T * k_slots, T, order, offsets, (int)P, k_slots, 0};
    return status(launch_f8_wgrad(static_cast<const uint16_t *>(dY), static_cast<const uint8_t *>(xq), dW,
                                  accumulate != 0, r, N, K, nullptr, on(stream)));
}

}  // extern "C"
