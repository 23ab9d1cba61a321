// Attention of new tokens over the paged cache (definitions in qgemv_attn.h).
//
// A workgroup per query head of a token: its four waves take every fourth
// token of the cache, 64 lanes hold a vector, one pass with the running
// maximum and sum of the softmax, the waves joined at the end.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "qgemv_attn_internal.h"

namespace qg {
namespace {

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / 64;

template <typename T>
__device__ __forceinline__ float element(const uint8_t *row, int i)
{
    return to_f32(reinterpret_cast<const T *>(row)[i]);
}

struct F8Code {
    uint8_t u;
};
template <>
__device__ __forceinline__ float element<F8Code>(const uint8_t *row, int i)
{
    return __builtin_amdgcn_cvt_f32_fp8((int)row[i], 0);
}

__device__ __forceinline__ float wave_sum(float v)
{
    v = group_sum<32>(v);
    const f2_t p = pair32(v);
    return p[0] + p[1];
}

template <typename TQ, typename TC, int D>
__global__ __launch_bounds__(kBlock) void attend_kernel(AttendArgs a)
{
    constexpr int kPer = D / 64;
    constexpr bool kF8 = sizeof(TC) == 1;
    __shared__ float o[kWaves][D], ml[kWaves][2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x;   // (b M + i) q_heads + query head
    const int qh = (int)(row % a.q_heads);
    const int64_t token = row / a.q_heads;
    const int b = (int)(token / a.M), i = (int)(token % a.M), head = qh / a.share;
    const int64_t most = (int64_t)a.width * a.cache.page;
    const int len = (int)min((int64_t)max(a.lens[b], 0), most);
    const int end = len - a.M + i + 1;
    const int begin = a.window ? max(0, end - a.window) : 0;
    float q[kPer], acc[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        q[j] = to_f32(static_cast<const TQ *>(a.q)[token * a.ldq + (int64_t)qh * D + lane * kPer + j]);
        acc[j] = 0.0f;
    }
    float m = -__builtin_inff(), l = 0.0f;
    for (int t = begin + wave; t < end; t += kWaves) {
        const int page = a.table[(int64_t)b * a.width + (t >> a.cache.log_page)];
        if ((uint32_t)page >= (uint32_t)a.cache.pages)
            continue;
        const uint8_t *base = a.cache.data + (int64_t)page * a.cache.page_bytes;
        const int at = head * 2 * a.cache.page + (t & (a.cache.page - 1));
        const uint8_t *k = base + (int64_t)at * D * sizeof(TC), *v = k + (int64_t)a.cache.page * D * sizeof(TC);
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            s += q[j] * element<TC>(k, lane * kPer + j);
        s = wave_sum(s);
        float vs = 1.0f;
        if constexpr (kF8) {
            s *= f8_scale(base[a.cache.scales + at]);
            vs = f8_scale(base[a.cache.scales + at + a.cache.page]);
        }
        s *= a.scale;
        if (a.softcap > 0.0f)
            s = a.softcap * tanhf(s / a.softcap);
        if (s == -__builtin_inff())
            continue;
        const float to = fmaxf(m, s);
        const float old = expf(m - to), p = expf(s - to);
        l = l * old + p;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            acc[j] = acc[j] * old + p * (element<TC>(v, lane * kPer + j) * vs);
        m = to;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j)
        o[wave][lane * kPer + j] = acc[j];
    if (lane == 0)
        ml[wave][0] = m, ml[wave][1] = l;
    __syncthreads();
    float top = -__builtin_inff(), sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w)
        top = fmaxf(top, ml[w][0]);
    const float from = top == -__builtin_inff() ? 0.0f : top;
    float weight[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        weight[w] = expf(ml[w][0] - from);
        sum += ml[w][1] * weight[w];
    }
    for (int d = threadIdx.x; d < D; d += kBlock) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            v += o[w][d] * weight[w];
        static_cast<TQ *>(a.out)[row * D + d] = from_f32<TQ>(sum == 0.0f ? 0.0f : v / sum);
    }
}

template <typename TQ, typename TC>
hipError_t of_dim(const AttendArgs &a, hipStream_t stream)
{
    void (*fn)(AttendArgs) = a.cache.dim == 64    ? &attend_kernel<TQ, TC, 64>
                             : a.cache.dim == 128 ? &attend_kernel<TQ, TC, 128>
                             : a.cache.dim == 192 ? &attend_kernel<TQ, TC, 192>
                                                  : &attend_kernel<TQ, TC, 256>;
    return launch_kernel(reinterpret_cast<const void *>(fn), dim3((unsigned)(a.B * a.M * a.q_heads)), dim3(kBlock), 0,
                         stream, a);
}

}  // namespace

size_t attend_workspace(int64_t, int, int, int, int, int, int64_t) { return 0; }

hipError_t launch_attend(const AttendArgs &a, int q_type, hipStream_t stream)
{
    if (a.cache.type == QG_F8)
        return q_type == QG_F16 ? of_dim<Fp16, F8Code>(a, stream) : of_dim<Bf16, F8Code>(a, stream);
    return q_type == QG_F16 ? of_dim<Fp16, Fp16>(a, stream) : of_dim<Bf16, Bf16>(a, stream);
}

}  // namespace qg
