// f8 conversions (formats in qgemv_f8.h): activations to packed f8 and back,
// packed weights to fp32 / fp16 and to the packed transposed matrix.
//
// All of them are bound by memory: sixteen values (one 16-byte word of codes) a
// lane.  Activations: each byte read and written once, one store of the codes
// and two or four loads.  8192 x 4096 in bf16: 17 us to quantize, 17 back, 101 MB
// each, 5.9 TB/s (a copy of a gigabyte runs at 5.2; part of the data is still in
// the last-level cache).  Transposed weights: 28672 x 4096 43 us, 5.5 TB/s; 4096
// x 4096 9.5, 3.5 TB/s.  Weights back to fp32 or fp16 run at 2.5 to 3.4 TB/s
// (28672 x 4096 190 and 142 us, 4096 x 4096 26 and 15): whole lines are written,
// but read in pieces of 16 bytes, 256 apart.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "qgemv_f8_internal.h"

namespace qg {
namespace {

template <typename T, int N>
__device__ __forceinline__ void store_row(T *p, int left, const float (&v)[N])
{
    if (left >= N) {
        constexpr int kPer = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < N / kPer; ++i) {
            Raw16 r;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4)
                    r.w[j] = __float_as_uint(v[i * kPer + j]);
                else
                    r.w[j] = pack2<T>(v[i * kPer + 2 * j], v[i * kPer + 2 * j + 1]);
            }
            *reinterpret_cast<Raw16 *>(p + i * kPer) = r;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left)
                p[i] = from_f32<T>(v[i]);
    }
}

__device__ __forceinline__ void widen16(const uint4 &c, float scale, float (&v)[16])
{
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        typedef float f2 __attribute__((ext_vector_type(2)));
        const f2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
        const f2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        v[4 * i] = a[0] * scale, v[4 * i + 1] = a[1] * scale;
        v[4 * i + 2] = b[0] * scale, v[4 * i + 3] = b[1] * scale;
    }
}

struct ActArgs {
    const void *x;
    uint8_t *xq;
    void *out;
    int64_t ldx, scales;
    uint32_t blocks;   // (row, block of 128) pairs of this launch, < 2^31
    int K, cb, ls;
    int64_t row0;      // first row of the launch
};

// Eight lanes a block: each holds 16 elements, the block's largest magnitude
// comes from three cross-lane steps, every lane then writes its 16 codes.
template <typename T>
__global__ __launch_bounds__(256) void act_quantize_kernel(ActArgs a)
{
    const uint32_t g = (uint32_t)blockIdx.x * 32 + threadIdx.x / 8;
    const int part = threadIdx.x & 7;
    if (g >= a.blocks)
        return;   // whole groups of eight lanes leave together
    const int64_t m = a.row0 + g / (uint32_t)a.cb;
    const int c = (int)(g % (uint32_t)a.cb);
    const int k = c * 128 + part * 16;
    float v[16];
    load_row(static_cast<const T *>(a.x) + m * a.ldx + k, a.K - k, v);
    uint32_t w[4];
    const uint32_t byte = f8_quantize16(v, w);
    *reinterpret_cast<uint4 *>(a.xq + (m * a.cb + c) * 128 + part * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    if (part == 0)
        a.xq[a.scales + m * a.ls + c] = (uint8_t)byte;
}

template <typename T>
__global__ __launch_bounds__(256) void act_dequant_kernel(ActArgs a)
{
    const uint32_t g = (uint32_t)blockIdx.x * 32 + threadIdx.x / 8;
    const int part = threadIdx.x & 7;
    if (g >= a.blocks)
        return;
    const int64_t m = a.row0 + g / (uint32_t)a.cb;
    const int c = (int)(g % (uint32_t)a.cb);
    const int k = c * 128 + part * 16;
    if (k >= a.K)
        return;
    float v[16];
    widen16(*reinterpret_cast<const uint4 *>(a.xq + (m * a.cb + c) * 128 + part * 16),
            f8_scale(a.xq[a.scales + m * a.ls + c]), v);
    store_row(static_cast<T *>(a.out) + m * a.K + k, a.K - k, v);
}

// Rows are launched in portions of at most 2^28 blocks (a grid holds fewer than
// 2^32 threads).
template <typename L>
hipError_t by_rows(int64_t M, ActArgs a, L launch)
{
    const int64_t most = std::max<int64_t>(1, ((int64_t)1 << 28) / a.cb);
    for (int64_t m = 0; m < M; m += most) {
        a.row0 = m;
        a.blocks = (uint32_t)(std::min(most, M - m) * a.cb);
        const hipError_t e = launch(dim3((a.blocks + 31) / 32), a);
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

struct WeightArgs {
    const uint8_t *W;
    void *out;
    uint8_t *WT;
    int64_t scales, scales_t;
    int64_t bytes_t;
    int N, K, cb, ls, rt;
    int cb_t, ls_t, rt_t;
};

// A workgroup per row tile and 16 columns per lane, neighbouring lanes on
// neighbouring columns of a row.
template <typename T>
__global__ __launch_bounds__(256) void f8_dequant_kernel(WeightArgs a)
{
    for (int t = blockIdx.x; t < a.rt; t += gridDim.x) {
        for (int i = threadIdx.x; i < 16 * 8 * a.cb; i += 256) {
            const int r = i / (8 * a.cb), ch = i % (8 * a.cb);
            const int n = 16 * t + r, k = 16 * ch;
            if (n >= a.N || k >= a.K)
                continue;
            float v[16];
            widen16(*reinterpret_cast<const uint4 *>(a.W + ((int64_t)t * a.cb + ch / 8) * 2048 + 256 * (ch & 7) +
                                                     16 * r),
                    f8_scale(a.W[a.scales + (int64_t)(n >> 7) * a.ls + (ch >> 3)]), v);
            store_row(static_cast<T *>(a.out) + (int64_t)n * a.K + k, a.K - k, v);
        }
    }
}

// A 128 x 128 block per workgroup.  In both matrices it is 8 x 8 pieces of 16
// x 16 codes, 256 contiguous bytes each: piece (row tile i, column group j)
// of the source is, transposed, piece (j, i) of the result.  Row tiles past
// the source's last are zeros (padding columns of the result).
__global__ __launch_bounds__(256) void f8_transpose_kernel(WeightArgs a)
{
    __shared__ uint8_t s[64][16][16 + 4];   // a pad of one bank against the column reads
    const int c = blockIdx.x, b = blockIdx.y;
    for (int i = threadIdx.x; i < 1024; i += 256) {
        const int tile = i >> 7, in = i & 127;   // 128 words of 16 bytes a tile
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (8 * b + tile < a.rt)
            v = *reinterpret_cast<const uint4 *>(a.W + ((int64_t)(8 * b + tile) * a.cb + c) * 2048 + in * 16);
        uint32_t *d = reinterpret_cast<uint32_t *>(&s[tile * 8 + (in >> 4)][in & 15][0]);
        d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 1024; i += 256) {
        const int tile = i >> 7, in = i & 127;   // of the result: 16 source columns, 8 groups of 16 source rows
        if (8 * c + tile >= a.rt_t)
            continue;
        const int group = in >> 4, k = in & 15;
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            w[q] = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[q] |= (uint32_t)s[group * 8 + tile][4 * q + e][k] << (8 * e);
        }
        *reinterpret_cast<uint4 *>(a.WT + ((int64_t)(8 * c + tile) * a.cb_t + b) * 2048 + in * 16) =
            make_uint4(w[0], w[1], w[2], w[3]);
    }
    // one scale; the last block of a row also pads it, the very last the matrix
    uint8_t *st = a.WT + a.scales_t + (int64_t)c * a.ls_t;
    if (threadIdx.x == 0)
        st[b] = a.W[a.scales + (int64_t)b * a.ls + c];
    if (b == (int)gridDim.y - 1) {
        for (int i = b + 1 + threadIdx.x; i < a.ls_t; i += 256)
            st[i] = 0;
        if (c == (int)gridDim.x - 1)
            for (int64_t i = a.scales_t + (int64_t)(c + 1) * a.ls_t + threadIdx.x; i < a.bytes_t; i += 256)
                a.WT[i] = 0;
    }
}

template <typename P>
hipError_t go(void (*fn)(P), dim3 grid, const P &a, hipStream_t stream)
{
    return launch_kernel(reinterpret_cast<const void *>(fn), grid, dim3(256), 0, stream, a);
}

}  // namespace

hipError_t launch_act_quantize(const void *x, int type, int64_t ldx, int64_t M, int64_t K, uint8_t *xq,
                               hipStream_t stream)
{
    const F8Acts f = f8_acts(M, K);
    ActArgs a{x, xq, nullptr, ldx, f.scales, 0, (int)K, f.cb, f.ls, 0};
    return by_rows(M, a, [&](dim3 grid, const ActArgs &p) {
        return type == QG_F32   ? go(&act_quantize_kernel<float>, grid, p, stream)
               : type == QG_F16 ? go(&act_quantize_kernel<Fp16>, grid, p, stream)
                                : go(&act_quantize_kernel<Bf16>, grid, p, stream);
    });
}

hipError_t launch_act_dequant(const uint8_t *xq, int64_t M, int64_t K, int type, void *out, hipStream_t stream)
{
    const F8Acts f = f8_acts(M, K);
    ActArgs a{nullptr, const_cast<uint8_t *>(xq), out, 0, f.scales, 0, (int)K, f.cb, f.ls, 0};
    return by_rows(M, a, [&](dim3 grid, const ActArgs &p) {
        return type == QG_F32   ? go(&act_dequant_kernel<float>, grid, p, stream)
               : type == QG_F16 ? go(&act_dequant_kernel<Fp16>, grid, p, stream)
                                : go(&act_dequant_kernel<Bf16>, grid, p, stream);
    });
}

namespace {

WeightArgs weight_args(const uint8_t *W, int64_t N, int64_t K)
{
    const F8Weights f = f8_weights(N, K), t = f8_weights(K, N);
    return WeightArgs{W, nullptr, nullptr, f.scales, t.scales, t.bytes, (int)N, (int)K, f.cb, f.ls, f.rt,
                      t.cb, t.ls, t.rt};
}

}  // namespace

hipError_t launch_f8_dequant(const uint8_t *W, int64_t N, int64_t K, bool fp16, void *out, hipStream_t stream)
{
    WeightArgs a = weight_args(W, N, K);
    a.out = out;
    return go(fp16 ? &f8_dequant_kernel<Fp16> : &f8_dequant_kernel<float>, dim3((unsigned)std::min(a.rt, 1 << 22)), a, stream);
}

hipError_t launch_f8_transpose(const uint8_t *W, int64_t N, int64_t K, uint8_t *WT, hipStream_t stream)
{
    WeightArgs a = weight_args(W, N, K);
    a.WT = WT;
    return go(&f8_transpose_kernel, dim3(a.cb, (unsigned)ceil_div(N, 128)), a, stream);
}

}  // namespace qg
