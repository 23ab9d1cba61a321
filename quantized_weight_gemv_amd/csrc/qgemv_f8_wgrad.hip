// Weight gradients from 8-bit checkpoints: dW[n][k] = sum_m dY[m][n] X[m][k],
// dY in bf16, X packed f8 activations; for one matrix or for each expert of a
// pool.
//
// The summed index m is the slow one of both operands, and the block scales
// of X change along it, so the 8-bit instructions cannot take X: its codes
// are widened to bf16 with their scale (exact) on the way into LDS, and the
// products run on v_mfma_f32_32x32x16_bf16.  Both sides lie in LDS as they do
// in memory, rows of 128 columns; the operands, which need eight consecutive
// m of a column per lane, are read with the transposing LDS load
// (ds_read_b64_tr_b16: sixteen lanes read four rows of sixteen columns and
// each receives the four rows of one column).  Rows are 256 bytes, all 64
// banks, in eight segments of 32 bytes; segment s of row r is at position
// s ^ 2 (r % 4), so that the four rows and two segments that half a wave reads
// lie in different banks.
// A workgroup owns a 128 x 128 tile of dW, which is one block of X's scales;
// dY's rows go straight from memory into LDS.  With few tiles the rows are
// split among workgroups, whose sums are added by a second kernel in a fixed
// order (workspace; no atomics).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "qgemv_f8_internal.h"

namespace qg {
namespace {

constexpr int kStep = 64;     // rows per step
constexpr int kThreads = 256;

typedef short s4_t __attribute__((ext_vector_type(4)));
typedef short s8_t __attribute__((ext_vector_type(8)));

struct WgradParams {
    const uint16_t *dY;
    const uint8_t *xq;
    float *dW;            // or the partial sums [splits][N][K]
    F8Rows rows;
    int64_t x_scales;
    int N, K, cb, x_ls;
    int tiles_n, splits;
    int64_t split_rows;   // rows of a split, a multiple of kStep
    bool accumulate, vec;
};

__device__ const uint4 g_zero = {0u, 0u, 0u, 0u};

__device__ __forceinline__ int seg_at(int row, int seg) { return seg ^ (2 * (row & 3)); }

// ALIGNED: rows of dY start at multiples of 16 bytes.
template <bool ALIGNED, bool GROUPED>
__global__ __launch_bounds__(kThreads, 2) void wgrad_kernel(WgradParams p)
{
    __shared__ uint4 Y0[kStep * 16], Y1[kStep * 16], X0[kStep * 16], X1[kStep * 16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave & 1, wk = wave >> 1;

    // blockIdx: (expert or split, column block of X, tile of dY's columns)
    const int tn = blockIdx.x % p.tiles_n;
    const int kb = (int)(blockIdx.x / p.tiles_n) % p.cb;
    const int part = (int)(blockIdx.x / p.tiles_n) / p.cb;
    const int n0 = tn * 128, k0 = kb * 128;
    int64_t r0, r1;
    float *out = p.dW + (int64_t)part * p.N * p.K;
    if constexpr (GROUPED) {
        const int64_t all = p.rows.rows;
        r0 = min(max((int64_t)p.rows.offsets[part], (int64_t)0), all);
        r1 = max(r0, min(max((int64_t)p.rows.offsets[part + 1], (int64_t)0), all));
        if (r0 == r1 && p.accumulate)
            return;
    } else {
        r0 = min(part * p.split_rows, p.rows.rows);
        r1 = min(r0 + p.split_rows, p.rows.rows);
    }

    // row of dY and of X of the at-th row; -1: none (zeros)
    auto rows_of = [&](int64_t at, int64_t &y, int64_t &x) {
        y = x = at < r1 ? at : -1;
        if constexpr (GROUPED) {
            const int s = at < r1 ? p.rows.order[at] : -1;
            const bool ok = s >= 0 && s < p.rows.rows;
            y = ok ? s : -1;
            x = ok ? min((int64_t)((uint32_t)s / (uint32_t)p.rows.k_slots), p.rows.x_rows - 1) : -1;
        }
    };
    // copies of dY: thread -> (row, 16-byte position) idx / 16, idx % 16
    auto copy_y = [&](uint4 *Y, int64_t m) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int idx = threadIdx.x + kThreads * i;
            const int r = idx >> 4, pos = idx & 15;
            const int n = n0 + 8 * (2 * seg_at(r, pos >> 1) + (pos & 1));
            int64_t y, x;
            rows_of(m + r, y, x);
            const uint16_t *src = p.dY + y * p.N + n;
            if constexpr (ALIGNED) {
                const void *from = y >= 0 && n < p.N ? static_cast<const void *>(src) : &g_zero;
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                                 (__attribute__((address_space(3))) void *)&Y[kThreads * i + 64 * wave],
                                                 16, 0, 0);
            } else {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t lo = y >= 0 && n + 2 * e < p.N ? src[2 * e] : 0u;
                    const uint32_t hi = y >= 0 && n + 2 * e + 1 < p.N ? src[2 * e + 1] : 0u;
                    w[e] = lo | hi << 16;
                }
                Y[idx] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    };
    // codes of X: thread -> (row, segment) idx / 8, idx % 8
    uint4 codes[2];
    float scale[2];
    auto load_x = [&](int64_t m) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int idx = threadIdx.x + kThreads * i;
            int64_t y, x;
            rows_of(m + (idx >> 3), y, x);
            codes[i] = make_uint4(0u, 0u, 0u, 0u);
            scale[i] = 1.0f;
            if (x >= 0) {
                codes[i] = *reinterpret_cast<const uint4 *>(p.xq + (x * p.cb + kb) * 128 + (idx & 7) * 16);
                scale[i] = f8_scale(p.xq[p.x_scales + x * p.x_ls + kb]);
            }
        }
    };
    auto store_x = [&](uint4 *X) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int idx = threadIdx.x + kThreads * i;
            const int r = idx >> 3;
            const int at = r * 16 + 2 * seg_at(r, idx & 7);
            X[at] = __builtin_bit_cast(uint4, f8_widen(codes[i].x, codes[i].y, scale[i]));
            X[at + 1] = __builtin_bit_cast(uint4, f8_widen(codes[i].z, codes[i].w, scale[i]));
        }
    };
    // eight consecutive rows 16 q + 8 (lane / 32) .. of column 32 t + lane % 32
    auto operand = [&](const uint4 *S, int q, int t) -> bf8_t {
        const int i = lane & 15;
        const int seg = 2 * t + ((lane >> 4) & 1);
        const char *base = reinterpret_cast<const char *>(S);
        s4_t v[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const int row = 16 * q + 8 * (lane >> 5) + 4 * o + (i >> 2);
            v[o] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4_t *)(
                base + row * 256 + 32 * seg_at(row, seg) + 8 * (i & 3)));
        }
        const s8_t w = __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(bf8_t, w);
    };

    f16v_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[i][j][e] = 0.0f;

    auto multiply = [&](const uint4 *Y, const uint4 *X) {
#pragma unroll
        for (int q = 0; q < kStep / 16; ++q) {
            bf8_t x[2], y[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[i] = operand(X, q, wk * 2 + i);
                y[i] = operand(Y, q, wn * 2 + i);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[i], y[j], acc[i][j], 0, 0, 0);
        }
    };
    auto turn = [&](int64_t m, uint4 *Y, uint4 *X, uint4 *Yn) {
        store_x(X);
        __builtin_amdgcn_s_waitcnt((0 & 15) | (7 << 4) | (15 << 8));   // this wave's copies have landed
        __syncthreads();
        if (m + kStep < r1) {
            copy_y(Yn, m + kStep);
            load_x(m + kStep);
        }
        multiply(Y, X);
    };
    if (r0 < r1) {
        copy_y(Y0, r0);
        load_x(r0);
        for (int64_t m = r0; m < r1; m += 2 * kStep) {
            turn(m, Y0, X0, Y1);
            if (m + kStep < r1)
                turn(m + kStep, Y1, X1, Y0);
        }
    }

    // lane: columns n of dY (lane % 32), four consecutive k each
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int n = n0 + (wn * 2 + j) * 32 + (lane & 31);
        if (n >= p.N)
            continue;
        float *row = out + (int64_t)n * p.K;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int k = k0 + (wk * 2 + i) * 32 + 8 * g + 4 * (lane >> 5);
                const float *v = reinterpret_cast<const float *>(&acc[i][j]) + 4 * g;
                if (p.vec && k + 4 <= p.K) {
                    f4_t w = {v[0], v[1], v[2], v[3]};
                    if (p.accumulate)
                        w += *reinterpret_cast<const f4_t *>(row + k);
                    *reinterpret_cast<f4_t *>(row + k) = w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (k + e < p.K)
                            row[k + e] = v[e] + (p.accumulate ? row[k + e] : 0.0f);
                }
            }
    }
}

struct JoinParams {
    const float *part;
    float *dW;
    int64_t n;
    int splits;
    bool accumulate;
};

__global__ __launch_bounds__(256) void join_kernel(JoinParams p)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.n; i += (int64_t)gridDim.x * 256) {
        float v = p.accumulate ? p.dW[i] : 0.0f;
        for (int s = 0; s < p.splits; ++s)
            v += p.part[s * p.n + i];
        p.dW[i] = v;
    }
}

// Splits of the rows: enough for two workgroups on each of 256 CUs, at least
// 512 rows each.
int splits_of(int64_t M, int64_t N, int64_t K)
{
    const int64_t tiles = ceil_div(N, 128) * ceil_div(K, 128);
    const int64_t want = std::min<int64_t>(512 / std::max<int64_t>(1, tiles), M / 512);
    return (int)std::max<int64_t>(1, want);
}

template <bool GROUPED>
hipError_t launch(const WgradParams &p, int64_t parts, hipStream_t stream)
{
    const bool al = p.N % 8 == 0 && (reinterpret_cast<uintptr_t>(p.dY) & 15) == 0;
    const void *fn = al ? reinterpret_cast<const void *>(&wgrad_kernel<true, GROUPED>)
                        : reinterpret_cast<const void *>(&wgrad_kernel<false, GROUPED>);
    return launch_kernel(fn, dim3((unsigned)(parts * p.tiles_n * p.cb)), dim3(kThreads), 0, stream, p);
}

}  // namespace

size_t f8_wgrad_workspace(int64_t M, int64_t N, int64_t K)
{
    const int s = splits_of(M, N, K);
    return s > 1 ? (size_t)s * N * K * sizeof(float) : 0;
}

hipError_t launch_f8_wgrad(const uint16_t *dY, const uint8_t *xq, float *dW, bool accumulate, const F8Rows &r,
                           int64_t N, int64_t K, float *workspace, int cus, hipStream_t stream)
{
    const F8Acts a = f8_acts(r.x_rows, K);
    WgradParams p{dY, xq, dW, r, a.scales, (int)N, (int)K, a.cb, a.ls, (int)ceil_div(N, 128), 1, r.rows, accumulate,
                  K % 4 == 0 && (reinterpret_cast<uintptr_t>(dW) & 15) == 0};
    if (r.order)
        return launch<true>(p, r.P, stream);
    p.splits = splits_of(r.rows, N, K);
    if (p.splits == 1)
        return launch<false>(p, 1, stream);
    p.split_rows = ceil_div(ceil_div(r.rows, p.splits), kStep) * kStep;
    p.dW = workspace;
    p.accumulate = false;
    p.vec = K % 4 == 0;
    const hipError_t e = launch<false>(p, p.splits, stream);
    if (e != hipSuccess)
        return e;
    const JoinParams j{workspace, dW, N * K, p.splits, accumulate};
    return launch_kernel(reinterpret_cast<const void *>(&join_kernel),
                         dim3((unsigned)std::min<int64_t>(ceil_div(j.n, 256), 8LL * cus)), dim3(256), 0, stream, j);
}

}  // namespace qg
