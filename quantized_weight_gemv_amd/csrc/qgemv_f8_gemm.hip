// f8 products of many rows: Y[m][n] = sum_k X[m][k] W[n][k] on the matrix
// cores, for one matrix or for the slots of each expert of a pool.
//
// A workgroup owns a tile of BM rows of X times BN rows of W.  Per step of
// 128 columns (one block: one scale byte a row and side) both operands go
// straight from memory into LDS (loads that write LDS: no registers):
//   * X, row-major: rows of 128 bytes, 16-byte chunk c of row r at position
//     c ^ ((r / 2) % 8), so that the 16 rows of a quarter of an operand read
//     touch all 64 banks;
//   * W, whose tiles are in operand order already: copied as they are; an
//     operand read is 256 consecutive bytes a quarter wave.
// Two buffers: while a step is multiplied, the next one's copies are in
// flight; one barrier a step.
// 16-bit outputs: v_mfma_scale_f32_32x32x64_f8f6f4 with the two block scales
// as its scale operands, so the fp32 sums need no further instruction.  fp32
// outputs: the codes are widened to bf16 with their scale (exact) and
// multiplied with v_mfma_f32_32x32x16_bf16: half the rate, but products and
// sums exact to fp32, where the 8-bit instructions keep about 13 bits below
// the largest of a few neighbouring products.
// W is the first operand, so a lane holds four consecutive n of a row of Y.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "qgemv_f8_internal.h"

namespace qg {
namespace {

struct GemmParams {
    const uint8_t *W, *xq;
    void *Y;
    F8Rows rows;
    int64_t w_scales, x_scales;
    int64_t units;       // tiles along the rows (grouped: an upper bound)
    int N, cb, x_ls, w_ls, rt, tiles_n;
    bool vec;
};

template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N >= 0 && N < 64, "vmcnt holds 6 bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

__device__ __forceinline__ void copy16(const uint8_t *from, void *to)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                     (__attribute__((address_space(3))) void *)to, 16, 0, 0);
}

// Tile shape: WM x WN waves, each 32 TM rows of X times 32 TN rows of W.
template <int WM, int WN, int TM, int TN>
struct Tile {
    static constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN, NT = 64 * WM * WN;
    static constexpr int XC = BM * 8 / NT, WC = BN * 8 / NT;   // 16-byte copies per thread and step
};

template <int WM, int WN, int TM, int TN, typename OUT, bool GROUPED>
__global__ __launch_bounds__(64 * WM *WN) void gemm_kernel(GemmParams p)
{
    using T = Tile<WM, WN, TM, TN>;
    constexpr bool kWide = sizeof(OUT) == 4;
    __shared__ uint4 X0[T::BM * 8], X1[T::BM * 8], W0[T::BN * 8], W1[T::BN * 8];
    __shared__ int out_row[T::BM];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int r32 = lane & 31, half = lane >> 5;

    const int64_t total = p.units * p.tiles_n;
    for (int64_t item = blockIdx.x; item < total; item += gridDim.x) {
        const int64_t unit = item / p.tiles_n;
        const int tn = (int)(item - unit * p.tiles_n);
        F8Unit u{0, unit * T::BM, min((unit + 1) * T::BM, p.rows.rows)};
        if constexpr (GROUPED) {
            u = f8_unit(p.rows.offsets, p.rows.P, p.rows.rows, T::BM, unit);
            if (u.r0 >= u.r1)
                return;   // uniform over the workgroup
        }
        const int n0 = tn * T::BN;
        const int rows = (int)(u.r1 - u.r0);

        // rows of X of this thread's copies, and of Y
        const uint8_t *xsrc[T::XC];
        auto x_row = [&](int r) -> int64_t {
            const int64_t at = u.r0 + min(r, rows - 1);
            if constexpr (!GROUPED)
                return at;
            const int s = p.rows.order[at];
            return s >= 0 && s < p.rows.rows ? min((int64_t)((uint32_t)s / (uint32_t)p.rows.k_slots), p.rows.x_rows - 1)
                                             : 0;
        };
        if constexpr (GROUPED) {
            for (int r = threadIdx.x; r < T::BM; r += T::NT) {
                int s = r < rows ? p.rows.order[u.r0 + r] : -1;
                out_row[r] = s >= 0 && s < p.rows.rows ? s : -1;
            }
        }
#pragma unroll
        for (int i = 0; i < T::XC; ++i) {
            const int idx = threadIdx.x + T::NT * i;
            const int r = idx >> 3, ch = (idx & 7) ^ ((r >> 1) & 7);
            xsrc[i] = p.xq + x_row(r) * p.cb * 128 + ch * 16;
        }
        const uint8_t *W = p.W + (GROUPED ? min(u.e, p.rows.P - 1) * p.rows.stride : 0);
        const uint8_t *wsrc[T::WC];
#pragma unroll
        for (int i = 0; i < T::WC; ++i) {
            const int idx = threadIdx.x + T::NT * i;
            const int t = min(n0 / 16 + (idx >> 7), p.rt - 1);   // rows past the matrix are never stored
            wsrc[i] = W + (int64_t)t * p.cb * 2048 + (idx & 127) * 16;
        }
        // scales: four steps' bytes a word
        const uint8_t *xs_src[TM];
        const uint8_t *ws_src;
#pragma unroll
        for (int i = 0; i < TM; ++i)
            xs_src[i] = p.xq + p.x_scales + x_row((wm * TM + i) * 32 + r32) * p.x_ls;
        static_assert(128 % (32 * TN) == 0, "a wave's rows of W lie in one block");
        ws_src = W + p.w_scales + (int64_t)min((n0 + wn * TN * 32) >> 7, (p.N - 1) >> 7) * p.w_ls;

        f16v_t acc[TM][TN];
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    acc[i][j][e] = 0.0f;

        if (!GROUPED || u.e < p.rows.P) {
            uint32_t xs[TM], ws;
            auto copies = [&](uint4 *X, uint4 *Wb) {
#pragma unroll
                for (int i = 0; i < T::XC; ++i) {
                    copy16(xsrc[i], &X[T::NT * i + 64 * wave]);
                    xsrc[i] += 128;
                }
#pragma unroll
                for (int i = 0; i < T::WC; ++i) {
                    copy16(wsrc[i], &Wb[T::NT * i + 64 * wave]);
                    wsrc[i] += 2048;
                }
            };
            auto step = [&](const uint4 *X, const uint4 *Wb) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint4 xv[TM][2], wv[TN][2];
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int ch = 4 * h + 2 * half + q;
#pragma unroll
                        for (int i = 0; i < TM; ++i) {
                            const int r = (wm * TM + i) * 32 + r32;
                            xv[i][q] = X[r * 8 + (ch ^ ((r >> 1) & 7))];
                        }
#pragma unroll
                        for (int j = 0; j < TN; ++j) {
                            const int t = (wn * TN + j) * 2 + (r32 >> 4);
                            wv[j][q] = Wb[t * 128 + ch * 16 + (r32 & 15)];
                        }
                    }
                    if constexpr (!kWide) {
#pragma unroll
                        for (int i = 0; i < TM; ++i)
#pragma unroll
                            for (int j = 0; j < TN; ++j) {
                                const i8_t a = {(int)wv[j][0].x, (int)wv[j][0].y, (int)wv[j][0].z, (int)wv[j][0].w,
                                                (int)wv[j][1].x, (int)wv[j][1].y, (int)wv[j][1].z, (int)wv[j][1].w};
                                const i8_t b = {(int)xv[i][0].x, (int)xv[i][0].y, (int)xv[i][0].z, (int)xv[i][0].w,
                                                (int)xv[i][1].x, (int)xv[i][1].y, (int)xv[i][1].z, (int)xv[i][1].w};
                                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc[i][j], 0, 0, 0,
                                                                                           (int)ws, 0, (int)xs[i]);
                            }
                    } else {
                        const float wf = f8_scale(ws & 255u);
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int o = 0; o < 2; ++o) {
                                bf8_t w[TN];
#pragma unroll
                                for (int j = 0; j < TN; ++j)
                                    w[j] = o ? f8_widen(wv[j][q].z, wv[j][q].w, wf)
                                             : f8_widen(wv[j][q].x, wv[j][q].y, wf);
#pragma unroll
                                for (int i = 0; i < TM; ++i) {
                                    const float xf = f8_scale(xs[i] & 255u);
                                    const bf8_t x = o ? f8_widen(xv[i][q].z, xv[i][q].w, xf)
                                                      : f8_widen(xv[i][q].x, xv[i][q].y, xf);
#pragma unroll
                                    for (int j = 0; j < TN; ++j)
                                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[j], x, acc[i][j], 0, 0,
                                                                                            0);
                                }
                            }
                    }
                }
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    xs[i] >>= 8;
                ws >>= 8;
            };
            copies(X0, W0);
            for (int s = 0; s < p.cb; s += 4) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (s + q >= p.cb)
                        break;   // uniform over the grid
                    if (q == 0) {
#pragma unroll
                        for (int i = 0; i < TM; ++i)
                            xs[i] = *reinterpret_cast<const uint32_t *>(xs_src[i] + s);
                        ws = *reinterpret_cast<const uint32_t *>(ws_src + s);
                    }
                    wait_vm<0>();        // this wave's copies of the step have landed,
                    __syncthreads();     // everyone's have, and the other buffer is free
                    if (s + q + 1 < p.cb)
                        copies(q & 1 ? X0 : X1, q & 1 ? W0 : W1);
                    step(q & 1 ? X1 : X0, q & 1 ? W1 : W0);
                }
            }
        }

        __syncthreads();   // out_row is written, and the buffers are free for the next tile
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int r = (wm * TM + i) * 32 + r32;
            const int64_t y = GROUPED ? out_row[r] : (r < rows ? u.r0 + r : -1);
            if (y < 0)
                continue;
            OUT *row = static_cast<OUT *>(p.Y) + y * p.N;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int n = n0 + (wn * TN + j) * 32 + 8 * g + 4 * half;
                    const float *v = reinterpret_cast<const float *>(&acc[i][j]) + 4 * g;
                    if (p.vec && n + 4 <= p.N) {
                        if constexpr (kWide)
                            *reinterpret_cast<f4_t *>(row + n) = f4_t{v[0], v[1], v[2], v[3]};
                        else
                            *reinterpret_cast<uint2 *>(row + n) =
                                make_uint2(from_f32<OUT>(v[0]).u | (uint32_t)from_f32<OUT>(v[1]).u << 16,
                                           from_f32<OUT>(v[2]).u | (uint32_t)from_f32<OUT>(v[3]).u << 16);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n + e < p.N)
                                row[n + e] = from_f32<OUT>(v[e]);
                    }
                }
        }
        if constexpr (GROUPED)
            __syncthreads();   // out_row is read before the next tile's is written
    }
}

template <int WM, int WN, int TM, int TN, typename OUT, bool GROUPED>
hipError_t launch(GemmParams &p, int cus, hipStream_t stream)
{
    using T = Tile<WM, WN, TM, TN>;
    p.tiles_n = (int)ceil_div(p.N, T::BN);
    p.units = GROUPED ? f8_units(p.rows.rows, p.rows.P, T::BM) : ceil_div(p.rows.rows, T::BM);
    const int64_t items = p.units * p.tiles_n;
    (void)cus;
    return launch_kernel(reinterpret_cast<const void *>(&gemm_kernel<WM, WN, TM, TN, OUT, GROUPED>),
                         dim3((unsigned)std::min<int64_t>(items, 1 << 22)), dim3(T::NT), 0, stream, p);
}

template <typename OUT, bool GROUPED>
hipError_t choose(GemmParams &p, int cus, hipStream_t stream)
{
    if constexpr (!GROUPED) {
        if (ceil_div(p.rows.rows, 256) * ceil_div(p.N, 256) >= cus)
            return launch<2, 4, 4, 2, OUT, GROUPED>(p, cus, stream);
        return launch<2, 2, 2, 2, OUT, GROUPED>(p, cus, stream);
    } else {
        return launch<2, 2, 1, 2, OUT, GROUPED>(p, cus, stream);
    }
}

}  // namespace

hipError_t launch_f8_gemm(const uint8_t *W, const uint8_t *xq, void *Y, int y_type, const F8Rows &r, int64_t N,
                          int64_t K, int cus, hipStream_t stream)
{
    const F8Weights f = f8_weights(N, K);
    const F8Acts a = f8_acts(r.x_rows, K);
    GemmParams p{W, xq, Y, r, f.scales, a.scales, 0, (int)N, f.cb, a.ls, f.ls, f.rt, 0,
                 N % 4 == 0 && (reinterpret_cast<uintptr_t>(Y) & (4 * type_bytes(y_type) - 1)) == 0};
    if (r.order)
        return y_type == QG_F32   ? choose<float, true>(p, cus, stream)
               : y_type == QG_F16 ? choose<Fp16, true>(p, cus, stream)
                                  : choose<Bf16, true>(p, cus, stream);
    return y_type == QG_F32   ? choose<float, false>(p, cus, stream)
           : y_type == QG_F16 ? choose<Fp16, false>(p, cus, stream)
                              : choose<Bf16, false>(p, cus, stream);
}

}  // namespace qg
