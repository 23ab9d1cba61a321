// f8 products of few rows: up to 64 tokens of one matrix, or experts with few
// tokens each.  y[m][n] = sum_k X[m][k] W[n][k].
//
// Bound by the bytes of W, each read once: a workgroup of eight waves owns 16
// R rows of W, its waves take the column blocks of 128 in turn (so the
// workgroup reads 16 KiB of consecutive memory a round) and add their sums
// through LDS at the end: no atomics, no second launch, and 16 rows a
// workgroup fill the card from 4096 rows up.
// A tile of W is in operand order in memory: a wave's lane l loads 16 codes of
// row l % 16 with each of two loads of a whole kilobyte, nothing goes through
// LDS.  The codes are widened to bf16 with their scale (exact: four
// significant bits and a power of two) and multiplied with
// v_mfma_f32_16x16x32_bf16.  The 8-bit matrix instructions would save the
// widening, but they align products to the largest of a few neighbours and
// lose what is 13 bits below (1.2e-5 of the result on normal data, against
// 7e-9), and the widening hides behind the loads.
// Activations: packed ones are read from L2 by every workgroup; with 1 to 8
// tokens in fp16, bf16 or fp32 each wave quantizes the column blocks that it
// multiplies itself into LDS first (wave-private: no barrier).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "qgemv_f8_internal.h"

namespace qg {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

struct SkinnyParams {
    const uint8_t *W;
    const uint8_t *xq;    // packed activations, or
    const void *x;        // [M][K] to quantize
    void *Y;
    F8Rows rows;
    int64_t w_scales, x_scales;
    int64_t units;        // tiles of tokens (grouped: an upper bound)
    int N, K, cb, ls, rt, row_groups;
    int y_type;
    bool vec;             // rows of Y take whole vectors of four
};

template <int R, int G>
struct Block {
    uint4 w[R][2];
    uint4 x[G][2];
    uint32_t ws[R], xs[G];
};

template <typename T>
__device__ __forceinline__ void store4(void *Y, int64_t at, const f4_t &v, int left, bool vec)
{
    T *y = static_cast<T *>(Y) + at;
    if (vec && left >= 4) {
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<f4_t *>(y) = v;
        else
            *reinterpret_cast<uint2 *>(y) =
                make_uint2(from_f32<T>(v[0]).u | (uint32_t)from_f32<T>(v[1]).u << 16,
                           from_f32<T>(v[2]).u | (uint32_t)from_f32<T>(v[3]).u << 16);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left)
                y[i] = from_f32<T>(v[i]);
    }
}

// SRC: void = packed activations, else the type of x.
template <typename SRC, int R, int G, bool GROUPED>
__global__ __launch_bounds__(kThreads) void skinny_kernel(SkinnyParams p)
{
    constexpr bool kPacked = sizeof(SRC) == 1;
    constexpr int U = R * G == 1 ? 4 : R * G <= 4 ? 2 : 1;   // column blocks in flight, twice
    extern __shared__ uint4 lds[];
    f4_t *part = reinterpret_cast<f4_t *>(lds);                      // [wave][R][G][64]
    uint4 *codes = lds + kWaves * R * G * 64;                        // [cb][2][32], quantizing
    uint8_t *scales = reinterpret_cast<uint8_t *>(codes + p.cb * 64);   // [cb][8]

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, c = lane >> 4;
    const int mine = (p.cb - wave + kWaves - 1) / kWaves;   // column blocks wave, wave + 8, ..

    if constexpr (!kPacked) {
        // lane (c, r) holds columns 16 c .. and 64 + 16 c .. of token r of a
        // block; a block's largest value is over the four lanes of a token
        const int m = min(r16 & 7, (int)p.rows.rows - 1);
        const SRC *row = static_cast<const SRC *>(p.x) + (int64_t)m * p.K;
        for (int j = 0; j < mine; ++j) {
            const int cb = wave + kWaves * j;
            float v[2][16];
            uint32_t amax = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = 128 * cb + 64 * h + 16 * c;
                load_row(row + k, p.K - k, v[h]);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    amax = max(amax, finite_mag(v[h][i]));
            }
            amax = max(amax, (uint32_t)__shfl_xor((int)amax, 16));
            amax = max(amax, (uint32_t)__shfl_xor((int)amax, 32));
            const uint32_t byte = f8_scale_byte(amax);
            const float inv = f8_inverse(byte);
            if (r16 < 8) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        w[i] = f8_pack4(f8_prepare(v[h][4 * i], inv), f8_prepare(v[h][4 * i + 1], inv),
                                        f8_prepare(v[h][4 * i + 2], inv), f8_prepare(v[h][4 * i + 3], inv));
                    codes[(cb * 2 + h) * 32 + c * 8 + r16] = make_uint4(w[0], w[1], w[2], w[3]);
                }
                if (c == 0)
                    scales[cb * 8 + r16] = (uint8_t)byte;
            }
        }
    }

    const int64_t total = p.units * p.row_groups;
    for (int64_t item = blockIdx.x; item < total; item += gridDim.x) {
        const int64_t unit = GROUPED ? item / p.row_groups : 0;
        const int rg = (int)(item - unit * p.row_groups);
        F8Unit u{0, 0, p.rows.rows};
        if constexpr (GROUPED) {
            u = f8_unit(p.rows.offsets, p.rows.P, p.rows.rows, 16 * G, unit);
            if (u.r0 >= u.r1)
                return;   // later units are past the end as well (uniform over the workgroup)
        }
        // this lane's tokens: rows of Y (-1: none) and of X
        int64_t y_row[G], x_row[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int64_t at = u.r0 + 16 * g + r16;
            y_row[g] = at < u.r1 ? at : -1;
            x_row[g] = min(at, u.r1 - 1);
            if constexpr (GROUPED) {
                const int64_t s = p.rows.order[x_row[g]];
                const bool ok = s >= 0 && s < p.rows.rows;
                y_row[g] = at < u.r1 && ok ? s : -1;
                x_row[g] = ok ? min((int64_t)((uint32_t)s / (uint32_t)p.rows.k_slots), p.rows.x_rows - 1) : 0;
            }
        }

        f4_t acc[R][G];
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int g = 0; g < G; ++g)
                acc[i][g] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};

        if (!GROUPED || u.e < p.rows.P) {
            const uint8_t *W = p.W + (GROUPED ? u.e * p.rows.stride : 0);
            const int t0 = rg * R;
            const auto rw = make_rsrc(W + (int64_t)t0 * p.cb * 2048, (int64_t)min(R, p.rt - t0) * p.cb * 2048);
            auto load = [&](Block<R, G>(&b)[U], int j0) {
#pragma unroll
                for (int q = 0; q < U; ++q) {
                    const int cb = wave + kWaves * min(j0 + q, mine - 1);
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        // a row tile past the matrix lies outside the descriptor: zeros
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            b[q].w[i][h] = GROUPED ? [&] {
                                const auto t = __builtin_amdgcn_raw_buffer_load_b128(
                                    rw, (uint32_t)((i * p.cb + cb) * 2048 + 1024 * h + 16 * lane), 0, 0);
                                return make_uint4(t[0], t[1], t[2], t[3]);
                            }() : stream_load16(rw, (uint32_t)((i * p.cb + cb) * 2048 + 1024 * h + 16 * lane));
                        b[q].ws[i] = W[p.w_scales + (int64_t)(min(t0 + i, p.rt - 1) >> 3) * p.ls + cb];
                    }
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        if constexpr (kPacked) {
                            const uint8_t *x = p.xq + (x_row[g] * p.cb + cb) * 128 + 16 * c;
                            b[q].x[g][0] = *reinterpret_cast<const uint4 *>(x);
                            b[q].x[g][1] = *reinterpret_cast<const uint4 *>(x + 64);
                            b[q].xs[g] = p.xq[p.x_scales + x_row[g] * p.ls + cb];
                        } else {
                            b[q].x[g][0] = codes[cb * 64 + c * 8 + (r16 & 7)];
                            b[q].x[g][1] = codes[cb * 64 + 32 + c * 8 + (r16 & 7)];
                            b[q].xs[g] = scales[cb * 8 + (r16 & 7)];
                        }
                    }
                }
            };
            auto multiply = [&](const Block<R, G>(&b)[U], int j0) {
#pragma unroll
                for (int q = 0; q < U; ++q) {
                    if (j0 + q >= mine)
                        break;   // uniform over the wave
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int o = 0; o < 2; ++o) {
                            bf8_t w[R], x[G];
#pragma unroll
                            for (int i = 0; i < R; ++i)
                                w[i] = o ? f8_widen(b[q].w[i][h].z, b[q].w[i][h].w, f8_scale(b[q].ws[i]))
                                         : f8_widen(b[q].w[i][h].x, b[q].w[i][h].y, f8_scale(b[q].ws[i]));
#pragma unroll
                            for (int g = 0; g < G; ++g)
                                x[g] = o ? f8_widen(b[q].x[g][h].z, b[q].x[g][h].w, f8_scale(b[q].xs[g]))
                                         : f8_widen(b[q].x[g][h].x, b[q].x[g][h].y, f8_scale(b[q].xs[g]));
#pragma unroll
                            for (int i = 0; i < R; ++i)
#pragma unroll
                                for (int g = 0; g < G; ++g)
                                    acc[i][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], x[g], acc[i][g], 0, 0, 0);
                        }
                }
            };
            if (mine > 0) {
                Block<R, G> b0[U], b1[U];
                load(b0, 0);
                for (int j = 0; j < mine; j += 2 * U) {
                    if (j + U < mine)
                        load(b1, j + U);
                    __builtin_amdgcn_sched_barrier(0);   // the next loads stay ahead of the products
                    multiply(b0, j);
                    if (j + 2 * U < mine)
                        load(b0, j + 2 * U);
                    __builtin_amdgcn_sched_barrier(0);
                    if (j + U < mine)
                        multiply(b1, j + U);
                }
            }
        }

        // D of a 16 x 16 product: lane (c, r) holds rows 4 c .. 4 c + 3 (of W)
        // of column r (token r)
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int g = 0; g < G; ++g)
                part[((wave * R + i) * G + g) * 64 + lane] = acc[i][g];
        __syncthreads();
        // the R G 64 vectors of four are spread over the waves: wave w adds
        // the pairs (i, g) w, w + 8, ..
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int g = 0; g < G; ++g)
                if (((i * G + g) & (kWaves - 1)) == wave) {
                    f4_t v = part[(i * G + g) * 64 + lane];
#pragma unroll
                    for (int w = 1; w < kWaves; ++w)
                        v += part[((w * R + i) * G + g) * 64 + lane];
                    const int n = (rg * R + i) * 16 + 4 * c;
                    if (y_row[g] >= 0 && n < p.N) {
                        const int64_t at = y_row[g] * p.N + n;
                        if (p.y_type == QG_F32)
                            store4<float>(p.Y, at, v, p.N - n, p.vec);
                        else if (p.y_type == QG_F16)
                            store4<Fp16>(p.Y, at, v, p.N - n, p.vec);
                        else
                            store4<Bf16>(p.Y, at, v, p.N - n, p.vec);
                    }
                }
        __syncthreads();   // part is free again
    }
}

struct Packed {
    uint8_t u;
};

template <typename SRC, int R, int G, bool GROUPED>
hipError_t launch(SkinnyParams &p, int cus, hipStream_t stream)
{
    p.row_groups = (p.rt + R - 1) / R;
    p.units = GROUPED ? f8_units(p.rows.rows, p.rows.P, 16 * G) : 1;
    const size_t lds = (size_t)kWaves * R * G * 1024 + (sizeof(SRC) == 1 ? 0 : (size_t)p.cb * (1024 + 8));
    const void *fn = reinterpret_cast<const void *>(&skinny_kernel<SRC, R, G, GROUPED>);
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess)
            return e;
    }
    // quantizing workgroups stay (each repeats the conversion); the others
    // come and go, so that one's loads cover another's sums
    const int64_t items = p.units * p.row_groups;
    const int64_t most = sizeof(SRC) == 1 ? (int64_t)1 << 22 : 2LL * cus;
    return launch_kernel(fn, dim3((unsigned)std::min(items, most)), dim3(kThreads), lds, stream, p);
}

}  // namespace

hipError_t launch_f8_skinny(const uint8_t *W, const uint8_t *xq, const void *x, int x_type, void *Y, int y_type,
                            const F8Rows &r, int64_t N, int64_t K, int cus, hipStream_t stream)
{
    const F8Weights f = f8_weights(N, K);
    SkinnyParams p{W, xq, x, Y, r, f.scales, f8_acts(r.x_rows, K).scales, 1, (int)N, (int)K, f.cb, f.ls, f.rt, 0,
                   y_type, N % 4 == 0 && (reinterpret_cast<uintptr_t>(Y) & (4 * type_bytes(y_type) - 1)) == 0};
    if (x)
        return x_type == QG_F32   ? launch<float, 1, 1, false>(p, cus, stream)
               : x_type == QG_F16 ? launch<Fp16, 1, 1, false>(p, cus, stream)
                                  : launch<Bf16, 1, 1, false>(p, cus, stream);
    if (r.order)
        return launch<Packed, 1, 1, true>(p, cus, stream);
    if (r.rows <= 16)
        return launch<Packed, 1, 1, false>(p, cus, stream);
    if (r.rows <= 32)
        return launch<Packed, 1, 2, false>(p, cus, stream);
    return launch<Packed, 2, 4, false>(p, cus, stream);
}

}  // namespace qg
