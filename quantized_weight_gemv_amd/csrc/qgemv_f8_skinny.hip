// f8 products of few rows: up to 64 tokens of one matrix, or experts with few
// tokens each.  y[m][n] = sum_k X[m][k] W[n][k].
//
// Bound by the bytes of W, each read once: a workgroup of eight waves owns 16
// rows of W, its waves take the column blocks of 128 in turn (so the
// workgroup reads 16 KiB of consecutive memory a round) and add their sums
// through LDS at the end: no atomics, no second launch, and 16 rows a
// workgroup fill the card from 4096 rows up.
// One and eight tokens (us): 4096 x 4096 6.2 and 7.7 in a row of launches (a
// launch and the latency of the first loads; 16.8 MB), 28672 x 4096 20.7 and
// 22 (5.3 to 5.7 TB/s, a copy's rate), 4096 x 14336 12.5 and 19.5 (every
// workgroup quantizes the tokens: 4.7 and 3.0 TB/s).  With four waves 6.8 and
// 9.3, 20.4 and 24, 14.8 and 24.9; with one block in flight instead of two
// 6.7 and 7.8, 20.8 and 23.2, 13.1 and 19.9; with 2, 3 or 4 workgroups a unit
// the same within 2 % (up to 6 % once).
// A tile of W is in operand order in memory: a wave's lane l loads 16 codes of
// row l % 16 with each of two loads of a whole kilobyte, nothing goes through
// LDS.  The codes are widened to bf16 with their scale (exact: four
// significant bits and a power of two) and multiplied with
// v_mfma_f32_16x16x32_bf16.  The 8-bit matrix instructions would save the
// widening, but they align products to the largest of a few neighbours and
// lose what is 13 bits below (1.2e-5 of the result on normal data, against
// 7e-9), and the widening hides behind the loads.
// Activations: packed ones are read from L2 by every workgroup; with 1 to 8
// tokens in fp16, bf16 or fp32 the workgroup quantizes them into LDS first,
// behind the loads of its first weights.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "qgemv_f8_internal.h"

namespace qg {
namespace {

struct Packed {
    uint8_t u;
};

struct SkinnyParams {
    const uint8_t *W;
    const uint8_t *xq;    // packed activations, or
    const void *x;        // [M][K] to quantize
    void *Y;
    F8Rows rows;
    int64_t w_scales, x_scales;
    int64_t units;        // tiles of tokens (grouped: an upper bound)
    int N, K, cb, ls, x_ls, rt, row_groups;
    int y_type;
    bool vec;             // rows of Y take whole vectors of four
};

// One column block of this wave's operands (X's only where it is packed, else
// it is read from LDS when it is multiplied).
struct Block {
    uint4 w[2], x[2];
    uint32_t ws, xs;
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
                make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left)
                y[i] = from_f32<T>(v[i]);
    }
}

// SRC: Packed, or the type of x; NW waves share K; U column blocks in flight
// (and U more while those are multiplied).
template <typename SRC, int NW, int U, bool GROUPED>
__global__ __launch_bounds__(64 * NW, 4) void skinny_kernel(SkinnyParams p)
{
    constexpr bool kPacked = sizeof(SRC) == 1;
    extern __shared__ uint4 lds[];
    f4_t *part = reinterpret_cast<f4_t *>(lds);                      // [2][wave][64]
    uint4 *codes = lds + 2 * NW * 64;                               // [cb][2][32], quantizing
    uint8_t *scales = reinterpret_cast<uint8_t *>(codes + p.cb * 64);   // [cb][8]

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, c = lane >> 4;
    const int mine = (p.cb - wave + NW - 1) / NW;       // this wave's column blocks: wave, wave + NW, ..
    const int batches = max(1, (mine + U - 1) / U);     // of U blocks, the last one may be short

    const int64_t total = p.units * p.row_groups;
    int64_t item = blockIdx.x;
    if (item >= total)
        return;
    F8Unit u{0, 0, p.rows.rows, 0, 1, 0, 0};
    int64_t y_row, x_row;   // this lane's rows of Y (-1: none) and of X
    const uint8_t *W = p.W;
    auto begin_unit = [&](int64_t unit) {
        if constexpr (GROUPED) {
            u = f8_unit(p.rows.offsets, p.rows.P, p.rows.rows, 16, unit);
            if (u.r0 >= u.r1)
                return;
            W = p.W + min(u.e, p.rows.P - 1) * p.rows.stride;
        }
        const int64_t at = u.r0 + r16;
        y_row = at < u.r1 ? at : -1;
        x_row = min(at, u.r1 - 1);
        if constexpr (GROUPED) {
            const int64_t s = p.rows.order[x_row];
            const bool ok = s >= 0 && s < p.rows.rows;
            y_row = at < u.r1 && ok ? s : -1;
            x_row = ok ? min((int64_t)((uint32_t)s / (uint32_t)p.rows.k_slots), p.rows.x_rows - 1) : 0;
        }
    };
    begin_unit(GROUPED ? item / p.row_groups : 0);
    if (GROUPED && u.r0 >= u.r1)
        return;   // past the last unit (uniform over the workgroup)

    auto load_w = [&](Block(&b)[U], int rg, int j0) {
        const auto rw = make_rsrc(W + (int64_t)rg * p.cb * 2048, (int64_t)p.cb * 2048);
#pragma unroll
        for (int q = 0; q < U; ++q) {
            // past the wave's last block: that one again, unused; a wave
            // without blocks reads outside the descriptor
            const int cb = wave + NW * max(0, min(j0 + q, mine - 1));
#pragma unroll
            for (int h = 0; h < 2; ++h)
                b[q].w[h] = stream_load16(rw, (uint32_t)(cb * 2048 + 1024 * h + 16 * lane));
            b[q].ws = W[p.w_scales + (int64_t)(rg >> 3) * p.ls + min(cb, p.cb - 1)];
        }
    };
    auto load_x = [&](Block(&b)[U], int j0) {
        if constexpr (kPacked) {
#pragma unroll
            for (int q = 0; q < U; ++q) {
                const int cb = min(wave + NW * max(0, min(j0 + q, mine - 1)), p.cb - 1);
                const uint8_t *x = p.xq + (x_row * p.cb + cb) * 128 + 16 * c;
                b[q].x[0] = *reinterpret_cast<const uint4 *>(x);
                b[q].x[1] = *reinterpret_cast<const uint4 *>(x + 64);
                b[q].xs = p.xq[p.x_scales + x_row * p.ls + cb];
            }
        }
    };

    f4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](const Block(&b)[U], int j0) {
#pragma unroll
        for (int q = 0; q < U; ++q) {
            if (j0 + q >= mine)
                break;   // uniform over the wave
            const int cb = wave + NW * (j0 + q);
            uint4 xv[2];
            uint32_t xb;
            if constexpr (kPacked) {
                xv[0] = b[q].x[0], xv[1] = b[q].x[1];
                xb = b[q].xs;
            } else {
                // tokens from M on hold what is in LDS: their sums are never stored
                xv[0] = codes[cb * 64 + c * 8 + (r16 & 7)];
                xv[1] = codes[cb * 64 + 32 + c * 8 + (r16 & 7)];
                xb = scales[cb * 8 + (r16 & 7)];
            }
            const float ws = f8_exponent(b[q].ws), xs = f8_exponent(xb);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f8_widen(b[q].w[h].x, b[q].w[h].y, ws),
                                                              f8_widen(xv[h].x, xv[h].y, xs), acc, 0, 0, 0);
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f8_widen(b[q].w[h].z, b[q].w[h].w, ws),
                                                              f8_widen(xv[h].z, xv[h].w, xs), acc, 0, 0, 0);
            }
        }
    };
    // D of a 16 x 16 product: lane (c, r) holds rows 4 c .. 4 c + 3 (of W) of
    // column r (token r).  The first wave adds the waves' vectors of four from
    // LDS.  Two buffers in turn: one barrier an item.
    int turn = 0;
    auto finish = [&](int rg) {
        f4_t *buf = part + turn * NW * 64;
        turn ^= 1;
        buf[wave * 64 + lane] = acc;
        wait_lds();
        bare_barrier();   // the next row group's loads stay in flight
        if (wave == 0) {
            f4_t v = buf[lane];
#pragma unroll
            for (int w = 1; w < NW; ++w)
                v += buf[w * 64 + lane];
            const int n = rg * 16 + 4 * c;
            if (y_row >= 0 && n < p.N) {
                const int64_t at = y_row * p.N + n;
                if (p.y_type == QG_F32)
                    store4<float>(p.Y, at, v, p.N - n, p.vec);
                else if (p.y_type == QG_F16)
                    store4<Fp16>(p.Y, at, v, p.N - n, p.vec);
                else
                    store4<Bf16>(p.Y, at, v, p.N - n, p.vec);
            }
        }
        acc = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
    };

    // The batches of `items` row groups from rg on, gridDim.x apart, as one
    // sequence: the next batch's loads are issued before a batch is multiplied,
    // across row groups as well.  b0 holds the first batch.  The loads of a
    // pair of batches stand on one path without branches, so that a wait for
    // a batch leaves the next one's loads in flight.
    Block b0[U], b1[U];
    auto run = [&](int rg, int items) {
        int t = 0;
        auto turn = [&](Block(&cur)[U], Block(&nxt)[U], bool more) {
            const bool last = t + 1 == batches;
            const int nt = last ? 0 : t + 1, nrg = last ? rg + (int)gridDim.x : rg;
            if (more) {   // known where it is called
                load_x(nxt, nt * U);
                load_w(nxt, nrg, nt * U);
                __builtin_amdgcn_sched_barrier(0);
            }
            multiply(cur, t * U);
            if (last)
                finish(rg);
            t = nt, rg = nrg;
        };
        int left = items * batches;
        for (; left > 2; left -= 2) {
            turn(b0, b1, true);
            turn(b1, b0, true);
        }
        if (left == 2) {
            turn(b0, b1, true);
            turn(b1, b0, false);
        } else {
            turn(b0, b1, false);
        }
    };
    if constexpr (GROUPED) {
        // one item after the other: its expert and its tokens have to be found
        for (;;) {
            const int rg = (int)(item % p.row_groups);
            if (u.e < p.rows.P) {
                load_x(b0, 0);
                load_w(b0, rg, 0);
                run(rg, 1);
            } else {
                finish(rg);   // no expert: zeros
            }
            item += gridDim.x;
            if (item >= total)
                return;
            begin_unit(item / p.row_groups);
            if (u.r0 >= u.r1)
                return;
        }
    } else {
        // Quantizing: a lane takes 16 columns of a token's block, eight lanes
        // the block; the workgroup's threads share the M cb blocks.
        constexpr int QB = 2;   // of a lane's pieces at a time
        float raw[kPacked ? 1 : QB][16];
        const int pieces = 8 * p.cb * (int)p.rows.rows;
        auto piece = [&](int q, int &m, int &blk, int &chunk) {
            const int id = threadIdx.x + 64 * NW * q;
            chunk = id & 7;
            m = (id >> 3) / p.cb;
            blk = (id >> 3) - m * p.cb;
            return id < pieces;   // whole groups of eight lanes
        };
        auto load_raw = [&](int q0) {
            if constexpr (!kPacked) {
#pragma unroll
                for (int q = 0; q < QB; ++q) {
                    int m, blk, chunk;
                    const bool in = piece(q0 + q, m, blk, chunk);
                    const int k = 128 * blk + 16 * chunk;
                    load_row(static_cast<const SRC *>(p.x) + (in ? (int64_t)m * p.K + k : 0), in ? p.K - k : 0,
                             raw[q]);
                }
            }
        };
        auto quantize = [&](int q0) {
            if constexpr (!kPacked) {
#pragma unroll
                for (int q = 0; q < QB; ++q) {
                    int m, blk, chunk;
                    const bool in = piece(q0 + q, m, blk, chunk);
                    uint32_t w[4];
                    const uint32_t byte = f8_quantize16(raw[q], w);
                    if (in) {
                        // columns 16 c .. of half h: read by lanes 16 c + r, r % 8 = token
                        codes[blk * 64 + (chunk >> 2) * 32 + (chunk & 3) * 8 + m] = make_uint4(w[0], w[1], w[2], w[3]);
                        if (chunk == 0)
                            scales[blk * 8 + m] = (uint8_t)byte;
                    }
                }
            }
        };
        if constexpr (!kPacked)
            load_raw(0);
        load_x(b0, 0);
        load_w(b0, (int)item, 0);
        if constexpr (!kPacked) {
            __builtin_amdgcn_sched_barrier(0);   // x first, the weights right behind it, then the conversion
            quantize(0);
            for (int q = QB; 64 * NW * q < pieces; q += QB) {
                load_raw(q);
                quantize(q);
            }
            wait_lds();
            bare_barrier();   // the weights stay in flight
        }
        run((int)item, (p.row_groups - (int)item + (int)gridDim.x - 1) / (int)gridDim.x);
    }
}

// 17 to 64 tokens of one matrix (G groups of 16; where N is large the tiled
// kernels take over): the same streaming of W, with
// X's blocks copied into LDS a block ahead (buffer loads that write LDS), by
// each wave for itself.  An operand read straight from memory takes 16 rows x
// 64 bytes, and the caches deliver 9.5 TB/s to such loads against 30 to the 8
// rows x 128 bytes of a copy; X, read by every workgroup, is most of what is
// read here.  Rows are 128 bytes, 16-byte chunk c of row r at position
// c ^ ((r / 2) % 8): the 16 rows of a quarter of an operand read touch all 64
// banks.  Every unit needs all of X: 64 x 4096 x 14336 takes 28 us, of which
// W alone is 14, the copies of X 11 (235 MB at 20 TB/s) and the products,
// behind them, 3: W's loads and X's copies share the way and add up; 17 tokens
// take 15, 32 19.  Four waves with four buffers each
// take as long (29, 15, 19).
template <int G>
__global__ __launch_bounds__(512, 2) void skinny_lds_kernel(SkinnyParams p)
{
    constexpr int NW = 8, kRows = 16 * G, kCopies = kRows / 8;
    // one variable a buffer, as the compiler then knows which copies a read waits for
    __shared__ uint4 XA[NW * kRows * 8], XB[NW * kRows * 8];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, c = lane >> 4;
    const int mine = (p.cb - wave + NW - 1) / NW;   // this wave's column blocks: wave, wave + 8, ..
    const int rows = (int)p.rows.rows;
    const auto rx = make_rsrc(p.xq, (int64_t)rows * p.cb * 128);

    uint32_t x_at[kCopies], xs_at[G];
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int r = 8 * i + (lane >> 3);
        x_at[i] = (uint32_t)(min(r, rows - 1) * p.cb * 128 + ((lane & 7) ^ ((r >> 1) & 7)) * 16);
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
        xs_at[g] = (uint32_t)(min(16 * g + r16, rows - 1) * p.x_ls);

    struct Regs {
        uint4 w[2];
        uint32_t ws, xs[G];
    };
    f4_t acc[G];
    auto clear = [&] {
#pragma unroll
        for (int g = 0; g < G; ++g)
            acc[g] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
    };
    auto load = [&](Regs &b, uint4 *X, int rg, int j) {
        const int cb = min(wave + NW * j, p.cb - 1);
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
            copy16(rx, &X[(wave * kRows + 8 * i) * 8], x_at[i], cb * 128);
        const auto rw = make_rsrc(p.W + (int64_t)rg * p.cb * 2048, (int64_t)p.cb * 2048);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            b.w[h] = stream_load16(rw, (uint32_t)(cb * 2048 + 1024 * h + 16 * lane));
        b.ws = p.W[p.w_scales + (int64_t)(rg >> 3) * p.ls + cb];
#pragma unroll
        for (int g = 0; g < G; ++g)
            b.xs[g] = p.xq[p.x_scales + xs_at[g] + cb];
    };
    auto multiply = [&](const Regs &b, const uint4 *X) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint4 x[G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int r = 16 * g + r16;
                x[g] = X[(wave * kRows + r) * 8 + ((c + 4 * h) ^ ((r >> 1) & 7))];
            }
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const bf8_t w = o ? f8_widen(b.w[h].z, b.w[h].w, f8_exponent(b.ws))
                                  : f8_widen(b.w[h].x, b.w[h].y, f8_exponent(b.ws));
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const bf8_t v = o ? f8_widen(x[g].z, x[g].w, f8_exponent(b.xs[g]))
                                      : f8_widen(x[g].x, x[g].y, f8_exponent(b.xs[g]));
                    acc[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, v, acc[g], 0, 0, 0);
                }
            }
        }
    };
    // the waves' sums are added through LDS, group g by wave g; XA or XB,
    // whichever the next block is not copied into, holds them
    auto finish = [&](int rg, uint4 *X) {
        f4_t *buf = reinterpret_cast<f4_t *>(X);
        wait_lds();
        bare_barrier();   // every wave has read its last block from X
#pragma unroll
        for (int g = 0; g < G; ++g)
            buf[(wave * G + g) * 64 + lane] = acc[g];
        wait_lds();
        bare_barrier();
        if (wave < G) {
            f4_t v = buf[wave * 64 + lane];
#pragma unroll
            for (int w = 1; w < NW; ++w)
                v += buf[(w * G + wave) * 64 + lane];
            const int n = rg * 16 + 4 * c, m = 16 * wave + r16;
            if (m < rows && n < p.N) {
                const int64_t at = (int64_t)m * p.N + n;
                if (p.y_type == QG_F32)
                    store4<float>(p.Y, at, v, p.N - n, p.vec);
                else if (p.y_type == QG_F16)
                    store4<Fp16>(p.Y, at, v, p.N - n, p.vec);
                else
                    store4<Bf16>(p.Y, at, v, p.N - n, p.vec);
            }
            wait_lds();
        }
        bare_barrier();   // X may be copied into again
        clear();
    };

    // a wave without column blocks multiplies the last one with zero sums: it
    // copies it, like the others, and leaves the products out
    const int batches = max(mine, 1);
    constexpr int kOps = kCopies + 3 + G;   // vector memory operations of a load
    Regs r0, r1;
    clear();
    for (int rg = blockIdx.x; rg < p.row_groups; rg += gridDim.x) {
        load(r0, XA, rg, 0);
        int t = 0;
        for (; t + 2 < batches; t += 2) {
            load(r1, XB, rg, t + 1);
            __builtin_amdgcn_sched_barrier(0);
            wait_vm<kOps>();   // block t is there, block t + 1 in flight
            multiply(r0, XA);
            wait_lds();   // what is copied into has been read
            __builtin_amdgcn_sched_barrier(0);
            load(r0, XA, rg, t + 2);
            __builtin_amdgcn_sched_barrier(0);
            wait_vm<kOps>();
            multiply(r1, XB);
            wait_lds();
            __builtin_amdgcn_sched_barrier(0);
        }
        if (t + 1 < batches) {
            load(r1, XB, rg, t + 1);
            __builtin_amdgcn_sched_barrier(0);
            wait_vm<kOps>();
            multiply(r0, XA);
            wait_vm<0>();
            multiply(r1, XB);
        } else {
            wait_vm<0>();
            if (mine > 0)
                multiply(r0, XA);
        }
        finish(rg, XA);
    }
}

template <int G>
hipError_t launch_lds(SkinnyParams &p, int cus, hipStream_t stream)
{
    p.row_groups = p.rt;
    return launch_kernel(reinterpret_cast<const void *>(&skinny_lds_kernel<G>),
                         dim3((unsigned)std::min(p.rt, cus * (G == 2 ? 2 : 1))), dim3(512), 0, stream, p);
}

template <typename SRC, int NW, int U, bool GROUPED>
hipError_t launch(SkinnyParams &p, int cus, hipStream_t stream)
{
    p.row_groups = p.rt;
    p.units = GROUPED ? f8_units(p.rows.rows, p.rows.P, 16) : 1;
    const size_t lds = (size_t)2 * NW * 1024 + (sizeof(SRC) == 1 ? 0 : (size_t)p.cb * (1024 + 8));
    const void *fn = reinterpret_cast<const void *>(&skinny_kernel<SRC, NW, U, GROUPED>);
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
        if (e != hipSuccess)
            return e;
    }
    const int64_t items = p.units * p.row_groups;
    const int64_t most = GROUPED ? (int64_t)1 << 22 : 3LL * cus;
    return launch_kernel(fn, dim3((unsigned)std::min(items, most)), dim3(64 * NW), lds, stream, p);
}

}  // namespace

hipError_t launch_f8_skinny(const uint8_t *W, const uint8_t *xq, const void *x, int x_type, void *Y, int y_type,
                            const F8Rows &r, int64_t N, int64_t K, int cus, hipStream_t stream)
{
    const F8Weights f = f8_weights(N, K);
    const F8Acts a = f8_acts(r.x_rows, K);
    SkinnyParams p{W, xq, x, Y, r, f.scales, a.scales, 1, (int)N, (int)K, f.cb, f.ls, a.ls, f.rt, 0, y_type, N % 4 == 0 && (reinterpret_cast<uintptr_t>(Y) & (4 * type_bytes(y_type) - 1)) == 0};
    if (x)
        return x_type == QG_F32   ? launch<float, 8, 2, false>(p, cus, stream)
               : x_type == QG_F16 ? launch<Fp16, 8, 2, false>(p, cus, stream)
                                  : launch<Bf16, 8, 2, false>(p, cus, stream);
    if (r.order)
        return launch<Packed, 4, 1, true>(p, cus, stream);
    if (r.rows <= 16)
        return launch<Packed, 8, 2, false>(p, cus, stream);
    if (r.rows <= 32)
        return launch_lds<2>(p, cus, stream);
    return launch_lds<4>(p, cus, stream);
}

}  // namespace qg
