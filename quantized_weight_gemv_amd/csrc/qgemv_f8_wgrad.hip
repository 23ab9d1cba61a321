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
// A workgroup of 2 x 2 waves owns a tile of 64 TN rows x 64 TM columns of dW.
// A step is 32 rows of both operands; dY's go straight from memory into LDS.
// A ring of four buffers: during step t the products run on operands read
// from buffers t and t + 1 (16 rows ahead), X's codes of step t + 3 are
// widened into their buffer, dY's copies of step t + 3 and the loads of X's
// codes of step t + 5 are issued.  One barrier a step.
// Tiles beyond whole rounds of the card's compute units are split along the
// rows among the units that would be idle; their parts go to the workspace
// and a second kernel adds them in a fixed order (no atomics).
// 8192 x 4096 x 4096, one round of tiles: 226 us, 1.22 PFLOP/s (a library
// product of bf16 operands 1.4, the instruction alone 2.4).  With nothing
// loaded it takes 153, without the widening as well 131, with the products
// alone 127.  8192 x 6144 x 4096: 350 us with the second kernel, of whose 18 us
// it is the rest; the matrix cores are busy 58 % of the waves' time, waves wait
// for loads and barriers 17 %, and a quarter of LDS cycles are conflicts.
// The compiler waits where the kernel does not ask for it: in dense calls it
// widens the scale bytes at the head of each four steps, behind a wait for all
// loads; per expert the slots' numbers are the newest loads when their rows are
// addressed, so every step waits for all of them, and unaligned rows of dY
// branch as well.  64 experts of 2048 x 2048 with 375 slots each take 856 us
// (writing 1.07 GB of dW would take 208), 16 of 4096 x 4096 with 1024 1250 us,
// 0.44 PFLOP/s.  The 256 x 256 form keeps 11 registers in scratch memory,
// outside of the loop.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "qgemv_f8_internal.h"

namespace qg {
namespace {

constexpr int kStep = 32;     // rows per step
constexpr int kThreads = 256;
// Compute units that a round of tiles fills.  Not asked from the device: the
// size of the workspace has to be the same for the query and the call, and the
// order of the sums the same on any device.
constexpr int kCus = 256;
constexpr int kPartRows = 1024;

typedef short s4_t __attribute__((ext_vector_type(4)));
typedef short s8_t __attribute__((ext_vector_type(8)));

struct WgradParams {
    const uint16_t *dY;
    const uint8_t *xq;
    float *dW;
    float *part;          // [split tiles][parts][BN][BK]
    F8Rows rows;
    int64_t x_scales;
    int N, K, cb, x_ls;
    int tiles_n, tiles;   // tiles of one matrix
    int whole;            // dense: tiles that are not split (the first ones)
    int parts;            // of each of the others
    int64_t part_rows;    // rows of a part, a multiple of kStep
    bool accumulate, vec;
};

__device__ const uint4 g_zero = {0u, 0u, 0u, 0u};

__device__ __forceinline__ int seg_at(int row, int seg) { return seg ^ (2 * (row & 3)); }

// ALIGNED: rows of dY start at multiples of 16 bytes and are copied straight
// into LDS; otherwise they go through registers, like X's.
template <int TM, int TN, bool ALIGNED, bool GROUPED>
__global__ __launch_bounds__(kThreads, TM == 4 ? 1 : 2) void wgrad_kernel(WgradParams p)
{
    constexpr int BK = 64 * TM, BN = 64 * TN;
    constexpr int YC = BN / 8, XC = BK / 16;                 // chunks of 16 bytes of a row: dY's, X's codes
    constexpr int NY = YC * kStep / kThreads, NX = XC * kStep / kThreads;   // per thread and step
    __shared__ uint4 Y0[kStep * YC], Y1[kStep * YC], Y2[kStep * YC], Y3[kStep * YC];
    __shared__ uint4 X0[kStep * XC * 2], X1[kStep * XC * 2], X2[kStep * XC * 2], X3[kStep * XC * 2];
    auto ybuf = [&](int q) -> uint4 * { return q == 0 ? Y0 : q == 1 ? Y1 : q == 2 ? Y2 : Y3; };
    auto xbuf = [&](int q) -> uint4 * { return q == 0 ? X0 : q == 1 ? X1 : q == 2 ? X2 : X3; };
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave & 1, wk = wave >> 1;

    // blockIdx.x: dense: the whole tiles, then the others' parts; else
    // (expert, tile)
    int tile, part = -1;
    int64_t r0 = 0, r1 = p.rows.rows;
    float *out = p.dW;
    if constexpr (GROUPED) {
        const int e = blockIdx.x / p.tiles;
        tile = blockIdx.x - e * p.tiles;
        r0 = min(max((int64_t)p.rows.offsets[e], (int64_t)0), p.rows.rows);
        r1 = max(r0, min(max((int64_t)p.rows.offsets[e + 1], (int64_t)0), p.rows.rows));
        if (r0 == r1 && p.accumulate)
            return;
        out += (int64_t)e * p.N * p.K;
    } else {
        tile = blockIdx.x;
        if (tile >= p.whole) {
            part = (tile - p.whole) % p.parts;
            tile = p.whole + (tile - p.whole) / p.parts;
            r0 = min(part * p.part_rows, p.rows.rows);
            r1 = min(r0 + p.part_rows, p.rows.rows);
        }
    }
    const int n0 = (tile % p.tiles_n) * BN, k0 = (tile / p.tiles_n) * BK;

    // Rows are numbered from r0 on, 0 .. count - 1.  Rows past the end become
    // zeros: they lie outside of the buffers that loads are made from.  Rows
    // of an expert are gathered with whole addresses instead; there dY's are
    // read from g_zero and X's codes masked, past the end as well as where a
    // slot names no row.  No branch where dY is copied: the loads of a step stay
    // in one sequence, which the waits below count.
    const int count = (int)(r1 - r0);
    const uint8_t *const dY = reinterpret_cast<const uint8_t *>(p.dY);
    const uint8_t *const zero = reinterpret_cast<const uint8_t *>(&g_zero);
    const int64_t y_bytes = 2LL * p.N, x_bytes = 128LL * p.cb;
    auto pick = [](bool ok, const uint8_t *a, const uint8_t *b) {
        return reinterpret_cast<const uint8_t *>(ok ? reinterpret_cast<uintptr_t>(a) : reinterpret_cast<uintptr_t>(b));
    };
    // this thread's chunks: row inside a step, column
    int y_r[NY], y_n[NY], x_r[NX];
    const uint8_t *y_at[NY];                // dense: row r0 + r; grouped: row 0
    const uint8_t *x_at[NX], *s_at[NX];     // grouped: row 0
#pragma unroll
    for (int i = 0; i < NY; ++i) {
        const int idx = threadIdx.x + kThreads * i, pos = idx % YC;
        y_r[i] = idx / YC;
        y_n[i] = n0 + 8 * (ALIGNED ? 2 * seg_at(y_r[i], pos >> 1) + (pos & 1) : pos);
        y_at[i] = dY + (GROUPED ? 0 : r0 + y_r[i]) * y_bytes + 2LL * y_n[i];
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        const int idx = threadIdx.x + kThreads * i;
        x_r[i] = idx / XC;
        const int col = k0 + 16 * (idx % XC), blk = min(col >> 7, p.cb - 1);
        x_at[i] = p.xq + 128 * blk + (col & 127);
        s_at[i] = p.xq + p.x_scales + blk;
    }
    // dense: the rows m .. m + 31 of `row_bytes` each from `base` (row r0) as a
    // buffer, and this thread's places in it; what it never reads lies beyond
    auto step_rows = [&](const uint8_t *base, int64_t row_bytes, int m) {
        const int left = __builtin_amdgcn_readfirstlane(min(max(count - m, 0), kStep));
        return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base + (left ? m : 0) * row_bytes), (short)0,
                                                 (int)(left * row_bytes), kRsrcWord3);
    };
    const uint8_t *const y_base = dY + r0 * y_bytes, *const x_base = p.xq + r0 * x_bytes,
                         *const s_base = p.xq + p.x_scales + r0 * (int64_t)p.x_ls;
    uint32_t y_off[NY], x_off[NX], s_off[NX];
    if constexpr (!GROUPED) {
#pragma unroll
        for (int i = 0; i < NY; ++i)
            y_off[i] = y_n[i] < p.N ? (uint32_t)(y_r[i] * y_bytes) + 2u * y_n[i] : 0x7FFFFF00u;
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int col = k0 + 16 * ((threadIdx.x + kThreads * i) % XC), blk = min(col >> 7, p.cb - 1);
            x_off[i] = (uint32_t)(x_r[i] * x_bytes) + 128u * blk + (col & 127);
            s_off[i] = (uint32_t)(x_r[i] * p.x_ls) + blk;
        }
    }
    int y_slot[NY], x_slot[NX];   // grouped: slots of the step whose loads come next
    auto load_y_slots = [&](int m) {
        if constexpr (GROUPED) {
#pragma unroll
            for (int i = 0; i < NY; ++i)
                y_slot[i] = p.rows.order[r0 + min(m + y_r[i], count - 1)];
        }
    };
    auto load_x_slots = [&](int m) {
        if constexpr (GROUPED) {
#pragma unroll
            for (int i = 0; i < NX; ++i)
                x_slot[i] = p.rows.order[r0 + min(m + x_r[i], count - 1)];
        }
    };
    auto is_slot = [&](int s) { return (uint32_t)s < (uint32_t)p.rows.rows; };
    auto y_from = [&](int i, int m, bool &ok) -> const uint8_t * {
        ok = (m + y_r[i] < count) & (y_n[i] < p.N);
        if constexpr (GROUPED) {
            ok &= is_slot(y_slot[i]);
            return y_at[i] + (ok ? y_slot[i] : 0) * y_bytes;
        }
        return y_at[i] + m * y_bytes;
    };
    // dY straight into LDS: thread -> (row, 16-byte position)
    auto copy_y = [&](uint4 *Y, int m, int i) {
        if constexpr (!GROUPED) {
            copy16(step_rows(y_base, y_bytes, m), &Y[kThreads * i + 64 * wave], y_off[i], 0);
        } else {
            bool ok;
            const uint8_t *at = y_from(i, m, ok);
            __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)pick(ok, at, zero),
                                             (__attribute__((address_space(3))) void *)&Y[kThreads * i + 64 * wave],
                                             16, 0, 0);
        }
    };
    // or through registers
    uint4 yreg[NY];
    auto load_y = [&](int m) {
#pragma unroll
        for (int i = 0; i < NY; ++i) {
            uint32_t w[4] = {0u, 0u, 0u, 0u};
            bool ok;
            const uint8_t *at = y_from(i, m, ok);
            if (ok) {
                if (y_n[i] + 8 <= p.N) {
                    const Raw16 raw = *reinterpret_cast<const Raw16 *>(at);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = raw.w[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (y_n[i] + e < p.N)
                            w[e / 2] |= (uint32_t) reinterpret_cast<const uint16_t *>(at)[e] << (16 * (e & 1));
                }
            }
            yreg[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    };
    auto store_y = [&](uint4 *Y) {
#pragma unroll
        for (int i = 0; i < NY; ++i) {
            const int ch = (threadIdx.x + kThreads * i) % YC;
            Y[y_r[i] * YC + 2 * seg_at(y_r[i], ch >> 1) + (ch & 1)] = yreg[i];
        }
    };
    // X: thread -> (row, 16 columns); columns past the last block repeat it
    // (never stored)
    struct Codes {   // of a step, in registers from two steps before they go to LDS
        uint4 code[NX];
        uint32_t sbyte[NX], keep[NX];
    };
    auto load_x = [&](Codes &c, int m) {
        if constexpr (!GROUPED) {
            const auto from = step_rows(x_base, x_bytes, m), scales = step_rows(s_base, p.x_ls, m);
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                c.code[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(from, x_off[i], 0, 0));
                c.sbyte[i] = __builtin_amdgcn_raw_buffer_load_b8(scales, s_off[i], 0, 0);
                c.keep[i] = ~0u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                const bool ok = (m + x_r[i] < count) & is_slot(x_slot[i]);
                const int64_t row =
                    min((int64_t)((uint32_t)(ok ? x_slot[i] : 0) / (uint32_t)p.rows.k_slots), p.rows.x_rows - 1);
                c.code[i] = *reinterpret_cast<const uint4 *>(pick(ok, x_at[i] + row * x_bytes, p.xq));
                c.sbyte[i] = *pick(ok, s_at[i] + row * p.x_ls, p.xq);
                c.keep[i] = ok ? ~0u : 0u;
            }
        }
    };
    auto store_x = [&](Codes &c, uint4 *X, int i) {
        const int at = x_r[i] * XC * 2 + 2 * seg_at(x_r[i], (threadIdx.x + kThreads * i) % XC);
        // what was loaded two steps ago is first touched here: without the
        // pin its users move up behind the load and wait for it there
        asm volatile("" : "+v"(c.sbyte[i]), "+v"(c.code[i].x), "+v"(c.code[i].y), "+v"(c.code[i].z),
                     "+v"(c.code[i].w));
        const uint32_t k = c.keep[i];   // a masked row's byte is any byte: not the scale of its zeros
        const float s = f8_exponent(c.sbyte[i] & k);
        X[at] = __builtin_bit_cast(uint4, f8_widen(c.code[i].x & k, c.code[i].y & k, s));
        X[at + 1] = __builtin_bit_cast(uint4, f8_widen(c.code[i].z & k, c.code[i].w & k, s));
    };
    // eight consecutive rows 16 h + 8 (lane / 32) .. of column 32 t + lane % 32
    auto operand = [&](const uint4 *S, int row_bytes, int h, int t) -> bf8_t {
        const int i = lane & 15;
        const int seg = 2 * t + ((lane >> 4) & 1);
        const char *base = reinterpret_cast<const char *>(S);
        s4_t v[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
            const int row = 16 * h + 8 * (lane >> 5) + 4 * o + (i >> 2);
            v[o] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4_t *)(
                base + row * row_bytes + 32 * seg_at(row, seg) + 8 * (i & 3)));
        }
        const s8_t w = __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(bf8_t, w);
    };
    struct Operands {
        bf8_t x[TM], y[TN];
    };
    // the o-th operand of a half, dY's first: every product of the next half's
    // first row takes them all
    auto read = [&](Operands &to, const uint4 *X, const uint4 *Y, int h, int o) {
        if (o < TN)
            to.y[o] = operand(Y, YC * 16, h, wn * TN + o);
        else
            to.x[o - TN] = operand(X, XC * 32, h, wk * TM + o - TN);
    };

    f16v_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[i][j][e] = 0.0f;
    // The products of half a step, a row of them at a time, with the reads of
    // the next half's operands and a share of the other work in front of each:
    // left to itself the compiler gathers the reads at the end and waits there
    auto half = [&](const Operands &now, Operands &next, const uint4 *X, const uint4 *Y, int h, auto work) {
        static_assert(TM == TN && NY == TM && NX <= TM, "");
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            read(next, X, Y, h, 2 * i);
            read(next, X, Y, h, 2 * i + 1);
            work(i);
#pragma unroll
            for (int j = 0; j < TN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(now.x[i], now.y[j], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };

    if (r0 < r1) {
        // Vector memory operations of a step (a lower bound): what may still
        // be in flight when the copies issued a step earlier, and all before
        // them, have to have landed.
        constexpr int kOps = (ALIGNED ? NY : 0) + 2 * NX;
        auto fill = [&](int q) {   // before the loop: buffer q
            load_y_slots(q * kStep);
            load_x_slots(q * kStep);
            if constexpr (!ALIGNED)
                load_y(q * kStep);
            Codes c;
            load_x(c, q * kStep);
            if constexpr (!ALIGNED)
                store_y(ybuf(q));
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                if constexpr (ALIGNED)
                    copy_y(ybuf(q), q * kStep, i);
                if (i < NX)
                    store_x(c, xbuf(q), i);
            }
        };
        fill(0);
        fill(1);
        fill(2);
        // in registers at the start of a step that multiplies rows m ..: X's
        // codes of m + 3 and m + 4 steps (and dY's, unaligned, of m + 3), the
        // slots of what is loaded next
        Codes c0, c1;
        load_x_slots(3 * kStep);
        load_x(c0, 3 * kStep);
        load_x_slots(4 * kStep);
        load_x(c1, 4 * kStep);
        load_x_slots(5 * kStep);
        load_y_slots(3 * kStep);
        if constexpr (!ALIGNED) {
            load_y(3 * kStep);
            load_y_slots(4 * kStep);
        }
        Operands first, second;
        wait_vm_lds<0>();
        bare_barrier();
#pragma unroll
        for (int o = 0; o < TM + TN; ++o)
            read(first, X0, Y0, 0, o);
        auto step = [&](int m, auto number) {
            constexpr int q = decltype(number)::value;
            wait_vm_lds<kOps>();   // and this wave's LDS writes are done
            bare_barrier();
            // buffer (q + 3) % 4 was last read in the step before
            half(first, second, xbuf(q), ybuf(q), 1, [&](int i) {
                if constexpr (ALIGNED) {
                    copy_y(ybuf((q + 3) & 3), m + 3 * kStep, i);
                    if (i == TM - 1)
                        load_y_slots(m + 4 * kStep);
                } else if (i == 0) {
                    store_y(ybuf((q + 3) & 3));
                    load_y(m + 4 * kStep);
                    load_y_slots(m + 5 * kStep);
                }
                if (i >= TM - NX)
                    store_x(q & 1 ? c1 : c0, xbuf((q + 3) & 3), i - (TM - NX));
            });
            half(second, first, xbuf((q + 1) & 3), ybuf((q + 1) & 3), 0, [&](int i) {
                if (i == 0) {
                    load_x(q & 1 ? c1 : c0, m + 5 * kStep);
                    load_x_slots(m + 6 * kStep);
                }
            });
        };
        // whole rounds of four steps: rows past the end are zeros
        for (int m = 0; m < count; m += 4 * kStep) {
            step(m, std::integral_constant<int, 0>{});
            step(m + kStep, std::integral_constant<int, 1>{});
            step(m + 2 * kStep, std::integral_constant<int, 2>{});
            step(m + 3 * kStep, std::integral_constant<int, 3>{});
        }
    }

    // lane: column n of dY (lane % 32), four consecutive k each
    float *tile_out = part < 0 ? nullptr
                               : p.part + ((int64_t)(tile - p.whole) * p.parts + part) * BN * BK;
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int nn = (wn * TN + j) * 32 + (lane & 31);
        if (n0 + nn >= p.N)
            continue;
        float *row = out + (int64_t)(n0 + nn) * p.K;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int kk = (wk * TM + i) * 32 + 8 * g + 4 * (lane >> 5);
                const int k = k0 + kk;
                f4_t w = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
                if (part >= 0) {
                    *reinterpret_cast<f4_t *>(tile_out + nn * BK + kk) = w;
                } else if (p.vec && k + 4 <= p.K) {
                    if (p.accumulate)
                        w += *reinterpret_cast<const f4_t *>(row + k);
                    *reinterpret_cast<f4_t *>(row + k) = w;
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (k + e < p.K)
                            row[k + e] = w[e] + (p.accumulate ? row[k + e] : 0.0f);
                }
            }
    }
}

struct JoinParams {
    const float *part;
    float *dW;
    int N, K, size, tiles_n, whole, parts;
    bool accumulate, vec;
};

// A workgroup per 1024 values of a split tile, four columns of a row per lane.
__global__ __launch_bounds__(256) void join_kernel(JoinParams p)
{
    const int groups = p.size * p.size / 1024;
    const int tile = blockIdx.x / groups, at = (blockIdx.x % groups) * 1024 + 4 * threadIdx.x;
    const int n = ((p.whole + tile) % p.tiles_n) * p.size + at / p.size;
    const int k = ((p.whole + tile) / p.tiles_n) * p.size + at % p.size;
    if (n >= p.N || k >= p.K)
        return;
    const float *from = p.part + (int64_t)tile * p.parts * p.size * p.size + at;
    float *to = p.dW + (int64_t)n * p.K + k;
    f4_t v = {0, 0, 0, 0};
    if (p.accumulate) {
        if (p.vec) {
            v = *reinterpret_cast<const f4_t *>(to);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = k + e < p.K ? to[e] : 0.0f;
        }
    }
    for (int s = 0; s < p.parts; ++s)
        v += *reinterpret_cast<const f4_t *>(from + (int64_t)s * p.size * p.size);
    if (p.vec) {   // K is a multiple of four
        *reinterpret_cast<f4_t *>(to) = v;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (k + e < p.K)
                to[e] = v[e];
    }
}

// How a dense dW is cut.  Tiles of 256 x 256 where they fill most of a round
// of compute units, else of 128 x 128, two to a unit.  The tiles beyond whole
// rounds are cut along the rows in as many parts as idle units allow: 8192 x
// 6144 x 4096 takes 350 us for 389 without, 16384 x 1024 x 1024 53 for 169, 4096
// x 1024 x 1024 29 for 47.  A part has at least 1024 rows, since the parts' way
// through memory and the second launch cost more than they save on fewer: 1024
// x 2048 x 2048 takes 21 us whole and 35 in parts of 512 rows.  Two parts of
// little more than that gain with few tiles (2048 x 1024 x 1024 23 us for 26)
// and lose with many (2048 x 2048 x 2048 39 for 32, 3000 x 2048 x 2048 46 for 42;
// from 4096 rows on they are even or gain).
struct Cut {
    int size, tiles_n, tiles, whole, parts;
};

Cut cut_of(int64_t M, int64_t N, int64_t K)
{
    Cut c;
    c.size = ceil_div(N, 256) * ceil_div(K, 256) >= kCus * 3 / 4 ? 256 : 128;
    c.tiles_n = (int)ceil_div(N, c.size);
    c.tiles = (int)(c.tiles_n * ceil_div(K, c.size));
    const int round = c.size == 256 ? kCus : 2 * kCus;   // two workgroups of the small tiles a unit
    const int rest = c.tiles % round;
    c.parts = rest ? (int)std::min<int64_t>(round / rest, M / kPartRows) : 1;
    if (c.parts < 2)
        c.parts = 1;
    c.whole = c.parts > 1 ? c.tiles - rest : c.tiles;
    return c;
}

template <int T, bool GROUPED>
hipError_t launch(const WgradParams &p, int64_t wgs, hipStream_t stream)
{
    const bool al = p.N % 8 == 0 && (reinterpret_cast<uintptr_t>(p.dY) & 15) == 0;
    const void *fn = al ? reinterpret_cast<const void *>(&wgrad_kernel<T, T, true, GROUPED>)
                        : reinterpret_cast<const void *>(&wgrad_kernel<T, T, false, GROUPED>);
    return launch_kernel(fn, dim3((unsigned)wgs), dim3(kThreads), 0, stream, p);
}

}  // namespace

size_t f8_wgrad_workspace(int64_t M, int64_t N, int64_t K)
{
    const Cut c = cut_of(M, N, K);
    return (size_t)(c.tiles - c.whole) * c.parts * c.size * c.size * sizeof(float);
}

hipError_t launch_f8_wgrad(const uint16_t *dY, const uint8_t *xq, float *dW, bool accumulate, const F8Rows &r,
                           int64_t N, int64_t K, float *workspace, hipStream_t stream)
{
    const F8Acts a = f8_acts(r.x_rows, K);
    WgradParams p{dY, xq, dW, workspace, r, a.scales, (int)N, (int)K, a.cb, a.ls, 0, 0, 0, 1, r.rows, accumulate,
                  K % 4 == 0 && (reinterpret_cast<uintptr_t>(dW) & 15) == 0};
    if (r.order) {
        p.tiles_n = (int)ceil_div(N, 128);
        p.tiles = (int)(p.tiles_n * ceil_div(K, 128));
        return launch<2, true>(p, (int64_t)r.P * p.tiles, stream);
    }
    const Cut c = cut_of(r.rows, N, K);
    p.tiles_n = c.tiles_n, p.tiles = c.tiles, p.whole = c.whole, p.parts = c.parts;
    p.part_rows = ceil_div(ceil_div(r.rows, c.parts), kStep) * kStep;
    const int64_t wgs = c.whole + (int64_t)(c.tiles - c.whole) * c.parts;
    const hipError_t e = c.size == 256 ? launch<4, false>(p, wgs, stream) : launch<2, false>(p, wgs, stream);
    if (e != hipSuccess || c.whole == c.tiles)
        return e;
    const JoinParams j{workspace, dW, (int)N, (int)K, c.size, c.tiles_n, c.whole, c.parts, accumulate, p.vec};
    return launch_kernel(reinterpret_cast<const void *>(&join_kernel),
                         dim3((unsigned)((c.tiles - c.whole) * (c.size * c.size / 1024))), dim3(256), 0, stream, j);
}

}  // namespace qg
