// f8 products of many rows: Y[m][n] = sum_k X[m][k] W[n][k] on the matrix
// cores, for one matrix or for the slots of each expert of a pool.
//
// A workgroup of 2 x 2 waves owns a tile of BM rows of X times BN rows of W.
// A step is 64 columns (half a block: one scale byte a
// row and side); its operands go straight from memory into LDS (buffer loads
// that write LDS: no registers, and what lies past an edge reads as zero):
//   * X, row-major, a block of 128 columns at a time: rows of 128 bytes, whole
//     lines (the caches deliver 30 TB/s to loads of 8 rows x 128 bytes and 9.5
//     to loads of 16 rows x 64 bytes), 16-byte chunk c of row r at position
//     c ^ ((r / 2) % 8), so that the 16 rows of a quarter of an operand read
//     touch all 64 banks;
//   * W, whose tiles are in operand order already: copied as they are, a step
//     at a time; an operand read is 256 consecutive bytes a quarter wave.
// X has D buffers (blocks), W 2 D (steps).  During step t the matrix cores
// multiply operands that were read from LDS during step t - 1, the operands of
// t + 1 are read, W's copies of step t + 2 D - 1 are issued into the buffer
// that step t - 2 read and, in a block's second step, X's copies of the block D
// further on into the one that step t - 1 read last.  One barrier a step;
// before it a wave waits for those of its own copies that step t reads and for
// its LDS reads, so that behind it every buffer's readers are done.  K takes
// whole rounds of D blocks; blocks past it are read as zeros.
// The codes are widened to bf16 with their scale (exact) and multiplied with
// v_mfma_f32_32x32x16_bf16, whatever the type of the outputs: products are
// exact and sums are fp32 sums.  The 8-bit instruction with the block scales as
// operands runs twice as fast, but it aligns neighbouring products to the
// largest of them and keeps about 13 bits below it: where products of 2^16
// cancel, it loses up to a tenth of the sum of 200 others of 1 to 6.
// W is the first operand, so a lane holds four consecutive n of a row of Y;
// the sums are turned through LDS for stores of whole lines.
// Bound by the matrix cores on large products: 8192 x 14336 x 4096 takes 671 to
// 710 us with bf16 outputs, 1.36 to 1.43 PFLOP/s, and 720 with fp32 (a library
// product of bf16 operands 1.41 PFLOP/s, the instruction alone, on registers,
// 2.4): they are busy 70 % of the time, at 1.9 GHz under that load; 2048 x 8192 x
// 4096 104 us.  Short products wait for their chain of steps: with one wave a SIMD
// (733 x 2053 x 5011, 29 us) a step of 64 columns takes 720 cycles, of which the
// products are 250, the widening beside them 240.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "qgemv_f8_internal.h"

namespace qg {
namespace {

struct GemmParams {
    const uint8_t *W, *xq;
    void *Y;
    F8Rows rows;
    int64_t w_scales, x_scales;
    uint32_t units;      // tiles along the rows (grouped: an upper bound)
    int N, cb, x_ls, w_ls, rt, tiles_n;
    bool vec;
};

// Tile shape: 2 x 2 waves, each 32 TM rows of X times 32 TN rows of W.
template <int TM, int TN>
struct Tile {
    static constexpr int BM = 64 * TM, BN = 64 * TN, NT = 256;
    static constexpr int XC = BM * 8 / NT, WC = BN * 4 / NT;   // 16-byte copies per thread: X's a block, W's a step
};

// Which tile a workgroup takes.  Workgroups go to the eight XCDs in turn, each
// with an L2 of its own: an XCD gets a contiguous share of the tiles.  Dense
// tiles are numbered in bands of kBand tiles of rows of X, so that those that
// are worked on at a time share rows of both operands.  Grouped tiles are
// numbered expert by expert, an expert's tiles of slots innermost: they read
// the same rows of W and start together, so that W comes into the L2 once.
constexpr uint32_t kXcds = 8, kBand = 8;

__device__ __forceinline__ bool place_of(uint32_t total, uint32_t &lin)
{
    const uint32_t share = (total + kXcds - 1) / kXcds;
    lin = blockIdx.x % kXcds * share + blockIdx.x / kXcds;
    return blockIdx.x / kXcds < share && lin < total;
}

__device__ __forceinline__ void dense_tile(uint32_t lin, uint32_t units, int tiles_n, uint32_t &unit, int &tn)
{
    const uint32_t band = lin / (uint32_t)(kBand * tiles_n);
    const uint32_t in = lin - band * kBand * tiles_n;
    const uint32_t rows = min(kBand, units - band * kBand);
    tn = (int)(in / rows);
    unit = band * kBand + (in - (uint32_t)tn * rows);
}

typedef uint32_t Words __attribute__((ext_vector_type(4)));

// Buffers that loads are made from: base and size of what they may read.
struct Source {
    const uint8_t *base;
    uint32_t bytes;
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const Source &s)
{
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(s.base), (short)0, (int)s.bytes, kRsrcWord3);
}

template <int TM, int TN, int D, typename OUT, bool GROUPED>
__global__ __launch_bounds__(256, TM *TN *D > 16 || D == 4 ? 1 : 2) void gemm_kernel(GemmParams p)
{
    using T = Tile<TM, TN>;
    // one variable a buffer: the compiler then knows which copies an operand
    // read has to wait for (none: the waits are the kernel's own)
    static_assert(D == 2 || D == 4, "");
    constexpr int kX = T::BM * 8, kW = T::BN * 4;   // 16-byte chunks of a buffer
    __shared__ uint4 X0[kX], X1[kX], X2[D > 2 ? kX : 1], X3[D > 2 ? kX : 1];
    __shared__ uint4 W0[kW], W1[kW], W2[kW], W3[kW];
    __shared__ uint4 W4[D > 2 ? kW : 1], W5[D > 2 ? kW : 1], W6[D > 2 ? kW : 1], W7[D > 2 ? kW : 1];
    constexpr int JN = sizeof(OUT) == 4 ? TN / 2 : TN;   // column tiles that are staged at a time
    constexpr bool kOwnStage = 4 * 32 * 32 * JN * (int)sizeof(OUT) > T::BM * 128;
    __shared__ uint4 stages[kOwnStage ? 4 * 2 * 32 * JN * (int)sizeof(OUT) : 1];
    __shared__ int out_row[GROUPED ? T::BM : 1];
    auto xbuf = [&](int q) -> uint4 * { return q == 0 ? X0 : q == 1 ? X1 : q == 2 ? X2 : X3; };
    auto wbuf = [&](int q) -> uint4 * {
        return q == 0 ? W0 : q == 1 ? W1 : q == 2 ? W2 : q == 3 ? W3 : q == 4 ? W4 : q == 5 ? W5 : q == 6 ? W6 : W7;
    };

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int r32 = lane & 31, half = lane >> 5;
    const int64_t ld = 128LL * p.cb;

    // ---- the tile
    uint32_t unit = 0, lin;
    int tn = 0;
    if (!place_of(p.units * p.tiles_n, lin))
        return;
    F8Unit u{0, 0, 0, 0, 1, 0, 0};
    if constexpr (GROUPED) {
        u = f8_unit(p.rows.offsets, p.rows.P, p.rows.rows, T::BM, lin / (uint32_t)p.tiles_n);
        if (u.r0 >= u.r1)
            return;   // past the last unit (uniform over the workgroup)
        const uint32_t local = lin - (uint32_t)u.first * p.tiles_n;
        tn = (int)(local / (uint32_t)u.tiles);
        f8_tile_of(u, local - tn * u.tiles, T::BM);
    } else {
        dense_tile(lin, p.units, p.tiles_n, unit, tn);
    }
    const int n0 = tn * T::BN;
    const int64_t m0 = (int64_t)unit * T::BM;

    // ---- where its operands are
    const uint8_t *const Wm = p.W + (GROUPED ? min(u.e, p.rows.P - 1) * p.rows.stride : 0);
    const int64_t x_rows = GROUPED ? p.rows.x_rows : min((int64_t)T::BM, p.rows.rows - m0);
    const Source x_src{p.xq + m0 * ld, (uint32_t)(x_rows * ld)};
    const Source xs_src{p.xq + p.x_scales + m0 * p.x_ls, (uint32_t)(x_rows * p.x_ls)};
    const int rt0 = n0 / 16;
    const Source w_src{Wm + (int64_t)rt0 * p.cb * 2048, (uint32_t)(min(T::BN / 16, p.rt - rt0) * p.cb * 2048)};
    static_assert(128 % (32 * TN) == 0, "a wave's rows of W lie in one block");
    const Source ws_src{Wm + p.w_scales + (int64_t)min((n0 + wn * TN * 32) >> 7, (p.N - 1) >> 7) * p.w_ls,
                        (uint32_t)p.w_ls};
    uint32_t ws_at = 0;
    asm("" : "+v"(ws_at));   // a lane's own: a word known to be the wave's would go to a scalar register, behind a wait
    // this thread's places in them
    uint32_t x_at[T::XC], w_at[T::WC], xs_at[TM];
    auto row_at = [&](int r) -> uint32_t {   // grouped: the row of X of a row of the tile; past its end: none
        if constexpr (!GROUPED)
            return (uint32_t)r;
        const int64_t at = u.r0 + r;
        const int s = at < u.r1 ? p.rows.order[at] : -1;
        return s >= 0 && s < p.rows.rows ? min((uint32_t)s / (uint32_t)p.rows.k_slots, (uint32_t)p.rows.x_rows - 1)
                                         : (uint32_t)p.rows.x_rows;
    };
    // (a row past the end: beyond the buffer, whose loads return zeros)
#pragma unroll
    for (int i = 0; i < T::XC; ++i) {
        const int idx = threadIdx.x + T::NT * i;
        const int r = idx >> 3, ch = (idx & 7) ^ ((r >> 1) & 7);
        x_at[i] = (uint32_t)(min((int64_t)row_at(r) * ld, (int64_t)0xFFFFFF00 - ld) + ch * 16);
    }
#pragma unroll
    for (int i = 0; i < T::WC; ++i) {
        const int idx = threadIdx.x + T::NT * i;
        w_at[i] = (uint32_t)((idx >> 6) * p.cb * 2048 + (idx & 63) * 16);
    }
#pragma unroll
    for (int i = 0; i < TM; ++i)
        xs_at[i] = (uint32_t)min((int64_t)row_at((wm * TM + i) * 32 + r32) * p.x_ls, (int64_t)0xFFFFFF00 - p.x_ls);
    if constexpr (GROUPED) {
        for (int r = threadIdx.x; r < T::BM; r += T::NT) {
            const int s = u.r0 + r < u.r1 ? p.rows.order[u.r0 + r] : -1;
            out_row[r] = s >= 0 && s < p.rows.rows ? s : -1;
        }
        __syncthreads();
    }

    // ---- the sums
    f16v_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[i][j][e] = 0.0f;
    // A wave's store of what its lanes hold would touch 32 rows.  So 32 rows x
    // 32 JN columns at a time go through LDS (wave-private, in X0 where it is
    // large enough; 16-byte chunks swizzled by row).
    constexpr int kRow = 32 * JN * (int)sizeof(OUT), kChunks = kRow / 16, kPer = 16 / (int)sizeof(OUT);
    constexpr int kStores = 32 * kChunks / 64;
    auto write = [&] {
        uint4 *stage = (kOwnStage ? stages : X0) + wave * (32 * kChunks);
        char *bytes = reinterpret_cast<char *>(stage);
        const bool whole = p.vec && n0 + T::BN <= p.N && (GROUPED || m0 + T::BM <= p.rows.rows);   // no edge
#pragma unroll
        for (int part = 0; part < TM * TN / JN; ++part) {
            const int i = part / (TN / JN), j0 = part % (TN / JN) * JN;
#pragma unroll
            for (int j = 0; j < JN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int at = (32 * j + 8 * g + 4 * half) * (int)sizeof(OUT);
                    char *to = bytes + r32 * kRow + (((at >> 4) ^ (r32 & (kChunks - 1))) << 4) + (at & 15);
                    const f16v_t &a = acc[i][j0 + j];
                    if constexpr (sizeof(OUT) == 4)
                        *reinterpret_cast<f4_t *>(to) = f4_t{a[4 * g], a[4 * g + 1], a[4 * g + 2], a[4 * g + 3]};
                    else
                        *reinterpret_cast<uint2 *>(to) =
                            make_uint2(pack2<OUT>(a[4 * g], a[4 * g + 1]), pack2<OUT>(a[4 * g + 2], a[4 * g + 3]));
                }
            // the c-th chunk of this lane: its row and column in the tile
            auto row_of = [&](int c) { return (wm * TM + i) * 32 + (64 * c + lane) / kChunks; };
            auto chunk_of = [&](int c) {
                const int r = (64 * c + lane) / kChunks, ch = (64 * c + lane) % kChunks;
                return stage[r * kChunks + (ch ^ (r & (kChunks - 1)))];
            };
            const int n = n0 + (wn * TN + j0) * 32 + lane % kChunks * kPer;   // 64 is a multiple of kChunks
            if (whole) {
                uint4 v[kStores];
#pragma unroll
                for (int c = 0; c < kStores; ++c)
                    v[c] = chunk_of(c);
#pragma unroll
                for (int c = 0; c < kStores; ++c) {
                    const int64_t y = GROUPED ? out_row[row_of(c)] : m0 + row_of(c);
                    if (!GROUPED || y >= 0)
                        *reinterpret_cast<uint4 *>(static_cast<OUT *>(p.Y) + y * p.N + n) = v[c];
                }
                continue;
            }
#pragma unroll 1
            for (int c = 0; c < kStores; ++c) {
                const int m = row_of(c);
                const uint4 v = chunk_of(c);
                const int64_t y = GROUPED ? out_row[m] : m0 + m < p.rows.rows ? m0 + m : -1;
                if (y < 0 || n >= p.N)
                    continue;
                OUT *to = static_cast<OUT *>(p.Y) + y * p.N + n;
                if (p.vec) {   // N is a multiple of a chunk
                    *reinterpret_cast<uint4 *>(to) = v;
                    continue;
                }
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (n + e < p.N) {
                        if constexpr (sizeof(OUT) == 4)
                            to[e] = __uint_as_float(w[e]);
                        else
                            to[e] = OUT{(uint16_t)(w[e / 2] >> (16 * (e & 1)))};
                    }
            }
        }
    };
    if (GROUPED && u.e >= p.rows.P) {   // slots without an expert: zeros
        write();
        return;
    }

    // ---- copies: the next block of X and step of W; past K nothing is read
    // and LDS gets zeros.  No branches: the products of a step would be moved
    // across them
    const int blocks = (p.cb + D - 1) / D * D;
    int x_ahead = 0, w_ahead = 0;
    auto copy_x = [&](uint4 *X) {
        const auto r = rsrc_of(Source{x_src.base, x_ahead < p.cb ? x_src.bytes : 0});
#pragma unroll
        for (int i = 0; i < T::XC; ++i)
            copy16(r, &X[T::NT * i + 64 * wave], x_at[i], x_ahead * 128);
        ++x_ahead;
    };
    auto copy_w = [&](uint4 *Wb) {
        const auto r = rsrc_of(Source{w_src.base, w_ahead < 2 * p.cb ? w_src.bytes : 0});
#pragma unroll
        for (int i = 0; i < T::WC; ++i)
            copy16(r, &Wb[T::NT * i + 64 * wave], w_at[i], w_ahead * 1024);
        ++w_ahead;
    };
    // scales: four blocks' bytes a word
    uint32_t xs[TM], ws, xword[TM], wword, xs_next[TM], ws_next;
    auto load_scales = [&](int word) {
        const auto r = rsrc_of(xs_src);
#pragma unroll
        for (int i = 0; i < TM; ++i)
            xs_next[i] = __builtin_amdgcn_raw_buffer_load_b32(r, xs_at[i], 4 * word, 0);
        ws_next = __builtin_amdgcn_raw_buffer_load_b32(rsrc_of(ws_src), ws_at, 4 * word, 0);
    };
    // (one load of 16 bytes: taken word by word, the compiler loses track of the
    // buffer that some of them are from and waits for every copy)
    struct Operands {
        Words x[TM][2], w[TN][2];
    };
    auto read = [&](Operands &o, const uint4 *X, int h, const uint4 *Wb) {   // h: half of X's block
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int ch = 2 * half + q;
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int r = (wm * TM + i) * 32 + r32;
                o.x[i][q] = *reinterpret_cast<const Words *>(&X[r * 8 + ((4 * h + ch) ^ ((r >> 1) & 7))]);
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int t = (wn * TN + j) * 2 + (r32 >> 4);
                o.w[j][q] = *reinterpret_cast<const Words *>(&Wb[t * 64 + ch * 16 + (r32 & 15)]);
            }
        }
    };
    auto multiply = [&](const Operands &o) {
        const float wf = f8_exponent(ws & 255u);
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                bf8_t w[TN];
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    w[j] = h ? f8_widen(o.w[j][q].z, o.w[j][q].w, wf) : f8_widen(o.w[j][q].x, o.w[j][q].y, wf);
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const float xf = f8_exponent(xs[i] & 255u);
                    const bf8_t x =
                        h ? f8_widen(o.x[i][q].z, o.x[i][q].w, xf) : f8_widen(o.x[i][q].x, o.x[i][q].y, xf);
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[j], x, acc[i][j], 0, 0, 0);
                }
            }
    };

    // Copies that may be in flight behind what a step waits for: those of the
    // 2 D - 3 steps before it, of which an even step has D - 1 with X's among
    // them, an odd one D - 2.  (The loads of a round's scales are not counted,
    // so the second step of a round waits for up to TM + 1 operations more.)
    constexpr int kEven = (2 * D - 3) * T::WC + (D - 1) * T::XC, kOdd = (2 * D - 3) * T::WC + (D - 2) * T::XC;
    constexpr int kFirst = (2 * D - 2) * T::WC + (D - 1) * T::XC;
    Operands even, odd;
    // step q of a round of D blocks, the first of which is b
    auto step = [&](int b, auto number) {
        constexpr int q = decltype(number)::value;
        wait_vm_lds<q & 1 ? kOdd : kEven>();   // the reads of step t - 1 as well: an odd step copies over them
        bare_barrier();
        if constexpr (q == 0) {
            // the scales of a round are loaded a round ahead
#pragma unroll
            for (int i = 0; i < TM; ++i)
                xword[i] = xs_next[i];
            wword = ws_next;
            load_scales(min((b + D) / 4, p.x_ls / 4 - 1));
        }
        if constexpr ((q & 1) == 0) {
            const int at = b + q / 2;   // blocks past K: zeros, with a scale that is a number
#pragma unroll
            for (int i = 0; i < TM; ++i)
                xs[i] = at < p.cb ? xword[i] >> (8 * (at & 3)) : 127u;
            ws = at < p.cb ? wword >> (8 * (at & 3)) : 127u;
        }
        read(q & 1 ? even : odd, xbuf((q + 1) % (2 * D) >> 1), (q + 1) & 1, wbuf((q + 1) % (2 * D)));
        if constexpr (q & 1)
            copy_x(xbuf(q >> 1));
        copy_w(wbuf((q + 2 * D - 1) % (2 * D)));
        multiply(q & 1 ? odd : even);
        // both behind the first products: left alone they gather at the end of
        // the step
        constexpr int kProducts = 4 * TM * TN, kReads = 2 * (TM + TN), kCopies = T::WC + (q & 1 ? T::XC : 0);
#pragma unroll
        for (int m = 0; m < kProducts; ++m) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one MFMA
            if (m < kReads)
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // an LDS read
            else if (m < kReads + kCopies)
                __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);   // a copy
        }
    };
    // what the 2 D - 1 steps before the first one would have copied
    load_scales(0);
#pragma unroll
    for (int s = 0; s < 2 * D - 1; ++s) {
        if ((s & 1) == 0)
            copy_x(xbuf(s / 2));
        copy_w(wbuf(s));
    }
    wait_vm<kFirst>();
    bare_barrier();
    read(even, X0, 0, W0);
    for (int b = 0; b < blocks; b += D) {
        step(b, std::integral_constant<int, 0>{});
        step(b, std::integral_constant<int, 1>{});
        step(b, std::integral_constant<int, 2>{});
        step(b, std::integral_constant<int, 3>{});
        if constexpr (D == 4) {
            step(b, std::integral_constant<int, 4>{});
            step(b, std::integral_constant<int, 5>{});
            step(b, std::integral_constant<int, 6>{});
            step(b, std::integral_constant<int, 7>{});
        }
    }
    wait_vm_lds<0>();   // no copy and no read is in flight when X0 is used for staging
    bare_barrier();
    write();
}

template <int TM, int TN, int D, typename OUT, bool GROUPED>
hipError_t launch(GemmParams &p, hipStream_t stream)
{
    using T = Tile<TM, TN>;
    p.tiles_n = (int)ceil_div(p.N, T::BN);
    p.units = (uint32_t)(GROUPED ? f8_units(p.rows.rows, p.rows.P, T::BM) : ceil_div(p.rows.rows, T::BM));
    const int64_t items = (int64_t)p.units * p.tiles_n;
    if (ceil_div(items, kXcds) * kXcds >= 1 << 24)   // a grid holds fewer than 2^32 threads
        return hipErrorInvalidValue;
    return launch_kernel(reinterpret_cast<const void *>(&gemm_kernel<TM, TN, D, OUT, GROUPED>),
                         dim3((unsigned)(ceil_div(items, kXcds) * kXcds)), dim3(T::NT), 0, stream, p);
}

// Tiles.  Large ones need fewer bytes from the caches, small ones fill the card;
// with few tiles it is rounds of them over the compute units that count.  Time
// of a round at K 4096 (us, any output type):
//   256 x 256, two blocks in flight, one a unit        103
//   128 x 128, two blocks, two a unit                  55, or 35 if half is empty
//   128 x 128, four blocks, one a unit                 30
//   64 x 128, four blocks, one a unit                  20
// The shape whose rounds add up to the least is taken.  Measured (us, in that
// order, bf16 out): 8192 x 14336 671 / 739 / 788 / 1073; 2048 x 8192 104 / 110 /
// 114 / 154; 1536 x 6144 78 / 78 / 79 / 94; 2304 x 8192 170 / 131 / 134 / 172;
// 1024 x 6144 76 / 50 / 52 / 60; 1024 x 4096 76 / 35 / 31 / 43; 640 x 4096 78 / 32
// / 26 / 39; 512 x 4096 75 / 30 / 26 / 23; fp32: 8192 x 14336 720 / 780 / 842 /
// 1053, 2304 x 8192 184 / 137 / 138 / 172, 640 x 4096 83 / 33 / 27 / 38.  At K 512
// rounds cost 21, 10 or 8, 7 and 4.5; the rule takes the best there or one up to
// 8 % slower (8192 x 4096: 41 / 38 / 52 / 67; 1024 x 4096: 16 / 8.2 / 8.7 / 11).
// Experts: 128 x 128, and 256 x 256 where they have 2048 slots each on average.
// 128 x 128 / 256 x 256, uneven experts (us), bf16 out: 64 of 2048 x 2048 with
// 128 slots each 130 / 149, 375 237 / 261, 1024 536 / 538, 2048 1061 / 955; 128
// of 640 x 2560: 375 191 / 243, 1024 427 / 501, 2048 811 / 886; 16 of 4096 x
// 4096: 512 280 / 296, 1024 498 / 489, 2048 944 / 869; fp32, 2048 slots: 1127 /
// 1021, 859 / 936, 1003 / 898.
template <typename OUT, bool GROUPED>
hipError_t choose(GemmParams &p, int cus, hipStream_t stream)
{
    if constexpr (!GROUPED) {
        auto tiles = [&](int bm, int bn) { return ceil_div(p.rows.rows, bm) * ceil_div(p.N, bn); };
        const int64_t middle = tiles(128, 128), last = middle % (2 * cus);
        const int64_t t256 = ceil_div(tiles(256, 256), cus) * 103,
                      t128 = middle / (2 * cus) * 55 + (last == 0 ? 0 : last <= cus ? 35 : 55),
                      t128d = ceil_div(middle, cus) * 30, t64 = ceil_div(tiles(64, 128), cus) * 20;
        const int64_t least = std::min(std::min(t256, t128), std::min(t128d, t64));
        if (least == t128)
            return launch<2, 2, 2, OUT, GROUPED>(p, stream);
        if (least == t256)
            return launch<4, 4, 2, OUT, GROUPED>(p, stream);
        if (least == t128d)
            return launch<2, 2, 4, OUT, GROUPED>(p, stream);
        return launch<1, 2, 4, OUT, GROUPED>(p, stream);
    } else {
        if (p.rows.rows >= 2048LL * p.rows.P)
            return launch<4, 4, 2, OUT, GROUPED>(p, stream);
        return launch<2, 2, 2, OUT, GROUPED>(p, stream);
    }
}

}  // namespace

hipError_t launch_f8_gemm(const uint8_t *W, const uint8_t *xq, void *Y, int y_type, const F8Rows &r, int64_t N,
                          int64_t K, int cus, hipStream_t stream)
{
    const F8Weights f = f8_weights(N, K);
    const F8Acts a = f8_acts(r.x_rows, K);
    GemmParams p{W, xq, Y, r, f.scales, a.scales, 0, (int)N, f.cb, a.ls, f.ls, f.rt, 0,
                 N * type_bytes(y_type) % 16 == 0 && (reinterpret_cast<uintptr_t>(Y) & 15) == 0};
    if (r.order)
        return y_type == QG_F32   ? choose<float, true>(p, cus, stream)
               : y_type == QG_F16 ? choose<Fp16, true>(p, cus, stream)
                                  : choose<Bf16, true>(p, cus, stream);
    return y_type == QG_F32   ? choose<float, false>(p, cus, stream)
           : y_type == QG_F16 ? choose<Fp16, false>(p, cus, stream)
                              : choose<Bf16, false>(p, cus, stream);
}

}  // namespace qg
