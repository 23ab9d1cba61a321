// f8 products of many rows: Y[m][n] = sum_k X[m][k] W[n][k] on the matrix
// cores, for one matrix or for the slots of each expert of a pool.
//
// A workgroup owns a tile of BM rows of X times BN rows of W.  A step is 64
// columns (half a block: one scale byte a row and side); its operands go
// straight from memory into LDS (loads that write LDS: no registers):
//   * X, row-major, a block of 128 columns at a time: rows of 128 bytes, whole
//     lines (the caches deliver 30 TB/s to loads of 8 rows x 128 bytes and 9.5
//     to loads of 16 rows x 64 bytes), 16-byte chunk c of row r at position
//     c ^ ((r / 2) % 8), so that the 16 rows of a quarter of an operand read
//     touch all 64 banks;
//   * W, whose tiles are in operand order already: copied as they are, a step
//     at a time; an operand read is 256 consecutive bytes a quarter wave.
// X has two buffers (blocks), W four (steps).  During step t the matrix cores
// multiply operands that were read from LDS during step t - 1, the operands of
// t + 1 are read, W's copies of step t + 3 are issued and, in a block's second
// step, X's copies of the block after the next one, both into buffers whose
// last reads fed products of step t - 1.  One barrier a step; before it a wave
// waits for those of its own copies that step t reads (issued in step t - 2 at
// the latest).
// 16-bit outputs: v_mfma_scale_f32_32x32x64_f8f6f4 with the two block scales
// as its scale operands, so the fp32 sums need no further instruction.  fp32
// outputs: the codes are widened to bf16 with their scale (exact) and
// multiplied with v_mfma_f32_32x32x16_bf16: half the rate, but products and
// sums exact to fp32, where the 8-bit instructions keep about 13 bits below
// the largest of a few neighbouring products.
// W is the first operand, so a lane holds four consecutive n of a row of Y;
// the tile is turned through LDS for whole-line stores.
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

__device__ __forceinline__ void copy16(const uint8_t *from, void *to)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                     (__attribute__((address_space(3))) void *)to, 16, 0, 0);
}

// Tile shape: WM x WN waves, each 32 TM rows of X times 32 TN rows of W.
template <int WM, int WN, int TM, int TN>
struct Tile {
    static constexpr int BM = 32 * TM * WM, BN = 32 * TN * WN, NT = 64 * WM * WN;
    static constexpr int XC = BM * 8 / NT, WC = BN * 4 / NT;   // 16-byte copies per thread: X's a block, W's a step
};

// Which tile a workgroup takes.  Workgroups go to the eight XCDs in turn, each
// with an L2 of its own: an XCD gets a contiguous share of the tiles, in
// bands of kBand tiles of rows of X (dense), so that the tiles it works on at
// a time share rows of both operands.
constexpr int kXcds = 8, kBand = 8;

template <bool GROUPED>
__device__ __forceinline__ bool tile_of(uint32_t item, uint32_t units, int tiles_n, uint32_t &unit, int &tn)
{
    const uint32_t total = units * tiles_n;
    const uint32_t share = (total + kXcds - 1) / kXcds;
    const uint32_t lin = (item % kXcds) * share + item / kXcds;
    if (item / kXcds >= share || lin >= total)
        return false;
    if constexpr (GROUPED) {
        unit = lin / (uint32_t)tiles_n;
        tn = (int)(lin - unit * tiles_n);
    } else {
        const uint32_t band = lin / (uint32_t)(kBand * tiles_n);
        const uint32_t in = lin - band * kBand * tiles_n;
        const uint32_t rows = min((uint32_t)kBand, units - band * kBand);
        tn = (int)(in / rows);
        unit = band * kBand + (in - (uint32_t)tn * rows);
    }
    return true;
}

template <int WM, int WN, int TM, int TN, typename OUT, bool GROUPED>
__global__ __launch_bounds__(64 * WM *WN, TM *TN == 16 ? 1 : 2) void gemm_kernel(GemmParams p)
{
    using T = Tile<WM, WN, TM, TN>;
    constexpr bool kWide = sizeof(OUT) == 4;
    // one variable a buffer: the compiler then knows which copies an operand
    // read has to wait for (none: the waits are the kernel's own)
    __shared__ uint4 X0[T::BM * 8], X1[T::BM * 8];
    __shared__ uint4 W0[T::BN * 4], W1[T::BN * 4], W2[T::BN * 4], W3[T::BN * 4];
    __shared__ int out_row[GROUPED ? T::BM : 1];
    auto xbuf = [&](int q) -> uint4 * { return q == 0 ? X0 : X1; };
    auto wbuf = [&](int q) -> uint4 * { return q == 0 ? W0 : q == 1 ? W1 : q == 2 ? W2 : W3; };

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave % WM, wn = wave / WM;
    const int r32 = lane & 31, half = lane >> 5;

    uint32_t unit;
    int tn;
    if (!tile_of<GROUPED>(blockIdx.x, p.units, p.tiles_n, unit, tn))
        return;
    F8Unit u{0, (int64_t)unit * T::BM, min((int64_t)(unit + 1) * T::BM, p.rows.rows)};
    if constexpr (GROUPED) {
        u = f8_unit(p.rows.offsets, p.rows.P, p.rows.rows, T::BM, unit);
        if (u.r0 >= u.r1)
            return;   // past the last unit (uniform over the workgroup)
    }
    const int n0 = tn * T::BN;
    const int rows = (int)(u.r1 - u.r0);

    // row of X for a row of the tile (rows past its end: the last one, never stored)
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
            const int s = r < rows ? p.rows.order[u.r0 + r] : -1;
            out_row[r] = s >= 0 && s < p.rows.rows ? s : -1;
        }
    }

    f16v_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
                acc[i][j][e] = 0.0f;

    if (!GROUPED || u.e < p.rows.P) {
        const uint8_t *W = p.W + (GROUPED ? u.e * p.rows.stride : 0);
        const uint8_t *xsrc[T::XC], *wsrc[T::WC];
#pragma unroll
        for (int i = 0; i < T::XC; ++i) {
            const int idx = threadIdx.x + T::NT * i;
            const int r = idx >> 3, ch = (idx & 7) ^ ((r >> 1) & 7);
            xsrc[i] = p.xq + x_row(r) * p.cb * 128 + ch * 16;
        }
#pragma unroll
        for (int i = 0; i < T::WC; ++i) {
            const int idx = threadIdx.x + T::NT * i;
            const int t = min(n0 / 16 + (idx >> 6), p.rt - 1);   // rows past the matrix are never stored
            wsrc[i] = W + (int64_t)t * p.cb * 2048 + (idx & 63) * 16;
        }
        // scales: four blocks' bytes a word, this word and the next
        const uint8_t *xs_src[TM];
#pragma unroll
        for (int i = 0; i < TM; ++i)
            xs_src[i] = p.xq + p.x_scales + x_row((wm * TM + i) * 32 + r32) * p.x_ls;
        static_assert(128 % (32 * TN) == 0, "a wave's rows of W lie in one block");
        const uint8_t *ws_src = W + p.w_scales + (int64_t)min((n0 + wn * TN * 32) >> 7, (p.N - 1) >> 7) * p.w_ls;
        uint32_t xs[TM], ws, xs_next[TM], ws_next;
        auto load_scales = [&](int word) {
            const int at = 4 * min(word, p.x_ls / 4 - 1);
#pragma unroll
            for (int i = 0; i < TM; ++i)
                xs_next[i] = *reinterpret_cast<const uint32_t *>(xs_src[i] + at);
            ws_next = *reinterpret_cast<const uint32_t *>(ws_src + at);
        };

        // the next block of X and step of W to copy; past the last one that
        // one again (never read).  No branch: the products of a step would be
        // moved across it
        const int steps = 2 * p.cb;
        int x_ahead = 0, w_ahead = 0;
        auto copy_x = [&](uint4 *X) {
#pragma unroll
            for (int i = 0; i < T::XC; ++i)
                copy16(xsrc[i], &X[T::NT * i + 64 * wave]);
            const int go = ++x_ahead < p.cb ? 128 : 0;
#pragma unroll
            for (int i = 0; i < T::XC; ++i)
                xsrc[i] += go;
        };
        auto copy_w = [&](uint4 *Wb) {
#pragma unroll
            for (int i = 0; i < T::WC; ++i)
                copy16(wsrc[i], &Wb[T::NT * i + 64 * wave]);
            const int go = ++w_ahead < steps ? 1024 : 0;
#pragma unroll
            for (int i = 0; i < T::WC; ++i)
                wsrc[i] += go;
        };
        struct Operands {
            uint4 x[TM][2], w[TN][2];
        };
        auto read = [&](Operands &o, const uint4 *X, int h, const uint4 *Wb) {   // h: half of X's block
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int ch = 2 * half + q;
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const int r = (wm * TM + i) * 32 + r32;
                    o.x[i][q] = X[r * 8 + ((4 * h + ch) ^ ((r >> 1) & 7))];
                }
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const int t = (wn * TN + j) * 2 + (r32 >> 4);
                    o.w[j][q] = Wb[t * 64 + ch * 16 + (r32 & 15)];
                }
            }
        };
        auto multiply = [&](const Operands &o) {
            if constexpr (!kWide) {
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) {
                        const i8_t a = {(int)o.w[j][0].x, (int)o.w[j][0].y, (int)o.w[j][0].z, (int)o.w[j][0].w,
                                        (int)o.w[j][1].x, (int)o.w[j][1].y, (int)o.w[j][1].z, (int)o.w[j][1].w};
                        const i8_t b = {(int)o.x[i][0].x, (int)o.x[i][0].y, (int)o.x[i][0].z, (int)o.x[i][0].w,
                                        (int)o.x[i][1].x, (int)o.x[i][1].y, (int)o.x[i][1].z, (int)o.x[i][1].w};
                        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc[i][j], 0, 0, 0,
                                                                                   (int)ws, 0, (int)xs[i]);
                    }
            } else {
                const float wf = f8_exponent(ws & 255u);
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        bf8_t w[TN];
#pragma unroll
                        for (int j = 0; j < TN; ++j)
                            w[j] = h ? f8_widen(o.w[j][q].z, o.w[j][q].w, wf)
                                     : f8_widen(o.w[j][q].x, o.w[j][q].y, wf);
#pragma unroll
                        for (int i = 0; i < TM; ++i) {
                            const float xf = f8_exponent(xs[i] & 255u);
                            const bf8_t x = h ? f8_widen(o.x[i][q].z, o.x[i][q].w, xf)
                                              : f8_widen(o.x[i][q].x, o.x[i][q].y, xf);
#pragma unroll
                            for (int j = 0; j < TN; ++j)
                                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(w[j], x, acc[i][j], 0, 0, 0);
                        }
                    }
            }
        };

        load_scales(0);
        copy_x(X0);
        copy_w(W0);
        copy_w(W1);
        copy_x(X1);
        copy_w(W2);
        Operands even, odd;
        wait_vm<T::XC + 2 * T::WC>();
        bare_barrier();
        read(even, X0, 0, W0);
        uint32_t xword[TM], wword;
        // step q of a pair of blocks, the first of which is b
        auto step = [&](int b, auto number) {
            constexpr int q = decltype(number)::value;
            // an even step leaves the copies of the step before it in flight
            // (X's and W's), an odd one's predecessor copied W only
            wait_vm<q & 1 ? T::WC : T::XC + T::WC>();
            bare_barrier();
            if constexpr (q == 0) {
                // the scales of a pair of blocks are loaded a pair ahead
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    xword[i] = xs_next[i];
                wword = ws_next;
                load_scales((b + 2) / 4);
            }
            if constexpr ((q & 1) == 0) {
                const int shift = 8 * ((b + q / 2) & 3);
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    xs[i] = xword[i] >> shift;
                ws = wword >> shift;
            }
            if constexpr (q & 1)
                copy_x(xbuf(q >> 1));
            copy_w(wbuf((q + 3) & 3));
            read(q & 1 ? even : odd, xbuf(((q + 1) & 3) >> 1), (q + 1) & 1, wbuf((q + 1) & 3));
            multiply(q & 1 ? odd : even);
            // reads and copies behind the first products: left alone they
            // gather at the end of the step
            if constexpr (!kWide) {
                constexpr int kProducts = TM * TN, kReads = 2 * (TM + TN), kCopies = T::WC + (q & 1 ? T::XC : 0);
                constexpr int kPer = (kCopies + kProducts - 1) / kProducts;
#pragma unroll
                for (int m = 0; m < kProducts; ++m) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);   // one MFMA
                    if (2 * m < kReads)
                        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);   // LDS reads
                    if (kPer * m < kCopies)
                        __builtin_amdgcn_sched_group_barrier(0x020, kPer, 0);   // copies
                }
            }
        };
        int b = 0;
        for (; b + 1 < p.cb; b += 2) {
            step(b, std::integral_constant<int, 0>{});
            step(b, std::integral_constant<int, 1>{});
            step(b, std::integral_constant<int, 2>{});
            step(b, std::integral_constant<int, 3>{});
        }
        if (b < p.cb) {
            step(b, std::integral_constant<int, 0>{});
            step(b, std::integral_constant<int, 1>{});
        }
        wait_vm<0>();   // no copy is in flight when the buffers are used again
    }

    __syncthreads();   // out_row is written, and the buffers are free
    // A lane has four consecutive n of one row, a wave's store of them
    // would touch 32 rows.  So 32 rows x 32 TN columns at a time go
    // through LDS (wave-private, 16-byte chunks swizzled by row) and are
    // stored whole lines at a time.
    constexpr int JN = kWide ? TN / 2 : TN;       // column tiles staged at a time
    constexpr int kRow = 32 * JN * (int)sizeof(OUT), kChunks = kRow / 16;
    static_assert(WM * WN == 4 && 4 * 32 * kRow <= T::BM * 128, "each wave stages in a quarter of X0");
    uint4 *stage = X0 + wave * (T::BM * 2);
    char *bytes = reinterpret_cast<char *>(stage);
    constexpr int kPer = 16 / (int)sizeof(OUT);   // elements of a chunk
    constexpr int kStores = 32 * kChunks / 64;    // per lane and 32 rows
    const bool whole = p.vec && n0 + T::BN <= p.N && (GROUPED || rows == T::BM);   // no edge in this tile
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
                if constexpr (kWide)
                    *reinterpret_cast<f4_t *>(to) = f4_t{a[4 * g], a[4 * g + 1], a[4 * g + 2], a[4 * g + 3]};
                else
                    *reinterpret_cast<uint2 *>(to) =
                        make_uint2(pack2<OUT>(a[4 * g], a[4 * g + 1]), pack2<OUT>(a[4 * g + 2], a[4 * g + 3]));
            }
        // the c-th chunk of this lane: its row and column in the tile
        auto row_at = [&](int c) { return (wm * TM + i) * 32 + (64 * c + lane) / kChunks; };
        auto chunk_at = [&](int c) {
            const int r = (64 * c + lane) / kChunks, ch = (64 * c + lane) % kChunks;
            return stage[r * kChunks + (ch ^ (r & (kChunks - 1)))];
        };
        const int n = n0 + (wn * TN + j0) * 32 + lane % kChunks * kPer;   // 64 is a multiple of kChunks
        if (whole) {
            uint4 v[kStores];
#pragma unroll
            for (int c = 0; c < kStores; ++c)
                v[c] = chunk_at(c);
#pragma unroll
            for (int c = 0; c < kStores; ++c) {
                const int64_t y = GROUPED ? out_row[row_at(c)] : u.r0 + row_at(c);
                if (!GROUPED || y >= 0)
                    *reinterpret_cast<uint4 *>(static_cast<OUT *>(p.Y) + y * p.N + n) = v[c];
            }
        } else {
#pragma unroll 1
            for (int c = 0; c < kStores; ++c) {
                const int m = row_at(c);
                const uint4 v = chunk_at(c);
                const int64_t y = GROUPED ? out_row[m] : u.r0 + m;
                if (!(GROUPED ? y >= 0 : m < rows) || n >= p.N)
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
                        if constexpr (kWide)
                            to[e] = __uint_as_float(w[e]);
                        else
                            to[e] = OUT{(uint16_t)(w[e / 2] >> (16 * (e & 1)))};
                    }
            }
        }
    }
}

template <int WM, int WN, int TM, int TN, typename OUT, bool GROUPED>
hipError_t launch(GemmParams &p, hipStream_t stream)
{
    using T = Tile<WM, WN, TM, TN>;
    p.tiles_n = (int)ceil_div(p.N, T::BN);
    p.units = (uint32_t)(GROUPED ? f8_units(p.rows.rows, p.rows.P, T::BM) : ceil_div(p.rows.rows, T::BM));
    const int64_t items = ceil_div((int64_t)p.units * p.tiles_n, kXcds) * kXcds;
    if (items >= 1 << 24)   // a grid holds fewer than 2^32 threads
        return hipErrorInvalidValue;
    return launch_kernel(reinterpret_cast<const void *>(&gemm_kernel<WM, WN, TM, TN, OUT, GROUPED>),
                         dim3((unsigned)items), dim3(T::NT), 0, stream, p);
}

template <typename OUT, bool GROUPED>
hipError_t choose(GemmParams &p, int cus, hipStream_t stream)
{
    if constexpr (!GROUPED) {
        if (ceil_div(p.rows.rows, 256) * ceil_div(p.N, 256) >= cus)
            return launch<2, 2, 4, 4, OUT, GROUPED>(p, stream);
        return launch<2, 2, 2, 2, OUT, GROUPED>(p, stream);
    } else {
        return launch<2, 2, 2, 2, OUT, GROUPED>(p, stream);
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
