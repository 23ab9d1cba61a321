// Attention of new tokens over the paged cache (definitions in qgemv_attn.h).
//
// Rows are the queries that share a key head: row i share + j is new token i of
// query head j of the group.  One workgroup takes up to 16 kTiles rows of a
// sequence and key head over a part of its cache, its four waves 32
// tokens each in turn, independently: running maximum, sum and accumulators in
// registers, joined through LDS at the end, chunks by a second launch.
//
// Products on v_mfma_f32_16x16x32 with the cache as the A operand:
//   S^T = K Q^T  (16 tokens x 16 rows; a lane gets four tokens of one row),
//   O^T = V^T P^T (16 of D x 16 rows; a lane's P operand is eight tokens of one
//   row: exactly those of two S^T tiles that it has).
// So the softmax's weights never move between lanes, a row's maximum and sum
// live in the row's lanes, and rescaling is a multiplication in place.  Which
// token is which k of the second product is free; K comes as the A operand by
// 16-byte loads (a lane holds one token), V needs eight tokens of one dimension
// in a lane: it loads D / 16 consecutive elements of eight tokens and turns the
// 8 x D / 16 piece with byte permutes in registers.  Nothing passes through LDS.
//
// 8-bit codes are widened exactly; a key's scale goes along (bf16) or multiplies
// its score (fp16), a value's scale its weight.  A weight (fp32) enters the second
// product as two 16-bit parts, hi = round(p), lo = round(p - hi): 2^-16 of it is
// lost, where one part would lose 2^-8, as much as the output's rounding, for a
// product that waits for memory anyway.  bf16 for f8 and bf16 values; with fp16
// values fp16, taken times 2^11 (they reach 2^4) so that small weights stay
// normal.
//
// Bound by the cache's bytes where rows are few: 262143 tokens of 8 key heads in f8
// (541 MB) 84 us, 6.4 TB/s, with the loads alone at 6.8; 64 ragged sequences in
// bf16 (877 MB) 136 us, 6.4 TB/s; vector units 37 and 15 % busy.  With 30 rows
// (f8, 230 MB) 48 us: the vector units are 58 % busy with softmax and conversions.
// Steps on the way (us, 262143 tokens / ragged / 30 rows): work in equal chunks of a
// sequence 108 / 167 / 79; scale factors by ldexp and with the widening, sums scaled
// anew only beyond a slack 102 / 169 / 74; loads that leave nothing in the caches, of
// whole lines 92 / 159 / 73; runs of equal length in one round of workgroups, and a
// bound on registers that keeps accumulators out of the other register file
// 92 / 148 / 60; a lighter join 90 / 139 / 57; scores as distances by one fma, the
// row's maximum across lanes only beyond the slack 89 / 139 / 56 (64 rows of 192
// dimensions 77 to 74).  More than 32 rows a key head (16 sequences of up to 8000, 64 rows in
// f8 53 us for 22 of bytes) are bound by the vector units: every group of rows loads, widens
// and turns the same tokens.  64 dimensions in f8 reach 3.7 TB/s over 100000 tokens: a step is
// 32 tokens whatever their width, so a wave has 4 KB in flight where 128 dimensions have 8.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <limits>

#include "qgemv_attn_internal.h"

namespace qg {
namespace {

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / 64;
constexpr int kStep = 32;                 // tokens of a wave's step
constexpr int kTile = kStep * kWaves;     // tokens of a workgroup's step
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kSlack = 4.0f;            // weights reach 2^kSlack before they are scaled anew

// Rounds of workgroups over the compute units (256) that the work is cut for.
constexpr int kUnits = 256;
constexpr int kRounds = 1;
constexpr int kManyRows = 1024;   // from here on a wave joins a row

typedef _Float16 h8_t __attribute__((ext_vector_type(8)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));

struct F8Code {};

// Tables and lengths are read through the scalar cache: addresses are the
// wave's.
typedef const __attribute__((address_space(4))) int32_t *ScalarInts;
__device__ __forceinline__ int scalar_int(const int32_t *p, int64_t i)
{
    return ((ScalarInts)(uintptr_t)p)[i];
}

// How the work is cut.  A sequence has `tiles` of kTile tokens, at least one
// (its rows are written in any case).  The tiles of all sequences, one after the
// other, are dealt out in runs of `run` to the workgroups of a key head, so each
// has the same work whatever the lengths are; a run may end inside a sequence
// and begin the next one.  Only sequences that a run's end cuts leave parts: at most
// one that the run before began and one that the run after goes on with.
struct Sequence {
    int len;
    int first;          // its first token that anybody sees, down to a multiple of 16
    int tiles;
};

struct Plan {
    int run, total;
    int b;              // sequence
    int base;           // its first tile among all
    Sequence seq;
};

__device__ __forceinline__ Sequence sequence(const AttendArgs &a, int len)
{
    const int64_t most = (int64_t)a.width << a.cache.log_page;
    Sequence s;
    s.len = (int)min((int64_t)max(len, 0), most);
    s.first = a.window ? max(0, s.len - a.M + 1 - a.window) & ~15 : 0;
    s.tiles = max(1, (s.len - s.first + kTile - 1) / kTile);
    return s;
}

// The length of the runs, from the lengths, by every wave itself, and either
// the sequence that holds the first tile of run `w` or sequence `w`.
template <bool kOfRun>
__device__ __forceinline__ Plan plan(const AttendArgs &a, int target, int w)
{
    const int lane = threadIdx.x & 63;
    Plan p{};
    int len = 0, mine = 0;
    auto take = [&](int b0) {
        const bool is = b0 + lane < a.B;
        len = is ? a.lens[b0 + lane] : 0;
        mine = is ? sequence(a, len).tiles : 0;
    };
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        take(b0);
        p.total += __builtin_amdgcn_readlane(prefix_sum(mine), 63);
    }
    p.run = (p.total + target - 1) / target;
    const int64_t tile = kOfRun ? (int64_t)w * p.run : 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        if (a.B > 64)
            take(b0);
        const int upto = prefix_sum(mine);
        int at = w - b0;
        bool here = at < 64;
        if (kOfRun) {
            const unsigned long long holds = __ballot(p.base + (int64_t)upto > tile);
            here = holds != 0;
            at = __ffsll(holds) - 1;
        }
        if (here) {
            p.b = b0 + at;
            p.base += __builtin_amdgcn_readlane(upto - mine, at);
            p.seq = sequence(a, __builtin_amdgcn_readlane(len, at));
            return p;
        }
        p.base += __builtin_amdgcn_readlane(upto, 63);
    }
    p.b = -1;
    return p;
}

// 16-bit arithmetic of a launch: operands of the products and conversions.
template <typename T>
struct Half;
template <>
struct Half<Bf16> {
    typedef bf8_t v8;
    static __device__ __forceinline__ f4_t mfma(v8 a, v8 b, f4_t c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Half<Fp16> {
    typedef h8_t v8;
    static __device__ __forceinline__ f4_t mfma(v8 a, v8 b, f4_t c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};

// Four codes of a word times a power of two as 16-bit values, two words.
template <typename T>
__device__ __forceinline__ u2_t widen4(uint32_t w, float scale)
{
    if constexpr (std::is_same_v<T, Bf16>) {
        return u2_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true))};
    } else {
        return u2_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, false)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, scale, true))};
    }
}

template <typename T>
__device__ __forceinline__ typename Half<T>::v8 widen8(uint32_t lo, uint32_t hi, float scale = 1.0f)
{
    const u2_t a = widen4<T>(lo, scale), b = widen4<T>(hi, scale);
    return __builtin_bit_cast(typename Half<T>::v8, u4_t{a[0], a[1], b[0], b[1]});
}

// e of the i-th of four scale bytes.
__device__ __forceinline__ int exponent_of(uint32_t bytes, int i) { return (int)((bytes >> (8 * i)) & 255u) - 127; }

// Words of the cache.  Where one workgroup reads each (kOnce), loads that leave
// nothing behind in the caches stream at 6.8 TB/s where ordinary ones reach 5.9
// (541 MB in pages of 64 tokens, loads alone); they have to take whole lines, or the
// other half is read again.  Where several groups of rows read the same cache,
// ordinary loads find it in the caches (16 sequences of up to 8000, 128 rows a key
// head in bf16 104 us for 120).
template <int kWords, bool kOnce>
__device__ __forceinline__ void load_words(const uint8_t *from, uint32_t *to)
{
    constexpr int kN = kWords % 4 == 0 ? 4 : kWords % 3 == 0 ? 3 : kWords % 2 == 0 ? 2 : 1;
    typedef uint32_t piece __attribute__((ext_vector_type(kN), aligned(4 * (kN == 3 ? 1 : kN))));
#pragma unroll
    for (int i = 0; i < kWords; i += kN) {
        const piece *at = reinterpret_cast<const piece *>(from + 4 * i);
        const piece p = kOnce ? __builtin_nontemporal_load(at) : *at;
#pragma unroll
        for (int j = 0; j < kN; ++j)
            to[i + j] = p[j];
    }
}

// 4 x 4 bytes turned: word i of the result has byte i of the four words.
__device__ __forceinline__ u4_t turn4(uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3)
{
    const uint32_t a = __builtin_amdgcn_perm(r1, r0, 0x05010400), b = __builtin_amdgcn_perm(r1, r0, 0x07030602);
    const uint32_t c = __builtin_amdgcn_perm(r3, r2, 0x05010400), d = __builtin_amdgcn_perm(r3, r2, 0x07030602);
    return u4_t{__builtin_amdgcn_perm(c, a, 0x05040100), __builtin_amdgcn_perm(c, a, 0x07060302),
                __builtin_amdgcn_perm(d, b, 0x05040100), __builtin_amdgcn_perm(d, b, 0x07060302)};
}

// The elements of a word that are NaN or infinite, as a mask.
template <typename T, bool kF8>
__device__ __forceinline__ uint32_t not_finite(uint32_t w)
{
    if constexpr (kF8)
        return ((((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 255u;
    else if constexpr (std::is_same_v<T, Bf16>)
        return ((((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u) >> 15) * 65535u;
    else
        return ((((w & 0x7C007C00u) + 0x04000400u) & 0x80008000u) >> 15) * 65535u;
}

// cap tanh(x), x = product to_cap, a score in powers of two.  Up to |x| = 1/2 it is the
// score without a cap times tanh(x) / x, a series in x^2 (its coefficients for the least
// largest error there, 2^-26 of the value): right to a few 2^-24 of the score however
// large the cap is, where 1 - 2 / (1 + e^2x) alone is off by as much of the cap.
__device__ __forceinline__ float capped_score(float product, float to_score, float to_cap, float cap)
{
    const float x = product * to_cap, z = x * x;
    const float ratio =
        fmaf(fmaf(fmaf(fmaf(0.01724149f, z, -0.05304549f), z, 0.13325879f), z, -0.33333144f), z, 1.0f);
    const float e2 = __builtin_amdgcn_exp2f(fabsf(x) * (2.0f * kLog2e));
    const float far = cap * fmaf(-2.0f, __builtin_amdgcn_rcpf(1.0f + e2), 1.0f);
    return fabsf(x) <= 0.5f ? product * to_score * ratio : copysignf(far, x);
}

__device__ __forceinline__ float max_over_groups(float v)
{
    f2_t p = pair16(v);
    v = fmaxf(p[0], p[1]);
    p = pair32(v);
    return fmaxf(p[0], p[1]);
}
__device__ __forceinline__ float sum_over_groups(float v)
{
    f2_t p = pair16(v);
    v = p[0] + p[1];
    p = pair32(v);
    return p[0] + p[1];
}

__device__ __forceinline__ float wave_max(float v)
{
    v = group_max<32>(v);
    const f2_t p = pair32(v);
    return fmaxf(p[0], p[1]);
}
__device__ __forceinline__ float wave_sum(float v)
{
    v = group_sum<32>(v);
    const f2_t p = pair32(v);
    return p[0] + p[1];
}

// Where the sums of a part go if its sequence has others: accumulators
// [part][key head][row][D], then (maximum, sum) [part][key head][row].
struct Parts {
    float *o;
    float *ml;
};
__host__ __device__ inline Parts parts_at(void *workspace, int64_t units, int heads, int rows, int D)
{
    Parts p;
    p.o = static_cast<float *>(workspace);
    p.ml = p.o + units * heads * rows * D;
    return p;
}

// Workgroups that a compute unit holds at once (a wave of each on every SIMD).
constexpr int resident(int D, bool f8, int tiles)
{
    if (tiles == 1)
        return D == 64 ? 4 : D == 128 ? (f8 ? 3 : 2) : D == 192 ? 2 : f8 ? 2 : 1;
    return D == 64 ? 3 : D == 128 ? 2 : 1;
}

struct AttendLaunch {
    AttendArgs a;
    int target;     // runs, at most, for each key head and row group
    int units;      // parts, at most
    int rows;       // M share
    int row_groups;
    bool by_sequence;   // a workgroup a sequence, nothing to find or to join
    bool by_run;        // no more runs than sequences
    float to_score;     // scale in powers of two
    float to_cap, cap;  // scale / softcap, the cap in powers of two
};

// The number of a run's part of a sequence that begins in it or before it: two of each
// run or, where that is fewer, run + sequence (both only grow along the runs).
template <bool kByRun>
__device__ __forceinline__ int part_of(int run, int b, bool begins)
{
    return kByRun ? 2 * run + (begins ? 1 : 0) : run + b;
}

// TQ: type of q, of the output and of 16-bit caches; kF8: an 8-bit cache; kOnce: no
// other group of rows reads the cache.
template <typename TQ, bool kF8, int D, int kTiles, bool kOnce>
__global__ __launch_bounds__(kBlock, resident(D, kF8, kTiles)) void attend_kernel(AttendLaunch la)
{
    using TV = std::conditional_t<kF8, Bf16, TQ>;   // of the second product
    using Q = Half<TQ>;
    using V = Half<TV>;
    constexpr int kItem = kF8 ? 1 : 2;
    constexpr int kRow = D * kItem;         // bytes of a vector
    constexpr int kSteps = D / 32;          // products of a score
    constexpr int kOut = D / 16;            // accumulator tiles, consecutive dimensions of a lane
    constexpr int kKeyLoads = kRow / 64;    // 16-byte loads of a tile of 16 tokens
    constexpr int kValWords = kOut * kItem / 4;
    constexpr bool kWholeLines = kRow % 128 == 0;
    // a key's scale: bf16 takes it with the widening, exactly; fp16 has not the range, the score takes it there
    constexpr bool kScaledKeys = kF8 && std::is_same_v<TQ, Bf16>;
    constexpr float kWeight = std::is_same_v<TV, Fp16> ? 2048.0f : 1.0f;

    const AttendArgs &a = la.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int heads = a.cache.heads;
    const int head = blockIdx.x % heads;
    const int group = (blockIdx.x / heads) % la.row_groups;
    const int run = blockIdx.x / (heads * la.row_groups);
    Plan p{};
    if (la.by_sequence) {
        p.b = run;
        p.run = p.total = INT32_MAX;
        p.seq = sequence(a, a.lens[run]);
    } else {
        p = plan<true>(a, la.target, run);
        if (p.b < 0)
            return;
    }
    const int run_begin = la.by_sequence ? 0 : run * p.run;
    const int run_end = min(run_begin + p.run, p.total);
    const int row0 = group * 16 * kTiles;
    __shared__ float o[kWaves][16][D + 4];
    __shared__ float ml[kWaves][16][2];

    // one sequence's part of the run after the other
    for (int tile = run_begin;;) {
        const Sequence seq = p.seq;
        const int t0 = tile - p.base, t1 = min(seq.tiles, run_end - p.base);

        // queries: row r is column r of the first product
        typename Q::v8 q[kTiles][kSteps];
        int mine[kTiles];                       // the row's new token
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
            const int row = row0 + 16 * n + r16;
            const int i = min(row / a.share, a.M - 1);
            mine[n] = i;
            const TQ *from = static_cast<const TQ *>(a.q) + ((int64_t)p.b * a.M + i) * a.ldq +
                             ((int64_t)head * a.share + row % a.share) * D;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int d = kF8 ? 64 * (s / 2) + 16 * g + 8 * (s & 1) : 32 * s + 8 * g;
                Raw16 w{};
                if (row < la.rows)
                    w = *reinterpret_cast<const Raw16 *>(from + d);
                q[n][s] = __builtin_bit_cast(typename Q::v8, w);
            }
        }

        const int64_t head_at = (int64_t)head * 2 * a.cache.page * kRow;
        const int64_t scale_at = a.cache.scales + (int64_t)head * 2 * a.cache.page;
        const int last_page = a.width - 1;
        auto page_of = [&](int token) {
            return scalar_int(a.table, (int64_t)p.b * a.width + min(token >> a.cache.log_page, last_page));
        };
        // where a tile of 16 tokens lies, and whether its page is there
        struct Where {
            const uint8_t *keys, *scales;
            bool there;
        };
        // what a step multiplies
        struct Stage {
            uint32_t kw[2][kKeyLoads][4];
            uint32_t vw[8][kValWords];
            uint32_t ks[2], vs[2];
            bool there[2];
        };
        auto where = [&](int page, int token) {
            Where w;
            w.there = (uint32_t)page < (uint32_t)a.cache.pages;
            const uint8_t *base = a.cache.data + (int64_t)(w.there ? page : 0) * a.cache.page_bytes;
            const int in = token & (a.cache.page - 1);
            w.keys = base + head_at + (int64_t)in * kRow;
            w.scales = base + scale_at + in;
            return w;
        };
        const int64_t values = (int64_t)a.cache.page * kRow;

        // Loads stay where they are written: one moved behind the values' loads would be waited for with all of them.
        // With live 0, behind the last step, every lane reads the first piece (the count of loads stays the same).
        auto keep_order = [] {
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        };
        auto load_keys = [&](Stage &b, const Where (&w)[2], int live) {
            keep_order();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                b.there[h] = w[h].there;
                if constexpr (kScaledKeys)
                    b.ks[h] = w[h].scales[r16];
                else if constexpr (kF8)
                    b.ks[h] = *reinterpret_cast<const uint32_t *>(w[h].scales + 4 * g);
            }
            const int at = (kWholeLines ? (r16 & 7) * kRow + 64 * (r16 >> 3) + 16 * g : r16 * kRow + 16 * g) & live;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int c = 0; c < kKeyLoads; ++c)
                    load_words<4, kOnce>(w[h].keys + (at + (kWholeLines ? 8 * (c & 1) * kRow + 128 * (c / 2) : 64 * c)),
                                 b.kw[h][c]);
            keep_order();
        };
        auto load_values = [&](Stage &b, const Where (&w)[2], int live) {
            keep_order();
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if constexpr (kF8)
                    b.vs[h] = *reinterpret_cast<const uint32_t *>(w[h].scales + a.cache.page + 4 * g);
            const int at = (4 * g * kRow + r16 * (4 * kValWords)) & live;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    load_words<kValWords, kOnce>(w[h].keys + values + (at + j * kRow), b.vw[4 * h + j]);
            keep_order();
        };
        // Lines to rows: lane r16 has half r16 / 8 of tokens r16 % 8 and 8 + r16 % 8, and wants both halves of r16's.
        auto key_rows = [&](Stage &b, int h) {
            if constexpr (kWholeLines) {
#pragma unroll
                for (int c = 0; c < kKeyLoads; c += 2)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int low = (int)b.kw[h][c][i], high = (int)b.kw[h][c + 1][i];
                        b.kw[h][c][i] = (uint32_t)__builtin_amdgcn_update_dpp(low, high, 0x128, 0xF, 0xC, false);
                        b.kw[h][c + 1][i] = (uint32_t)__builtin_amdgcn_update_dpp(high, low, 0x128, 0xF, 0x3, false);
                    }
            }
        };

        f4_t acc[kTiles][kOut];
        // A row's scores are held as their distance from `from`; the sums are taken anew from a larger one if a
        // distance passes `limit`: any does while the row has seen nothing.
        float from[kTiles], limit[kTiles], sum[kTiles];
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
            from[n] = 0.0f;
            limit[n] = -__builtin_inff();
            sum[n] = 0.0f;
#pragma unroll
            for (int d = 0; d < kOut; ++d)
                acc[n][d] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
        }

        using V8 = typename V::v8;
        auto add = [&](const V8 &v, const V8 (&hi)[kTiles], const V8 (&lo)[kTiles], int d) {
#pragma unroll
            for (int n = 0; n < kTiles; ++n)
                acc[n][d] = V::mfma(v, lo[n], V::mfma(v, hi[n], acc[n][d]));
        };

        // places that every row sees: from all_from on, below all_end
        const int all_end = seq.len - a.M + 1;
        const int all_from = a.window ? max(0, seq.len - a.window) : 0;
        const int any_from = a.window ? max(0, all_end - a.window) : 0;
        // (under a cap products stay as they are until capped_score)
        const float scale = a.softcap > 0.0f ? 1.0f : la.to_score;

        auto edge = [&](int at) { return at + kStep > all_end || at < all_from; };
        bool left_out = false;   // values that are not finite, of places that some rows do not see

        const int first = seq.first + t0 * kTile + wave * kStep;
        int token = first;
        const int end = min(seq.first + t1 * kTile, seq.len);
        if (token < end) {
            // pages a step ahead of their loads, loads a half step ahead of their products (another set of registers,
            // and loads a whole step ahead, gained nothing: 92 us for 92, 142 for 143, 88 for 83 on 256 dimensions)
            int next = token, page[2] = {page_of(next), page_of(next + 16)};
            Stage b;
            {
                const Where now[2] = {where(page[0], next), where(page[1], next + 16)};
                load_keys(b, now, -1);
                load_values(b, now, -1);
                next += kTile;
                page[0] = page_of(next), page[1] = page_of(next + 16);
            }
            for (;;) {
                // scores
                float s[kTiles][8];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    key_rows(b, h);
                    f4_t c[kTiles];
#pragma unroll
                    for (int n = 0; n < kTiles; ++n)
                        c[n] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int st = 0; st < kSteps; ++st) {
                        typename Q::v8 k;
                        if constexpr (kF8) {
                            const uint32_t (&w)[4] = b.kw[h][st / 2];
                            const float to = kScaledKeys ? f8_exponent(b.ks[h]) : 1.0f;
                            k = (st & 1) ? widen8<TQ>(w[2], w[3], to) : widen8<TQ>(w[0], w[1], to);
                        } else {
                            k = __builtin_bit_cast(typename Q::v8, b.kw[h][st]);
                        }
#pragma unroll
                        for (int n = 0; n < kTiles; ++n)
                            c[n] = Q::mfma(k, q[n][st], c[n]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
#pragma unroll
                        for (int n = 0; n < kTiles; ++n) {
                            float product = c[n][i];
                            if constexpr (kF8 && !kScaledKeys)
                                product = ldexpf(product, exponent_of(b.ks[h], i));
                            s[n][4 * h + i] = fmaf(product, scale, a.softcap > 0.0f ? 0.0f : -from[n]);
                        }
                    }
                }
                const bool whole_tiles = b.there[0] && b.there[1], there[2] = {b.there[0], b.there[1]};
                // the keys of a step to come
                const int live = next < end ? -1 : 0;
                const Where now[2] = {where(page[0], next), where(page[1], next + 16)};
                load_keys(b, now, live);
                if (a.softcap > 0.0f) {
#pragma unroll
                    for (int n = 0; n < kTiles; ++n)
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            s[n][i] = capped_score(s[n][i], la.to_score, la.to_cap, la.cap) - from[n];
                }
                if (edge(token) || !whole_tiles) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int at = token + 16 * (i / 4) + 4 * g + (i & 3);
                        const bool is = there[i / 4];
#pragma unroll
                        for (int n = 0; n < kTiles; ++n) {
                            const int stop = seq.len - a.M + 1 + mine[n], start = a.window ? stop - a.window : 0;
                            if (!is || at >= stop || at < start)
                                s[n][i] = -__builtin_inff();
                        }
                        const bool seen = is && at < seq.len && at >= any_from;
#pragma unroll
                        for (int c = 0; c < kValWords; ++c) {
                            if (!seen)
                                b.vw[i][c] = 0;
                            // 0 times what is not finite is not 0: what some rows see and others do not comes later
                            const uint32_t odd = not_finite<TQ, kF8>(b.vw[i][c]);
                            if (a.M > 1 && odd) {
                                b.vw[i][c] &= ~odd;
                                left_out = true;
                            }
                        }
                    }
                }
                // softmax
                typename V::v8 hi[kTiles], lo[kTiles];
#pragma unroll
                for (int n = 0; n < kTiles; ++n) {
                    float m = s[n][0];
#pragma unroll
                    for (int i = 1; i < 8; ++i)
                        m = fmaxf(m, s[n][i]);
                    // weights up to 2^kSlack are as good as up to 1: only beyond is the row's largest score looked for
                    // (its lanes are four) and everything scaled anew
                    if (__any(m > limit[n])) {
                        m = max_over_groups(m);
                        const bool fresh = limit[n] == -__builtin_inff(), none = m == -__builtin_inff();
                        const float by = fresh ? (none ? 0.0f : m) : fmaxf(m, 0.0f);
                        const float old = fresh ? 0.0f : __builtin_amdgcn_exp2f(-by);
                        sum[n] *= old;
#pragma unroll
                        for (int d = 0; d < kOut; ++d)
                            acc[n][d] *= old;
                        from[n] += by;
                        if (!none)
                            limit[n] = kSlack;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            s[n][i] -= by;
                    }
                    float w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float e = __builtin_amdgcn_exp2f(s[n][i]);
                        sum[n] += e;
                        w[i] = e * kWeight;
                        if constexpr (kF8)   // (of 0 too: the scale of a place without a token may be anything)
                            w[i] = ldexpf(e, exponent_of(b.vs[i / 4], i & 3));
                    }
                    u4_t h4, l4;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        h4[i] = pack2<TV>(w[2 * i], w[2 * i + 1]);
                        const float a0 = to_f32(TV{(uint16_t)h4[i]}), a1 = to_f32(TV{(uint16_t)(h4[i] >> 16)});
                        l4[i] = pack2<TV>(w[2 * i] - a0, w[2 * i + 1] - a1);
                    }
                    hi[n] = __builtin_bit_cast(typename V::v8, h4);
                    lo[n] = __builtin_bit_cast(typename V::v8, l4);
                }
#pragma unroll
                for (int c = 0; c < kValWords; ++c) {
                    if constexpr (kF8) {
                        const u4_t x = turn4(b.vw[0][c], b.vw[1][c], b.vw[2][c], b.vw[3][c]);
                        const u4_t y = turn4(b.vw[4][c], b.vw[5][c], b.vw[6][c], b.vw[7][c]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            add(widen8<TV>(x[i], y[i]), hi, lo, 4 * c + i);
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const uint32_t half = i ? 0x07060302 : 0x05040100;
                            u4_t pairs;
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                pairs[j] = __builtin_amdgcn_perm(b.vw[2 * j + 1][c], b.vw[2 * j][c], half);
                            add(__builtin_bit_cast(V8, pairs), hi, lo, 2 * c + i);
                        }
                    }
                }
                load_values(b, now, live);
                token += kTile;
                if (token >= end)
                    break;
                next += kTile;
                page[0] = page_of(next), page[1] = page_of(next + 16);
            }
        }

        // What was left out reaches the rows that see its place: infinities and NaNs of the values themselves (weights
        // are positive).
        if (__any(left_out)) {
#pragma unroll 1
            for (int at = first; at < end; at += kTile) {
                if (!edge(at) && (uint32_t)page_of(at) < (uint32_t)a.cache.pages &&
                    (uint32_t)page_of(at + 16) < (uint32_t)a.cache.pages)
                    continue;
#pragma unroll 1
                for (int t = at; t < min(at + kStep, seq.len); ++t) {
                    const Where w = where(page_of(t), t);
                    if (!w.there)
                        continue;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const auto *from =
                            reinterpret_cast<const uint32_t *>(w.keys + values + (4 * g + e) * (4 * kValWords));
#pragma unroll
                        for (int c = 0; c < kValWords; ++c) {
                            const uint32_t word = from[c] & not_finite<TQ, kF8>(from[c]);
#pragma unroll
                            for (int i = 0; i < 4 / kItem; ++i) {
                                float v;
                                if constexpr (kF8)
                                    v = ((word >> (8 * i)) & 255u) ? __builtin_nanf("") : 0.0f;
                                else
                                    v = to_f32(TQ{(uint16_t)(word >> (16 * i))});
#pragma unroll
                                for (int n = 0; n < kTiles; ++n) {
                                    const int stop = all_end + mine[n], start = a.window ? stop - a.window : 0;
                                    acc[n][4 / kItem * c + i][e] += t < stop && t >= start ? v : 0.0f;
                                }
                            }
                        }
                    }
                }
            }
        }

        // the waves' sums, one tile of rows after the other
        const bool whole = p.base / p.run == (p.base + seq.tiles - 1) / p.run;   // the sequence is in this run alone
        const Parts parts = parts_at(a.workspace, la.units, heads, la.rows, D);
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
            const float l = sum_over_groups(sum[n]);
            __syncthreads();   // (the last tile's or sequence's readers)
            if (g == 0)
                ml[wave][r16][0] = limit[n] == kSlack ? from[n] : -__builtin_inff(), ml[wave][r16][1] = l;
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int d = 0; d < kOut; d += 4)
                    *reinterpret_cast<f4_t *>(&o[wave][r16][(4 * g + e) * kOut + d]) =
                        f4_t{acc[n][d][e], acc[n][d + 1][e], acc[n][d + 2][e], acc[n][d + 3][e]};
            __syncthreads();
            const int r = threadIdx.x >> 4, row = row0 + 16 * n + r;
            if (row >= la.rows)
                continue;
            float m = -__builtin_inff(), total = 0.0f, weight[kWaves];
#pragma unroll
            for (int w = 0; w < kWaves; ++w)
                m = fmaxf(m, ml[w][r][0]);
            const float from = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                weight[w] = __builtin_amdgcn_exp2f(ml[w][r][0] - from);
                total += ml[w][r][1] * weight[w];
            }
            const int part = la.by_run ? part_of<true>(run, p.b, p.base >= run_begin) : part_of<false>(run, p.b, false);
            const int64_t part_row = ((int64_t)part * heads + head) * la.rows + row;
            const int i = row / a.share;
            TQ *out = static_cast<TQ *>(a.out) +
                      (((int64_t)p.b * a.M + i) * heads + head) * a.share * D + (int64_t)(row % a.share) * D;
            const float inverse = total == 0.0f ? 0.0f : 1.0f / (total * kWeight);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
                const int d = 64 * c + 4 * (threadIdx.x & 15);
                f4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < kWaves; ++w)
                    v += *reinterpret_cast<const f4_t *>(&o[w][r][d]) * weight[w];
                if (whole) {
                    if (total == 0.0f)
                        v = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
                    v *= inverse;
                    *reinterpret_cast<Raw8 *>(out + d) = Raw8{pack2<TQ>(v[0], v[1]), pack2<TQ>(v[2], v[3])};
                } else {
                    *reinterpret_cast<f4_t *>(parts.o + part_row * D + d) = v * (1.0f / kWeight);
                }
            }
            if (!whole && (threadIdx.x & 15) == 0) {
                parts.ml[2 * part_row] = m;
                parts.ml[2 * part_row + 1] = total;
            }
        }
        tile = p.base + t1;
        if (tile >= run_end || la.by_sequence)
            break;
        p.base += seq.tiles;
        ++p.b;
        p.seq = sequence(a, scalar_int(a.lens, p.b));
    }
}

// Joins the parts of a row of each sequence, or of each that the end of a run cuts first
// where runs are no more than sequences (every row looks for its sequence among all
// lengths: rows times sequences): kWavesRow waves (all four, or one where rows are
// many: 3840 rows 9.8 us with four, 6.1 with one), 16-byte pieces of D in
// consecutive lanes, the parts over the rest.
template <typename TQ, int D, int kWavesRow, bool kByRun>
__global__ __launch_bounds__(kBlock) void join_kernel(AttendLaunch la)
{
    constexpr int kPer = D / 4, kRows = 64 * kWavesRow / kPer, kThreads = 64 * kWavesRow;
    const AttendArgs &a = la.a;
    const int heads = a.cache.heads;
    const int number = blockIdx.x * (kBlock / kThreads) + (kWavesRow == 1 ? (int)threadIdx.x / 64 : 0);
    if (number >= (kByRun ? la.target - 1 : a.B) * heads * la.rows)
        return;
    const int thread = threadIdx.x % kThreads;
    const int row = number % la.rows, head = (number / la.rows) % heads;
    const int unit = __builtin_amdgcn_readfirstlane(number / (la.rows * heads));
    const Plan p = plan<kByRun>(a, la.target, kByRun ? unit + 1 : unit);   // what the run behind a cut goes on with
    if (p.b < 0)
        return;
    const int b = p.b;
    const int from_run = p.base / p.run, n = (p.base + p.seq.tiles - 1) / p.run - from_run + 1;
    if (n == 1 || (kByRun && from_run != unit))
        return;
    const Parts parts = parts_at(a.workspace, la.units, heads, la.rows, D);
    const int64_t stride = (int64_t)heads * la.rows;
    const int64_t at0 = part_of<kByRun>(from_run, b, false) * stride + (int64_t)head * la.rows + row;
    auto at_part = [&](int c) { return at0 + (kByRun ? 2 * c + (c == 0 ? 1 : 0) : c) * stride; };
    __shared__ float o[kWavesRow == 1 ? 1 : kRows][D], ml[2][kWaves];
    const int lane = thread % kPer, mine = thread / kPer;
    // the largest maximum and the sum under it: a part a thread
    float m = -__builtin_inff();
    for (int c = thread; c < n; c += kThreads)
        m = fmaxf(m, parts.ml[2 * at_part(c)]);
    m = wave_max(m);
    if constexpr (kWavesRow > 1) {
        if ((threadIdx.x & 63) == 0)
            ml[0][threadIdx.x >> 6] = m;
        __syncthreads();
        m = fmaxf(fmaxf(ml[0][0], ml[0][1]), fmaxf(ml[0][2], ml[0][3]));
    }
    const float from = m == -__builtin_inff() ? 0.0f : m;
    float total = 0.0f;
    for (int c = thread; c < n; c += kThreads) {
        const int64_t at = at_part(c);
        total += parts.ml[2 * at + 1] * __builtin_amdgcn_exp2f(parts.ml[2 * at] - from);
    }
    total = wave_sum(total);
    f4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (mine < kRows) {
#pragma unroll 8
        for (int c = mine; c < n; c += kRows) {
            const int64_t at = at_part(c);
            v += *reinterpret_cast<const f4_t *>(parts.o + at * D + 4 * lane) *
                 __builtin_amdgcn_exp2f(parts.ml[2 * at] - from);
        }
    }
    if constexpr (kWavesRow > 1) {
        if ((threadIdx.x & 63) == 0)
            ml[1][threadIdx.x >> 6] = total;
        if (mine < kRows)
            *reinterpret_cast<f4_t *>(&o[mine][4 * lane]) = v;
        __syncthreads();
        total = (ml[1][0] + ml[1][1]) + (ml[1][2] + ml[1][3]);
        if (mine == 0) {
#pragma unroll
            for (int r = 1; r < kRows; ++r)
                v += *reinterpret_cast<const f4_t *>(&o[r][4 * lane]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (kRows >= 4) {
                const f2_t x = pair16(v[i]);
                v[i] = x[0] + x[1];
            }
            if constexpr (kRows >= 2) {
                const f2_t x = pair32(v[i]);
                v[i] = x[0] + x[1];
            }
        }
    }
    if (mine > 0)
        return;
    const float inverse = 1.0f / total;
    if (total == 0.0f)
        v = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
    else
        v *= inverse;
    TQ *out = static_cast<TQ *>(a.out) + (((int64_t)b * a.M + row / a.share) * heads + head) * a.share * D +
              (int64_t)(row % a.share) * D;
    *reinterpret_cast<Raw8 *>(out + 4 * lane) = Raw8{pack2<TQ>(v[0], v[1]), pack2<TQ>(v[2], v[3])};
}

// Tiles of 16 rows a workgroup takes: one or two, more rows in groups that read the
// cache each.  (Four tiles, one wave a SIMD, at 128 dimensions, the cache in part in the
// last-level one: 64 rows a key head in f8 74 us for 56, 128 rows 109 for 85; in bf16 74
// for 55, 106 for 91.)  Two spill 37 registers at 256 dimensions in 16 bits: there one up
// to 48 rows, where two save one group's reading of the cache at most.  One tile / two (us,
// bf16, 20, 48, 64, 96 and 256 rows a key head): 16 sequences of up to 8000, 8 key heads 111 /
// 126, 152 / 155, 178 / 164, 265 / 204, 575 / 380; 8 of 20000, 1 head 36 / 50, 47 / 64, 54 /
// 65, 77 / 75, 110 / 122; 4 of 30000, 8 heads 114 / 125, 159 / 149, 186 / 154, 276 / 190, 610 /
// 364; 64 of 1500, 4 heads 66 / 92, 86 / 124, 108 / 128, 148 / 150, 324 / 292; 1 of 100000,
// 2 heads 69 / 63, 95 / 82, 121 / 83, 120 / 110, 249 / 157.
constexpr bool spills(int D, bool f8) { return D == 256 && !f8; }
int tiles_of_rows(int rows, int D, bool f8) { return rows <= (spills(D, f8) ? 48 : 16) ? 1 : 2; }

struct Cut {
    int rows, tiles, row_groups, target;
    int64_t units;
    bool by_sequence, by_run;
};

Cut cut(int64_t B, int M, int q_heads, int kv_heads, int dim, bool f8, int page, int64_t width, int window)
{
    Cut c;
    c.rows = M * (q_heads / kv_heads);
    c.tiles = tiles_of_rows(c.rows, dim, f8);
    c.row_groups = (c.rows + 16 * c.tiles - 1) / (16 * c.tiles);
    c.target = std::max(1, kRounds * kUnits * resident(dim, f8, c.tiles) / (kv_heads * c.row_groups));
    // no sequence has more tiles than this: no more runs than tiles
    const int64_t places = window ? std::min<int64_t>(width * page, (int64_t)window + M + 16) : width * page;
    const int64_t most = ceil_div(places, kTile);
    c.target = (int)std::min<int64_t>(c.target, B * most);
    c.by_run = c.target <= B;
    c.units = std::min<int64_t>(2 * c.target, c.target + B);
    // A workgroup a sequence: no plan, no second launch (5 us), but the longest sequence is one workgroup's.  Measured
    // (us, runs / a sequence each; f8, D 128, 8 key heads, lengths from 0 to the table's): 1 sequence of 333 9.7 / 7.3,
    // of 1000 9.8 / 11.7 (with the host's part of a second launch 14.4 / 12.1), of 2000 10.2 / 19.0; 32 of up to 2000
    // 22.7 / 19.8, of 4000 32.6 / 35.6; 64 of 4000 49 / 47; 128 of 2000 58 / 47, of 4000 91 / 84.  By bytes of a key
    // head's longest sequence; in bf16 64 of 8190 147 / 167.  In windows of 1200 and 1500 32 of 2000 21.5 / 16.1 and
    // 23.0 / 17.3, of 1500 and 3000 64 of 4000 38 / 33 and 52 / 53.
    // The workspace is sized without the window, so a window may never turn this off: it shortens the sequences of
    // the first rule (down from the table's), the others ask for the table's own.
    const int64_t token = dim * (f8 ? 2 : 4), groups = B * kv_heads * c.row_groups;
    const int64_t bytes = most * kTile * token, table = ceil_div(width * page, kTile) * kTile * token;
    c.by_sequence = bytes <= 256 << 10 || (table <= 512 << 10 && groups >= 256) ||
                    (table <= 1024 << 10 && groups >= 512);
    if (c.by_sequence)
        c.target = (int)B;
    return c;
}

template <typename TQ, bool kF8, int D>
hipError_t launch(const AttendLaunch &la, const Cut &c, hipStream_t stream)
{
    void (*fn)(AttendLaunch);
    if constexpr (spills(D, kF8))   // (two tiles are always groups there)
        fn = c.row_groups == 1 ? &attend_kernel<TQ, kF8, D, 1, true>
             : c.tiles == 1    ? &attend_kernel<TQ, kF8, D, 1, false>
                               : &attend_kernel<TQ, kF8, D, 2, false>;
    else
        fn = c.row_groups > 1 ? &attend_kernel<TQ, kF8, D, 2, false>
             : c.tiles == 1   ? &attend_kernel<TQ, kF8, D, 1, true>
                              : &attend_kernel<TQ, kF8, D, 2, true>;
    const hipError_t e = launch_kernel(reinterpret_cast<const void *>(fn),
                                       dim3((unsigned)(c.target * la.a.cache.heads * c.row_groups)), dim3(kBlock), 0,
                                       stream, la);
    if (e != hipSuccess || c.by_sequence)
        return e;
    const int64_t rows = (int64_t)(c.by_run ? c.target - 1 : la.a.B) * la.a.cache.heads * c.rows;
    if (rows == 0)
        return e;
    const bool many = rows >= kManyRows;
    void (*join)(AttendLaunch) = many ? c.by_run ? &join_kernel<TQ, D, 1, true> : &join_kernel<TQ, D, 1, false>
                                 : c.by_run ? &join_kernel<TQ, D, kWaves, true>
                                            : &join_kernel<TQ, D, kWaves, false>;
    return launch_kernel(reinterpret_cast<const void *>(join),
                         dim3((unsigned)(many ? ceil_div(rows, kBlock / 64) : rows)), dim3(kBlock), 0, stream, la);
}

template <typename TQ, bool kF8>
hipError_t of_dim(const AttendLaunch &la, const Cut &c, hipStream_t stream)
{
    switch (la.a.cache.dim) {
    case 64: return launch<TQ, kF8, 64>(la, c, stream);
    case 128: return launch<TQ, kF8, 128>(la, c, stream);
    case 192: return launch<TQ, kF8, 192>(la, c, stream);
    default: return launch<TQ, kF8, 256>(la, c, stream);
    }
}

}  // namespace

size_t attend_workspace(int64_t B, int M, int q_heads, int kv_heads, int dim, int cache_type, int page, int64_t width)
{
    const Cut c = cut(B, M, q_heads, kv_heads, dim, cache_type == QG_F8, page, width, 0);
    return !c.by_sequence ? (size_t)c.units * kv_heads * c.rows * (dim + 2) * sizeof(float) : 0;
}

hipError_t launch_attend(const AttendArgs &a, int q_type, hipStream_t stream)
{
    // (a window only makes the parts fewer)
    const Cut c = cut(a.B, a.M, a.q_heads, a.cache.heads, a.cache.dim, a.cache.type == QG_F8, a.cache.page, a.width,
                      a.window);
    if (!c.by_sequence && !a.workspace)
        return hipErrorInvalidValue;
    const AttendLaunch la{a, c.target, (int)c.units, c.rows, c.row_groups, c.by_sequence, c.by_run, a.scale * kLog2e,
                          a.softcap > 0.0f ? a.scale / a.softcap : 0.0f,
                          std::min(a.softcap * kLog2e, std::numeric_limits<float>::max())};
    if (a.cache.type == QG_F8)
        return q_type == QG_F16 ? of_dim<Fp16, true>(la, c, stream) : of_dim<Bf16, true>(la, c, stream);
    return q_type == QG_F16 ? of_dim<Fp16, false>(la, c, stream) : of_dim<Bf16, false>(la, c, stream);
}

}  // namespace qg
