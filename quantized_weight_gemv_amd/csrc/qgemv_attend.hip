// Attention of new tokens over the paged cache (definitions in qgemv_attn.h).
//
// Rows are the queries that share a key head: row i share + j is new token i of
// query head j of the group.  One workgroup takes up to 16 kTiles rows of a
// sequence and key head over a part of the cache ("chunk"), its four waves 32
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
// 8-bit codes are widened as they are (exact); a key's scale multiplies its
// score, a value's scale its weight.  A weight (fp32) enters the second product
// as two 16-bit parts, hi = round(p), lo = round(p - hi): 2^-16 of it is lost.
// bf16 for f8 and bf16 values; with fp16 values fp16, taken times 2^14 so that
// small weights stay normal.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "qgemv_attn_internal.h"

namespace qg {
namespace {

constexpr int kBlock = 256;
constexpr int kWaves = kBlock / 64;
constexpr int kStep = 32;                 // tokens of a wave's step
constexpr int kTile = kStep * kWaves;     // tokens of a workgroup's step
constexpr float kLog2e = 1.44269504088896340736f;

// Workgroups that the work is cut for, over all sequences and key heads.
constexpr int kTargetGroups = 1024;

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

// How the work is cut.  A sequence has `tiles` of kTile tokens from `first`
// on; chunks hold up to `chunk` of them.
struct Plan {
    int b;              // sequence
    int part, parts;    // chunk of it, of how many
    int tiles;          // its tiles
    int first;          // its first token that anybody sees, down to a multiple of 16
    int len;
    int base;           // number of its first chunk among all
};

__device__ __forceinline__ int held_length(const AttendArgs &a, int b)
{
    const int64_t most = (int64_t)a.width << a.cache.log_page;
    return (int)min((int64_t)max(a.lens[b], 0), most);
}

__device__ __forceinline__ int first_seen(const AttendArgs &a, int len)
{
    return a.window ? max(0, len - a.M + 1 - a.window) & ~15 : 0;
}

__device__ __forceinline__ int tiles_of(const AttendArgs &a, int len)
{
    return (len - first_seen(a, len) + kTile - 1) / kTile;
}

// Sum over the wave.
__device__ __forceinline__ int wave_total(int v) { return __builtin_amdgcn_readlane(prefix_sum(v), 63); }

// Tiles a chunk: as many as give the target number of workgroups; every wave
// finds it by itself from the lengths.
__device__ __forceinline__ int chunk_tiles(const AttendArgs &a, int target)
{
    const int lane = threadIdx.x & 63;
    int64_t total = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        const int b = b0 + lane;
        total += wave_total(b < a.B ? tiles_of(a, held_length(a, b)) : 0);
    }
    return (int)max((int64_t)1, (total + target - 1) / target);
}

// A sequence without tokens is one chunk without tiles, so that its rows are
// written.
__device__ __forceinline__ int parts_of(int tiles, int chunk) { return max(1, (tiles + chunk - 1) / chunk); }

__device__ __forceinline__ Plan plan_of(const AttendArgs &a, int b, int part, int base, int chunk)
{
    Plan p;
    p.b = b;
    p.len = held_length(a, b);
    p.first = first_seen(a, p.len);
    p.tiles = tiles_of(a, p.len);
    p.parts = parts_of(p.tiles, chunk);
    p.part = part;
    p.base = base;
    return p;
}

// The unit-th chunk of all sequences; b = -1 past the last one.
__device__ __forceinline__ Plan find_chunk(const AttendArgs &a, int unit, int chunk)
{
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int b0 = 0; b0 < a.B; b0 += 64) {
        const int b = b0 + lane;
        const int mine = b < a.B ? parts_of(tiles_of(a, held_length(a, b)), chunk) : 0;
        const int incl = prefix_sum(mine);
        const unsigned long long holds = __ballot(base + incl > unit);
        if (holds) {
            const int src = __ffsll(holds) - 1;
            const int before = base + __builtin_amdgcn_readlane(incl - mine, src);
            return plan_of(a, b0 + src, unit - before, before, chunk);
        }
        base += __builtin_amdgcn_readlane(incl, 63);
    }
    Plan none{};
    none.b = -1;
    return none;
}

// The chunks in front of sequence b.
__device__ __forceinline__ Plan find_sequence(const AttendArgs &a, int b, int chunk)
{
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int b0 = 0; b0 < b; b0 += 64) {
        const int i = b0 + lane;
        base += wave_total(i < b ? parts_of(tiles_of(a, held_length(a, i)), chunk) : 0);
    }
    return plan_of(a, b, 0, base, chunk);
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

// Four codes of a word as 16-bit values, two words.
template <typename T>
__device__ __forceinline__ u2_t widen4(uint32_t w)
{
    if constexpr (std::is_same_v<T, Bf16>) {
        return u2_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))};
    } else {
        return u2_t{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false)),
                    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true))};
    }
}

template <typename T>
__device__ __forceinline__ typename Half<T>::v8 widen8(uint32_t lo, uint32_t hi)
{
    const u2_t a = widen4<T>(lo), b = widen4<T>(hi);
    return __builtin_bit_cast(typename Half<T>::v8, u4_t{a[0], a[1], b[0], b[1]});
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

// Where a chunk's sums go if its sequence has others: accumulators [chunk][key
// head][row][D], then (maximum, sum) [chunk][key head][row].
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

struct AttendLaunch {
    AttendArgs a;
    int target;     // chunks to cut for, per key head and row group
    int units;      // chunks at most
    int rows;       // M share
    int row_groups;
};

// TQ: type of q, of the output and of 16-bit caches; kF8: an 8-bit cache.
template <typename TQ, bool kF8, int D, int kTiles>
__global__ __launch_bounds__(kBlock) void attend_kernel(AttendLaunch la)
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
    constexpr float kWeight = std::is_same_v<TV, Fp16> ? 16384.0f : 1.0f;

    const AttendArgs &a = la.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g = lane >> 4;
    const int heads = a.cache.heads;
    const int head = blockIdx.x % heads;
    const int group = (blockIdx.x / heads) % la.row_groups;
    const int unit = blockIdx.x / (heads * la.row_groups);
    const int chunk = chunk_tiles(a, la.target);
    const Plan p = find_chunk(a, unit, chunk);
    if (p.b < 0)
        return;
    // the tiles of this chunk, even among the chunks of the sequence
    const int t0 = (int)((int64_t)p.part * p.tiles / p.parts), t1 = (int)((int64_t)(p.part + 1) * p.tiles / p.parts);

    // queries: row r is column r of the first product
    typename Q::v8 q[kTiles][kSteps];
    int mine[kTiles];                       // the row's new token
    const int row0 = group * 16 * kTiles;
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
    // a tile's page, and whether there is one
    struct Where {
        const uint8_t *keys, *scales;
        bool there;
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

    u4_t kw[2][kKeyLoads];
    uint32_t vw[8][kValWords];
    uint32_t ks[2], vs[2];
    auto load_keys = [&](const Where (&w)[2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int c = 0; c < kKeyLoads; ++c)
                kw[h][c] = *reinterpret_cast<const u4_t *>(w[h].keys + (r16 * kRow + 64 * c + 16 * g));
            if constexpr (kF8)
                ks[h] = *reinterpret_cast<const uint32_t *>(w[h].scales + 4 * g);
        }
    };
    auto load_values = [&](const Where (&w)[2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t *from = reinterpret_cast<const uint32_t *>(
                    w[h].keys + values + ((4 * g + j) * kRow + r16 * (4 * kValWords)));
                __builtin_memcpy(vw[4 * h + j], __builtin_assume_aligned(from, kValWords % 4 == 0 ? 16 : kValWords % 2 == 0 ? 8 : 4),
                                 4 * kValWords);
            }
            if constexpr (kF8)
                vs[h] = *reinterpret_cast<const uint32_t *>(w[h].scales + a.cache.page + 4 * g);
        }
    };

    f4_t acc[kTiles][kOut];
    float top[kTiles], sum[kTiles];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
        top[n] = -__builtin_inff();
        sum[n] = 0.0f;
#pragma unroll
        for (int d = 0; d < kOut; ++d)
            acc[n][d] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }

    auto add = [&](const typename V::v8 &v, const typename V::v8 (&hi)[kTiles], const typename V::v8 (&lo)[kTiles], int d) {
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
            acc[n][d] = V::mfma(v, lo[n], V::mfma(v, hi[n], acc[n][d]));
    };

    // places that every row sees: from all_from on, below all_end
    const int all_end = p.len - a.M + 1;
    const int all_from = a.window ? max(0, p.len - a.window) : 0;
    const int any_from = a.window ? max(0, all_end - a.window) : 0;
    const float scale = a.softcap > 0.0f ? a.scale / a.softcap : a.scale * kLog2e;
    const float cap = a.softcap * kLog2e;

    auto edge = [&](int at) { return at + kStep > all_end || at < all_from; };
    bool left_out = false;   // values that are not finite, of places that some rows do not see

    const int first = p.first + t0 * kTile + wave * kStep;
    int token = first;
    const int end = min(p.first + t1 * kTile, p.len);
    if (token < end) {
        // pages a step ahead of the loads, loads a half step ahead of their products
        int page[2] = {page_of(token), page_of(token + 16)};
        Where now[2] = {where(page[0], token), where(page[1], token + 16)};
        load_keys(now);
        load_values(now);
        int ahead = token + kTile < end ? token + kTile : token;
        page[0] = page_of(ahead), page[1] = page_of(ahead + 16);
        for (;;) {
            const bool there[2] = {now[0].there, now[1].there};
            // scores
            float s[kTiles][8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f4_t c[kTiles];
#pragma unroll
                for (int n = 0; n < kTiles; ++n)
                    c[n] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int st = 0; st < kSteps; ++st) {
                    typename Q::v8 k;
                    if constexpr (kF8) {
                        const u4_t w = kw[h][st / 2];
                        k = (st & 1) ? widen8<TQ>(w[2], w[3]) : widen8<TQ>(w[0], w[1]);
                    } else {
                        k = __builtin_bit_cast(typename Q::v8, kw[h][st]);
                    }
#pragma unroll
                    for (int n = 0; n < kTiles; ++n)
                        c[n] = Q::mfma(k, q[n][st], c[n]);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float f = scale;
                    if constexpr (kF8)
                        f *= f8_scale((ks[h] >> (8 * i)) & 255u);
#pragma unroll
                    for (int n = 0; n < kTiles; ++n)
                        s[n][4 * h + i] = c[n][i] * f;
                }
            }
            // the next step's keys
            now[0] = where(page[0], ahead), now[1] = where(page[1], ahead + 16);
            load_keys(now);
            if (a.softcap > 0.0f) {
#pragma unroll
                for (int n = 0; n < kTiles; ++n)
#pragma unroll
                    for (int i = 0; i < 8; ++i)   // cap tanh(x) log2 e, from e^2x
                        s[n][i] = cap - 2.0f * cap * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(s[n][i] * (2.0f * kLog2e)));
            }
            if (edge(token) || !there[0] || !there[1]) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = token + 16 * (i / 4) + 4 * g + (i & 3);
                    const bool is = there[i / 4];
#pragma unroll
                    for (int n = 0; n < kTiles; ++n) {
                        const int stop = p.len - a.M + 1 + mine[n], start = a.window ? stop - a.window : 0;
                        if (!is || at >= stop || at < start)
                            s[n][i] = -__builtin_inff();
                    }
                    const bool seen = is && at < p.len && at >= any_from;
#pragma unroll
                    for (int c = 0; c < kValWords; ++c) {
                        if (!seen)
                            vw[i][c] = 0;
                        // 0 times what is not finite is not 0: what some rows see and others do not comes afterwards
                        const uint32_t odd = not_finite<TQ, kF8>(vw[i][c]);
                        if (a.M > 1 && odd) {
                            vw[i][c] &= ~odd;
                            left_out = true;
                        }
                    }
                }
            }
            // softmax
            typename V::v8 hi[kTiles], lo[kTiles];
#pragma unroll
            for (int n = 0; n < kTiles; ++n) {
                float m = top[n];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    m = fmaxf(m, s[n][i]);
                m = max_over_groups(m);
                if (__any(m > top[n])) {
                    const float old = __builtin_amdgcn_exp2f(top[n] - (m == -__builtin_inff() ? 0.0f : m));
                    sum[n] *= old;
#pragma unroll
                    for (int d = 0; d < kOut; ++d)
                        acc[n][d] *= old;
                    top[n] = m;
                }
                const float from = m == -__builtin_inff() ? 0.0f : m;
                float w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float e = __builtin_amdgcn_exp2f(s[n][i] - from);
                    sum[n] += e;
                    w[i] = e * kWeight;
                    if constexpr (kF8) {
                        const float f = f8_scale((vs[i / 4] >> (8 * (i & 3))) & 255u);
                        w[i] = e == 0.0f ? 0.0f : e * f;   // (the scale of a place without a token may be anything)
                    }
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
                    const u4_t x = turn4(vw[0][c], vw[1][c], vw[2][c], vw[3][c]);
                    const u4_t y = turn4(vw[4][c], vw[5][c], vw[6][c], vw[7][c]);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        add(widen8<TV>(x[i], y[i]), hi, lo, 4 * c + i);
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t half = i ? 0x07060302 : 0x05040100;
                        add(__builtin_bit_cast(typename V::v8, u4_t{__builtin_amdgcn_perm(vw[1][c], vw[0][c], half),
                                                                    __builtin_amdgcn_perm(vw[3][c], vw[2][c], half),
                                                                    __builtin_amdgcn_perm(vw[5][c], vw[4][c], half),
                                                                    __builtin_amdgcn_perm(vw[7][c], vw[6][c], half)}),
                            hi, lo, 2 * c + i);
                    }
                }
            }
            load_values(now);
            token += kTile;
            if (token >= end)
                break;
            ahead = token + kTile < end ? token + kTile : token;
            page[0] = page_of(ahead), page[1] = page_of(ahead + 16);
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
            for (int t = at; t < min(at + kStep, p.len); ++t) {
                const Where w = where(page_of(t), t);
                if (!w.there)
                    continue;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t *from = reinterpret_cast<const uint32_t *>(w.keys + values + (4 * g + e) * (4 * kValWords));
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
    __shared__ float o[kWaves][16][D + 4];
    __shared__ float ml[kWaves][16][2];
    const Parts parts = parts_at(a.workspace, la.units, heads, la.rows, D);
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
        const float l = sum_over_groups(sum[n]);
        if (n > 0)
            __syncthreads();
        if (g == 0)
            ml[wave][r16][0] = top[n], ml[wave][r16][1] = l;
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
        const int64_t part_row = ((int64_t)unit * heads + head) * la.rows + row;
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
            if (p.parts == 1) {
                if (total == 0.0f)
                    v = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
                v *= inverse;
                *reinterpret_cast<Raw8 *>(out + d) = Raw8{pack2<TQ>(v[0], v[1]), pack2<TQ>(v[2], v[3])};
            } else {
                *reinterpret_cast<f4_t *>(parts.o + part_row * D + d) = v * (1.0f / kWeight);
            }
        }
        if (p.parts > 1 && (threadIdx.x & 15) == 0) {
            parts.ml[2 * part_row] = m;
            parts.ml[2 * part_row + 1] = total;
        }
    }
}

// Joins the chunks of a row: a workgroup per row of a sequence and key head,
// 16-byte pieces of D in consecutive threads, the chunks over the rest.
template <typename TQ, int D>
__global__ __launch_bounds__(kBlock) void join_kernel(AttendLaunch la)
{
    constexpr int kPer = D / 4, kRows = kBlock / kPer;
    const AttendArgs &a = la.a;
    const int heads = a.cache.heads;
    const int row = blockIdx.x % la.rows, head = (blockIdx.x / la.rows) % heads, b = blockIdx.x / (la.rows * heads);
    const int chunk = chunk_tiles(a, la.target);
    const Plan p = find_sequence(a, b, chunk);
    if (p.parts == 1)
        return;
    const Parts parts = parts_at(a.workspace, la.units, heads, la.rows, D);
    const int64_t stride = (int64_t)heads * la.rows, at0 = (int64_t)p.base * stride + (int64_t)head * la.rows + row;
    __shared__ float o[kRows][D], ml[kRows][2];
    const int lane = threadIdx.x % kPer, mine = threadIdx.x / kPer;
    float m = -__builtin_inff(), total = 0.0f;
    f4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
    if (mine < kRows) {
        for (int c = mine; c < p.parts; c += kRows) {
            const int64_t at = at0 + c * stride;
            const float mc = parts.ml[2 * at], lc = parts.ml[2 * at + 1];
            const f4_t x = *reinterpret_cast<const f4_t *>(parts.o + at * D + 4 * lane);
            const float to = fmaxf(m, mc), from = to == -__builtin_inff() ? 0.0f : to;
            const float wm = __builtin_amdgcn_exp2f(m - from), wc = __builtin_amdgcn_exp2f(mc - from);
            v = v * wm + x * wc;
            total = total * wm + lc * wc;
            m = to;
        }
        *reinterpret_cast<f4_t *>(&o[mine][4 * lane]) = v;
        if (lane == 0)
            ml[mine][0] = m, ml[mine][1] = total;
    }
    __syncthreads();
    if (mine > 0)
        return;
    m = -__builtin_inff();
#pragma unroll
    for (int r = 0; r < kRows; ++r)
        m = fmaxf(m, ml[r][0]);
    const float from = m == -__builtin_inff() ? 0.0f : m;
    total = 0.0f;
    v = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        const float w = __builtin_amdgcn_exp2f(ml[r][0] - from);
        v += *reinterpret_cast<const f4_t *>(&o[r][4 * lane]) * w;
        total += ml[r][1] * w;
    }
    const float inverse = 1.0f / total;
    if (total == 0.0f)
        v = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
    else
        v *= inverse;
    TQ *out = static_cast<TQ *>(a.out) + (((int64_t)b * a.M + row / a.share) * heads + head) * a.share * D +
              (int64_t)(row % a.share) * D;
    *reinterpret_cast<Raw8 *>(out + 4 * lane) = Raw8{pack2<TQ>(v[0], v[1]), pack2<TQ>(v[2], v[3])};
}

// Tiles of 16 rows a workgroup takes: all rows where their accumulators fit the
// registers, else several groups read the cache anew.
int tiles_of_rows(int rows, int D)
{
    const int most = D <= 128 ? 4 : 2;
    const int tiles = (rows + 15) / 16;
    return tiles <= 1 ? 1 : tiles == 2 ? 2 : most;
}

struct Cut {
    int rows, tiles, row_groups, target;
    int64_t units;
    bool join;
};

Cut cut(int64_t B, int M, int q_heads, int kv_heads, int dim, int page, int64_t width)
{
    Cut c;
    c.rows = M * (q_heads / kv_heads);
    c.tiles = tiles_of_rows(c.rows, dim);
    c.row_groups = (c.rows + 16 * c.tiles - 1) / (16 * c.tiles);
    c.target = std::max(1, kTargetGroups / (kv_heads * c.row_groups));
    // a sequence has at most this many tiles (a window's first one may be cut); chunks of one tile at least
    const int64_t most = ceil_div(width * page, kTile) + 1;
    c.units = std::min(B * most, c.target + B);
    c.join = width * page > kTile;
    if (!c.join)
        c.units = B;
    return c;
}

template <typename TQ, bool kF8, int D>
hipError_t launch(const AttendLaunch &la, const Cut &c, hipStream_t stream)
{
    void (*fn)(AttendLaunch) = nullptr;
    if (c.tiles == 1)
        fn = &attend_kernel<TQ, kF8, D, 1>;
    else if (c.tiles == 2)
        fn = &attend_kernel<TQ, kF8, D, 2>;
    else if constexpr (D <= 128)
        fn = &attend_kernel<TQ, kF8, D, 4>;
    const hipError_t e = launch_kernel(reinterpret_cast<const void *>(fn),
                                       dim3((unsigned)(c.units * la.a.cache.heads * c.row_groups)), dim3(kBlock), 0,
                                       stream, la);
    if (e != hipSuccess || !c.join)
        return e;
    void (*join)(AttendLaunch) = &join_kernel<TQ, D>;
    return launch_kernel(reinterpret_cast<const void *>(join), dim3((unsigned)(la.a.B * la.a.cache.heads * c.rows)),
                         dim3(kBlock), 0, stream, la);
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

size_t attend_workspace(int64_t B, int M, int q_heads, int kv_heads, int dim, int page, int64_t width)
{
    const Cut c = cut(B, M, q_heads, kv_heads, dim, page, width);
    return c.join ? (size_t)c.units * kv_heads * c.rows * (dim + 2) * sizeof(float) : 0;
}

hipError_t launch_attend(const AttendArgs &a, int q_type, hipStream_t stream)
{
    const Cut c = cut(a.B, a.M, a.q_heads, a.cache.heads, a.cache.dim, a.cache.page, a.width);
    const AttendLaunch la{a, c.target, (int)c.units, c.rows, c.row_groups};
    if (a.cache.type == QG_F8)
        return q_type == QG_F16 ? of_dim<Fp16, true>(la, c, stream) : of_dim<Bf16, true>(la, c, stream);
    return q_type == QG_F16 ? of_dim<Fp16, false>(la, c, stream) : of_dim<Bf16, false>(la, c, stream);
}

}  // namespace qg
