// Norms of query and key heads with the rotation of positions, forward and
// backward, and the paged cache written and read back (definitions in
// qgemv_attn.h).
//
// L lanes hold a head vector (8, 16 or 32 for up to 64, 128 and 256 elements), a
// wave 64 / L heads of one token.  A lane's eight elements are four pairs of the
// rotation: halves (i and i + rot / 2, two pieces of four) or neighbours (eight
// in a row), so nothing moves between lanes but the sum of squares.  The four
// cosines and sines of a lane are the same for every head of a token: a wave
// takes them once and walks over the heads.
//
// Bound by bytes from some ten thousand tokens on: 16384 tokens of 32 + 8 heads of 128
// in bf16 forward 66 us (5.1 TB/s), backward 89 (5.6) and 5 for the sums of the
// gains, in fp32 124 (5.4) and 187 (5.4); 8192 tokens of 40 + 8 + 8 heads into a 16-bit
// cache 48 us (4.9), with norms into an 8-bit one 58 (3.8: the keys in 64 bits take 127
// registers and more, and three waves a SIMD); 16384 tokens of 8 heads into an 8-bit cache 19
// us (5.2), back 18 (5.7).  Some thousand tokens are bound by the vector units: 2731 of 14
// + 2 heads of 96 on three axes 12 us forward for 3.3 us of bytes, since every group of lanes
// of a wave, and the token's other wave, computes the same cosines in 64 bits.  A few
// tokens take 4 us: a launch, the loads' latency and the series.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "qgemv_attn_internal.h"

namespace qg {
namespace {

constexpr int kBlock = 256;
constexpr int kMaxBlocks = 1 << 20;
// 1 / (2 pi) and what its 64 bits leave out.
constexpr double kInvTwoPi = 0.15915494309189535, kInvTwoPiRest = -9.839338337591243e-18;

struct __attribute__((packed, aligned(4))) Raw16f {
    uint32_t w[4];
};

// A lane's eight elements as they lie in memory, loaded ahead of their use.
template <typename T>
struct Eight {
    typedef uint32_t Piece __attribute__((ext_vector_type(sizeof(T)), aligned(sizeof(T))));
    Piece p[2];
    template <bool kOnce = false>
    __device__ __forceinline__ void load(const T *row, int lo, int hi)
    {
        if constexpr (kOnce) {
            p[0] = __builtin_nontemporal_load(reinterpret_cast<const Piece *>(row + lo));
            p[1] = __builtin_nontemporal_load(reinterpret_cast<const Piece *>(row + hi));
        } else {
            p[0] = *reinterpret_cast<const Piece *>(row + lo);
            p[1] = *reinterpret_cast<const Piece *>(row + hi);
        }
    }
    // all zeros unless `on`
    template <typename F>
    __device__ __forceinline__ void values(bool on, F (&v)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x;
            if constexpr (sizeof(T) == 4)
                x = __uint_as_float(p[i / 4][i & 3]);
            else
                x = to_f32(T{(uint16_t)(p[i / 4][(i & 3) / 2] >> (16 * (i & 1)))});
            v[i] = on ? x : 0.0f;
        }
    }
};

template <typename T>
__device__ __forceinline__ void load4(const T *p, float *v)
{
    if constexpr (sizeof(T) == 4) {
        const Raw16f r = *reinterpret_cast<const Raw16f *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = __uint_as_float(r.w[i]);
    } else {
        const Raw8 r = *reinterpret_cast<const Raw8 *>(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = to_f32(T{(uint16_t)(r.w[i / 2] >> (16 * (i & 1)))});
    }
}

// Stores of large outputs leave nothing behind in the caches (kOnce).
template <bool kOnce, typename T>
__device__ __forceinline__ void store4(T *p, float a, float b, float c, float d)
{
    typedef uint32_t Piece __attribute__((ext_vector_type(sizeof(T)), aligned(sizeof(T))));
    Piece r;
    if constexpr (sizeof(T) == 4)
        r = Piece{__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d)};
    else
        r = Piece{pack2<T>(a, b), pack2<T>(c, d)};
    if constexpr (kOnce)
        __builtin_nontemporal_store(r, reinterpret_cast<Piece *>(p));
    else
        *reinterpret_cast<Piece *>(p) = r;
}

// A lane's eight elements from `lo` and `hi` of a vector; the type is the
// launch's, so the branches are the wave's.
__device__ __forceinline__ void load8_as(int type, const void *base, int64_t at, int lo, int hi, float (&v)[8])
{
    if (type == QG_F32) {
        load4(static_cast<const float *>(base) + at + lo, v);
        load4(static_cast<const float *>(base) + at + hi, v + 4);
    } else if (type == QG_F16) {
        load4(static_cast<const Fp16 *>(base) + at + lo, v);
        load4(static_cast<const Fp16 *>(base) + at + hi, v + 4);
    } else {
        load4(static_cast<const Bf16 *>(base) + at + lo, v);
        load4(static_cast<const Bf16 *>(base) + at + hi, v + 4);
    }
}
template <bool kOnce, typename T>
__device__ __forceinline__ void store8(T *row, int lo, int hi, const float (&v)[8])
{
    store4<kOnce>(row + lo, v[0], v[1], v[2], v[3]);
    store4<kOnce>(row + hi, v[4], v[5], v[6], v[7]);
}
template <bool kOnce = false>
__device__ __forceinline__ void store8_as(int type, void *base, int64_t at, int lo, int hi, const float (&v)[8])
{
    // (a copy in front of the branches keeps the values in registers)
    const float w[8] = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
    if (type == QG_F32)
        store8<kOnce>(static_cast<float *>(base) + at, lo, hi, w);
    else if (type == QG_F16)
        store8<kOnce>(static_cast<Fp16 *>(base) + at, lo, hi, w);
    else
        store8<kOnce>(static_cast<Bf16 *>(base) + at, lo, hi, w);
}

// (the declaration of fp32 stands beside that of 64 bits)
using qg::dpp;

template <int kCtrl>
__device__ __forceinline__ double dpp(double v)
{
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, kCtrl, 0xF, 0xF, true);
    const uint32_t hi =
        (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), kCtrl, 0xF, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// A wave's lane inside its head vector.
struct Place {
    int sub, l;     // head of the group, lane of the head
    bool on;        // has elements
    bool turned;    // its pairs are turned
    int lo, hi;     // its elements: lo .. lo + 3, hi .. hi + 3
};

template <int L>
__device__ __forceinline__ Place place(int D, int half, bool interleaved)
{
    const int lane = threadIdx.x & 63;
    Place p;
    p.sub = lane / L;
    p.l = lane % L;
    p.on = 8 * p.l < D;
    p.turned = p.on && 4 * p.l < half;
    // (nothing turned: halves of the vector, whose pieces are whole lines over the lanes)
    const bool halves = half == 0 || (p.turned && !interleaved);
    p.lo = halves ? 4 * p.l : 8 * p.l;
    p.hi = halves ? (half ? half : D / 2) + 4 * p.l : 8 * p.l + 4;
    return p;
}

// sin and cos of `turn` whole turns, to a few 2^-53: the nearest quarter is taken
// out, the rest, up to an eighth, goes through the series of both (coefficients
// (2 pi)^k / k!, the first term left out below 2^-54).
__device__ __forceinline__ void sin_cos(double turn, double &s, double &c)
{
    constexpr double kSin[] = {6.283185307179586, -41.34170224039976, 81.60524927607506, -76.70585975306139,
                               42.058693944897655, -15.09464257682299, 3.819952584848282, -0.7181223017785006};
    constexpr double kCos[] = {1.0, -19.739208802178716, 64.9393940226683, -85.45681720669373,
                               60.24464137187666, -26.4262567833744, 7.903536371318469, -1.714390711088672,
                               0.28200596845579123};
    const double quarter = rint(4.0 * turn);
    const double r = fma(quarter, -0.25, turn), z = r * r;
    double a = kSin[7], b = kCos[8];
#pragma unroll
    for (int i = 6; i >= 0; --i)
        a = fma(a, z, kSin[i]);
#pragma unroll
    for (int i = 7; i >= 0; --i)
        b = fma(b, z, kCos[i]);
    a *= r;
    const int q = (int)quarter;
    s = (q & 1) ? b : a;
    c = (q & 1) ? a : b;
    s = (q & 2) ? -s : s;
    c = ((q + 1) & 2) ? -c : c;
}

// position * freq / 2 pi without its whole turns.  The product of the two is exact in
// two parts, 1 / 2 pi has two parts, and the whole turns leave by an fma: the error is
// 2^-53 of a turn wherever the position is, where products of one part are off by
// 2^-53 of all the turns (half a step of an fp32 cosine from positions of 2^27 on).
__device__ __forceinline__ double turn_of(int position, float freq)
{
    const double angle = (double)position * (double)freq;
    const double rest = fma((double)position, (double)freq, -angle);
    const double whole = rint(angle * kInvTwoPi);
    return fma(angle, kInvTwoPi, -whole) + fma(angle, kInvTwoPiRest, rest * kInvTwoPi);
}

// Cosines and sines of the four pairs of a lane at a token's positions, in 64 bits
// too (the vector units do those as fast as fp32), so that in fp32 they are the
// nearest ones but for a value within a few 2^-53 of a border.
template <typename F>
__device__ __forceinline__ void turns(const HeadArgs &a, const Place &p, int64_t t, F (&c)[4], F (&s)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = 1, s[i] = 0;
    if (!p.turned)
        return;
    const Raw16f f = *reinterpret_cast<const Raw16f *>(a.freq + 4 * p.l);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int axis = 0;
        for (int j = 0; j + 1 < a.axes; ++j)
            axis += 4 * p.l + i >= a.sections[j] ? 1 : 0;
        double sine, cosine;
        sin_cos(turn_of(a.positions[axis * a.T + t], __uint_as_float(f.w[i])), sine, cosine);
        c[i] = (F)cosine, s[i] = (F)sine;
    }
}

// kCopy: a copy in front of the branches keeps the values in registers.  The gradient
// needs it (without one a lane's eight values went to memory and back for every head
// with fp32 inputs: 16384 tokens of 32 + 8 heads, inputs and gradients in fp32, 282 us
// for 196); the kernels that write a cache would take five more registers and a wave less.
template <bool kCopy = false, typename F>
__device__ __forceinline__ void turn(const Place &p, bool interleaved, const F (&c)[4], const F (&s)[4], F (&v)[8])
{
#pragma clang fp contract(off)   // each product rounds by itself, as in a program of separate operations
    if (!p.turned)
        return;   // (what is not turned is left as it is, infinities too)
    const F copy[8] = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
    const F(&w)[8] = kCopy ? copy : v;
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const F x = w[2 * i], y = w[2 * i + 1];
            v[2 * i] = x * c[i] - y * s[i];
            v[2 * i + 1] = y * c[i] + x * s[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const F x = w[i], y = w[4 + i];
            v[i] = x * c[i] - y * s[i];
            v[4 + i] = y * c[i] + x * s[i];
        }
    }
}

// 1 / sqrt(v), the nearest fp32 value: the hardware's 64-bit estimate (2^-24) and one
// step of Newton's method, which squares its error.
__device__ __forceinline__ float inverse_root(float v)
{
    const double x = v, r = __builtin_amdgcn_rsq(x);
    const double better = fma(0.5 * r, fma(-x * r, r, 1.0), r);
    return v > 0.0f && v < __builtin_inff() ? (float)better : rsqrtf(v);
}
__device__ __forceinline__ double inverse_root(double v) { return 1.0 / sqrt(v); }

// One step of a sum over the lanes of a group: lanes `kStep` apart hold sums of as
// many lanes each.
template <int kStep, typename F>
__device__ __forceinline__ F add_lanes(F v)
{
    if constexpr (kStep == 16 && sizeof(F) == 4) {
        const f2_t p = pair16(v);
        return p[0] + p[1];
    } else if constexpr (kStep == 16) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const f2_t lo = pair16(__uint_as_float((uint32_t)u)), hi = pair16(__uint_as_float((uint32_t)(u >> 32)));
        auto of = [](float h, float l) {
            return __builtin_bit_cast(double, (uint64_t)__float_as_uint(h) << 32 | __float_as_uint(l));
        };
        return of(hi[0], lo[0]) + of(hi[1], lo[1]);
    } else {
        return v + dpp<kStep == 1 ? 0xB1 : kStep == 2 ? 0x4E : kStep == 4 ? 0x141 : 0x140>(v);
    }
}

// 1 / sqrt(mean of squares + eps).  Squares round by themselves and are summed four
// neighbours first (one after the other; in pairs up to 64 elements), then
// neighbouring fours: the order in which the mean of a row of 64, 128 or 256 is
// taken by separate operations on this card.  Any order is as exact; in this one those
// give the same bits (a test compares them), so that 16-bit caches hold the same bytes
// whichever of the two wrote them.  The first `split` lanes (a power of two) have one four of either half of the turned
// elements: the halves are summed apart until they are neighbours.
template <int L, typename F>
__device__ __forceinline__ F inverse_norm(const F (&v)[8], int split, F inverse_dim, float eps)
{
#pragma clang fp contract(off)
    F four[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const F a = v[4 * i] * v[4 * i], b = v[4 * i + 1] * v[4 * i + 1];
        const F c = v[4 * i + 2] * v[4 * i + 2], d = v[4 * i + 3] * v[4 * i + 3];
        four[i] = L == 8 ? (a + b) + (c + d) : ((a + b) + c) + d;
    }
    const bool apart = (int)(threadIdx.x % L) < split;
    F ss = apart ? four[0] : four[0] + four[1], other = apart ? four[1] : (F)0;
    auto step = [&](auto lanes) {
        constexpr int kStep = decltype(lanes)::value;
        if (kStep == split)
            ss += other;
        ss = add_lanes<kStep>(ss);
        if (kStep < split)
            other = add_lanes<kStep>(other);
    };
    step(std::integral_constant<int, 1>{});
    step(std::integral_constant<int, 2>{});
    step(std::integral_constant<int, 4>{});
    if constexpr (L >= 16)
        step(std::integral_constant<int, 8>{});
    if constexpr (L >= 32)
        step(std::integral_constant<int, 16>{});
    if (split >= L)
        ss += other;
    return inverse_root(ss * inverse_dim + (F)eps);
}

// The same of 192 elements: separate operations take 32 sums there, the first 16 of
// two fours added element by element.  No lanes hold those, so the squares go through
// LDS, within the wave (8192 tokens of 40 + 8 + 8 heads into a 16-bit cache and read
// back 113 us, 111 in the lanes' own order).
__device__ __forceinline__ float inverse_norm_192(const Place &p, const float (&v)[8], float eps)
{
#pragma clang fp contract(off)
    __shared__ __attribute__((aligned(16))) float squares[kBlock / 64][2][192];
    float *row = squares[threadIdx.x >> 6][p.sub];
    if (p.on) {
        *reinterpret_cast<f4_t *>(row + p.lo) = f4_t{v[0] * v[0], v[1] * v[1], v[2] * v[2], v[3] * v[3]};
        *reinterpret_cast<f4_t *>(row + p.hi) = f4_t{v[4] * v[4], v[5] * v[5], v[6] * v[6], v[7] * v[7]};
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    f4_t q = *reinterpret_cast<const f4_t *>(row + 4 * p.l);
    if (p.l < 16)
        q += *reinterpret_cast<const f4_t *>(row + 128 + 4 * p.l);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();   // (the next vector's squares)
    float ss = ((q[0] + q[1]) + q[2]) + q[3];
    ss = add_lanes<1>(ss);
    ss = add_lanes<2>(ss);
    ss = add_lanes<4>(ss);
    ss = add_lanes<8>(ss);
    ss = add_lanes<16>(ss);
    return inverse_root(ss * (1.0f / 192.0f) + eps);
}

// A lane's eight values of an f8 vector held by L lanes: codes and scale byte,
// by the rule of f8_quantize16.
template <int L>
__device__ __forceinline__ uint32_t quantize8(float (&v)[8], uint32_t (&w)[2])
{
    auto largest = [&] {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = fmaxf(m, fabsf(v[i]));
        return group_max<L>(m);
    };
    float amax = largest();
    if (__any(amax == __builtin_inff())) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = fabsf(v[i]) < __builtin_inff() ? v[i] : __builtin_nanf("");
        amax = largest();
    }
    const uint32_t byte = f8_scale_byte(__float_as_uint(amax));
    if (__any(byte == 120 + 127)) {
        const float most = byte == 120 + 127 ? 0x1.ep127f : __builtin_inff();
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = fabsf(v[i]) > most ? copysignf(most, v[i]) : v[i];
    }
    const float inv = f8_inverse(byte);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = f8_pack4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
    return byte;
}

// The fp32 value below a 64-bit one in magnitude with the last bit set if
// anything was cut: rounding it to fewer bits gives what rounding the 64-bit
// value gives.
__device__ __forceinline__ float sticky(double v)
{
    const float f = __double2float_rz(v);
    return (double)f != v ? __uint_as_float(__float_as_uint(f) | 1u) : f;
}

// A head's vector of a cache slot: element and scale addresses.
struct SlotAt {
    uint8_t *codes, *scale;
};
__device__ __forceinline__ SlotAt slot_at(const KvCache &c, int slot, int head, int kv)
{
    uint8_t *page = c.data + (int64_t)(slot >> c.log_page) * c.page_bytes;
    const int row = (head * 2 + kv) * c.page + (slot & (c.page - 1));
    return SlotAt{page + (int64_t)row * c.dim * (c.type == QG_F8 ? 1 : 2), page + c.scales + row};
}

// Eight values of a lane into a slot's vector.
template <int L>
__device__ __forceinline__ void put(const KvCache &c, int slot, int head, int kv, bool on, int l, int lo, int hi,
                                    float (&v)[8])
{
    if (c.type == QG_F8) {
        uint32_t w[2];
        const uint32_t byte = quantize8<L>(v, w);
        if (on) {
            const SlotAt at = slot_at(c, slot, head, kv);
            *reinterpret_cast<uint32_t *>(at.codes + lo) = w[0];
            *reinterpret_cast<uint32_t *>(at.codes + hi) = w[1];
            if (l == 0)
                *at.scale = (uint8_t)byte;
        }
    } else if (on) {
        store8_as(c.type, slot_at(c, slot, head, kv).codes, 0, lo, hi, v);
    }
}

// A head's vector normed and turned, in fp32 or 64 bits.
template <int L, typename F>
__device__ __forceinline__ void norm_turn(const HeadArgs &a, const Place &p, const float (&gain)[8], const F (&c)[4],
                                          const F (&s)[4], F (&v)[8])
{
#pragma clang fp contract(off)
    if (a.gain[0]) {
        F r;
        if constexpr (L == 32 && sizeof(F) == 4)
            r = a.D == 192 ? inverse_norm_192(p, v, a.eps) : inverse_norm<L>(v, a.split, (F)1 / (F)a.D, a.eps);
        else
            r = inverse_norm<L>(v, a.split, (F)1 / (F)a.D, a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = v[i] * r * (F)gain[i];
    }
    turn(p, a.interleaved, c, s, v);
}

// A wave takes the blockIdx.y-th part of a token's groups of heads: query heads,
// key heads and, when they are written to a cache, value heads.  The next group is
// loaded ahead; the first one lies behind the cosines.
template <typename T, int L, bool kWrite, bool kF8, bool kOnce>
__global__ __launch_bounds__(kBlock) void head_kernel(HeadArgs a)
{
    const Place p = place<L>(a.D, a.half, a.interleaved);
    const int k0 = a.groups[0], v0 = k0 + a.groups[1], all = v0 + (kWrite ? a.groups[2] : 0);
    // (lanes without elements take the first ones' gains: a vector's quantization looks at their zeros too)
    float gain[2][8];
    if (a.gain[0]) {
        const int lo = p.on ? p.lo : 0, hi = p.on ? p.hi : 4;
        load8_as(a.gain_type, a.gain[0], 0, lo, hi, gain[0]);
        load8_as(a.gain_type, a.gain[1], 0, lo, hi, gain[1]);
    }
    const int first = (int)(blockIdx.y * all / gridDim.y), upto = (int)((blockIdx.y + 1) * all / gridDim.y);
    for (int64_t t = (int64_t)blockIdx.x * (kBlock / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); t < a.T;
         t += (int64_t)gridDim.x * (kBlock / 64)) {
        int last = upto;
        int slot = 0;
        if constexpr (kWrite) {
            if (last > k0) {
                slot = a.slots[t];
                if ((uint32_t)slot >= (uint32_t)a.cache.pages << a.cache.log_page)
                    last = min(last, k0);
            }
        }
        if (first >= last)
            continue;
        Eight<T> x;
        int head;
        bool on;
        auto fetch = [&](int group) {
            const int kind = group < k0 ? 0 : !kWrite || group < v0 ? 1 : 2;
            head = (group - (kind == 0 ? 0 : kind == 1 ? k0 : v0)) * (64 / L) + p.sub;
            on = p.on && head < (kind == 0 ? a.heads[0] : a.heads[1]);
            const void *base = kind == 0 ? a.x[0] : kind == 1 ? a.x[1] : a.x[2];
            const int64_t ld = kind == 0 ? a.ldx[0] : kind == 1 ? a.ldx[1] : a.ldx[2];
            if (on)
                x.template load<kWrite>(static_cast<const T *>(base) + t * ld + head * a.D, p.lo, p.hi);
        };
        fetch(first);
        float c[4], s[4];
        double cd[4], sd[4];
        if (first < v0) {
            if constexpr (kF8) {
                turns(a, p, t, cd, sd);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    c[i] = (float)cd[i], s[i] = (float)sd[i];
            } else {
                turns(a, p, t, c, s);
            }
        }
        for (int group = first; group < last; ++group) {
            const Eight<T> now = x;
            const int h = head;
            const bool is = on;
            if (group + 1 < last)
                fetch(group + 1);
            float v[8];
            if (kWrite && kF8 && group >= k0 && group < v0) {
                double w[8];
                now.values(is, w);
                norm_turn<L>(a, p, gain[1], cd, sd, w);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = sticky(w[i]);
                put<L>(a.cache, slot, h, 0, is, p.l, p.lo, p.hi, v);
                continue;
            }
            now.values(is, v);
            if (group < k0) {
                norm_turn<L>(a, p, gain[0], c, s, v);
                if (is)
                    store8_as<kOnce>(a.y_type, a.y[0], t * a.ldy[0] + h * a.D, p.lo, p.hi, v);
            } else if (group < v0) {
                norm_turn<L>(a, p, gain[1], c, s, v);
                if constexpr (kWrite)
                    put<L>(a.cache, slot, h, 0, is, p.l, p.lo, p.hi, v);
                else if (is)
                    store8_as<kOnce>(a.y_type, a.y[1], t * a.ldy[1] + h * a.D, p.lo, p.hi, v);
            } else if constexpr (kWrite) {
                put<L>(a.cache, slot, h, 1, is, p.l, p.lo, p.hi, v);
            }
        }
    }
}

// The gradient.  With h the output's gradient turned back and n = x r the
// normed row:  dgain += h n,  dx = r (h gain - n mean(h gain n)).  A lane keeps
// its eight sums of each gain over all the heads and tokens of its wave; the
// workgroup leaves one row of sums.
template <typename T, typename TY, int L, bool kOnce>
__global__ __launch_bounds__(kBlock) void head_backward_kernel(HeadGradArgs ga)
{
    const HeadArgs &a = ga.h;
    const Place p = place<L>(a.D, a.half, a.interleaved);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const bool normed = a.gain[0] != nullptr;
    const float inverse_dim = 1.0f / (float)a.D;
    float dg[2][8], gain[2][8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            dg[k][i] = 0.0f, gain[k][i] = 1.0f;
        if (normed && p.on)
            load8_as(a.gain_type, a.gain[k], 0, p.lo, p.hi, gain[k]);
    }
    const int all = a.groups[0] + a.groups[1];
    const int first = (int)(blockIdx.y * all / gridDim.y), last = (int)((blockIdx.y + 1) * all / gridDim.y);
    for (int64_t t = (int64_t)blockIdx.x * (kBlock / 64) + wave; t < a.T; t += (int64_t)gridDim.x * (kBlock / 64)) {
        Eight<T> x;
        Eight<TY> dy;
        int head;
        bool on;
        const int k0 = a.groups[0];
        auto fetch = [&](int group) {
            const bool key = group >= k0;
            head = (key ? group - k0 : group) * (64 / L) + p.sub;
            on = p.on && head < (key ? a.heads[1] : a.heads[0]);
            if (on) {
                dy.load(static_cast<const TY *>(key ? a.y[1] : a.y[0]) + t * (key ? a.ldy[1] : a.ldy[0]) + head * a.D,
                        p.lo, p.hi);
                if (normed)
                    x.load(static_cast<const T *>(key ? a.x[1] : a.x[0]) + t * (key ? a.ldx[1] : a.ldx[0]) +
                               head * a.D, p.lo, p.hi);
            }
        };
        fetch(first);
        float c[4], s[4];
        turns(a, p, t, c, s);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            s[i] = -s[i];
        auto one = [&](auto kind, int group) {
            constexpr int k = decltype(kind)::value;
            const Eight<T> now = x;
            const int at = head;
            const bool is = on;
            float h[8];
            dy.values(is, h);
            if (group + 1 < last)
                fetch(group + 1);
            turn<true>(p, a.interleaved, c, s, h);
            if (normed) {
                float v[8], ss = 0.0f, dot = 0.0f;
                now.values(is, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ss += v[i] * v[i];
                    dot += h[i] * gain[k][i] * v[i];
                }
                const float r = inverse_root(group_sum<L>(ss) * inverse_dim + a.eps);
                const float mean = group_sum<L>(dot) * r * inverse_dim;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float n = v[i] * r;
                    dg[k][i] += is ? h[i] * n : 0.0f;
                    h[i] = r * (h[i] * gain[k][i] - n * mean);
                }
            }
            if (is) {
                T *to = static_cast<T *>(ga.g[k]) + t * ga.ldg[k] + at * a.D;
                store8<kOnce>(to, p.lo, p.hi, h);
            }
        };
        for (int group = first; group < min(last, k0); ++group)
            one(std::integral_constant<int, 0>{}, group);
        for (int group = max(first, k0); group < last; ++group)
            one(std::integral_constant<int, 1>{}, group);
    }
    if (!normed)
        return;
    // the heads of a wave, then the waves, in their order
    __shared__ float sums[kBlock / 64][2][64 / L][8 * L];
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (p.on)
                sums[wave][k][p.sub][(i < 4 ? p.lo : p.hi - 4) + i] = dg[k][i];
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.D; i += kBlock) {
        const int k = i >= a.D ? 1 : 0, at = i - k * a.D;
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kBlock / 64; ++w)
#pragma unroll
            for (int j = 0; j < 64 / L; ++j)
                sum += sums[w][k][j][at];
        ga.workspace[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 * a.D + i] = sum;
    }
}

// The workgroups' rows of sums, 16 columns a workgroup, 64 threads a column.
__global__ __launch_bounds__(1024) void gain_join_kernel(HeadGradArgs ga)
{
    __shared__ double sums[64][17];
    const int col = threadIdx.x & 15, row = threadIdx.x >> 4;
    const int at = blockIdx.x * 16 + col, width = 2 * ga.h.D;
    double sum = 0.0;
#pragma unroll 8
    for (int r = row; r < ga.rows; r += 64)
        sum += (double)ga.workspace[(int64_t)r * width + at];
    sums[row][col] = sum;
    __syncthreads();
    if (row < 8) {
#pragma unroll
        for (int r = 8; r < 64; r += 8)
            sum += sums[row + r][col];
        sums[row][col] = sum;
    }
    __syncthreads();
    if (row == 0) {
#pragma unroll
        for (int r = 1; r < 8; ++r)
            sum += sums[r][col];
        ga.g_gain[at] = (float)sum;
    }
}

// The vectors of a token ([keys, values][head]) over the groups of L lanes: a
// wave takes several tokens where they fit, or blockIdx.y-th part of one token's.
// (Found once a wave: a division for each vector had kept the vector units busy
// 97 % of the time.)
template <int L>
struct KvPlace {
    int l;              // lane of the vector
    int head, kv;
    int64_t token;      // first token
    int64_t step;
    bool on;
    __device__ __forceinline__ KvPlace(const KvArgs &a)
    {
        constexpr int kGroups = 64 / L;
        const int all = 2 * a.cache.heads, group = (threadIdx.x & 63) / L;
        const int per = all <= kGroups ? kGroups / all : 1;
        const int of = all <= kGroups ? group / all : 0;
        const int j = (int)blockIdx.y * kGroups + group - of * all;
        const int64_t wave = (int64_t)blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6);
        l = threadIdx.x % L;
        kv = j >= a.cache.heads ? 1 : 0;
        head = j - kv * a.cache.heads;
        token = wave * per + of;
        step = (int64_t)gridDim.x * (kBlock / 64) * per;
        on = of < per && j < all && 8 * l < a.cache.dim;
    }
};

template <typename T, int L>
__global__ __launch_bounds__(kBlock) void kv_write_kernel(KvArgs a)
{
    const KvPlace<L> p(a);
    const int lo = 4 * p.l, hi = a.cache.dim / 2 + 4 * p.l;
    const T *from = static_cast<const T *>(p.kv ? a.v : a.k) + p.head * a.cache.dim;
    const int64_t ld = p.kv ? a.ldv : a.ldk;
    // (lanes of a vector, and so of a group that is quantized together, have one token)
    for (int64_t t = p.token; t < a.T; t += p.step) {
        const int slot = a.slots[t];
        const bool on = p.on && (uint32_t)slot < (uint32_t)a.cache.pages << a.cache.log_page;
        Eight<T> in;
        if (on)
            in.load(from + t * ld, lo, hi);
        float x[8];
        in.values(on, x);
        put<L>(a.cache, slot, p.head, p.kv, on, p.l, lo, hi, x);
    }
}

template <typename TY, int L, bool kOnce>
__global__ __launch_bounds__(kBlock) void kv_read_kernel(KvArgs a)
{
    const KvPlace<L> p(a);
    if (!p.on)
        return;
    const int lo = 4 * p.l, hi = a.cache.dim / 2 + 4 * p.l;
    TY *to = static_cast<TY *>(p.kv ? a.yv : a.yk) + p.head * a.cache.dim;
    const int64_t ld = (int64_t)a.cache.heads * a.cache.dim;
    for (int64_t t = p.token; t < a.T; t += p.step) {
        const int slot = a.slots[t];
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = 0.0f;
        if ((uint32_t)slot < (uint32_t)a.cache.pages << a.cache.log_page) {
            const SlotAt at = slot_at(a.cache, slot, p.head, p.kv);
            if (a.cache.type == QG_F8) {
                const float scale = f8_scale(*at.scale);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int w = *reinterpret_cast<const int *>(at.codes + (i ? hi : lo));
                    x[4 * i] = __builtin_amdgcn_cvt_f32_fp8(w, 0) * scale;
                    x[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8(w, 1) * scale;
                    x[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8(w, 2) * scale;
                    x[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8(w, 3) * scale;
                }
            } else {
                load8_as(a.cache.type, at.codes, 0, lo, hi, x);
            }
        }
        store8<kOnce>(to + t * ld, lo, hi, x);
    }
}

template <typename P>
hipError_t go(void (*fn)(P), dim3 grid, const P &a, hipStream_t stream)
{
    return launch_kernel(reinterpret_cast<const void *>(fn), grid, dim3(kBlock), 0, stream, a);
}

// fn<T, L> of the element type and of the lanes that a head takes.
template <typename P, typename Pick>
hipError_t by_type(int type, int D, Pick pick, dim3 grid, const P &a, hipStream_t stream)
{
    auto lanes = [&](auto t) {
        return D <= 64    ? pick(t, std::integral_constant<int, 8>{})
               : D <= 128 ? pick(t, std::integral_constant<int, 16>{})
                          : pick(t, std::integral_constant<int, 32>{});
    };
    void (*fn)(P) = type == QG_F32 ? lanes(0.0f) : type == QG_F16 ? lanes(Fp16{}) : lanes(Bf16{});
    return go(fn, grid, a, stream);
}

int lanes_of(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }

// Outputs of at least a quarter of the last-level cache: their readers find
// little of them there, and stores that go past it are faster (16384 tokens of 32
// + 8 heads of 128 in bf16, forward and backward: 155 us for 172), if the lanes'
// pieces make whole lines.  Inputs are loaded so only by the call that writes a
// cache (8192 tokens with 40 query heads: 66 us for 70).
bool large(int64_t vectors, int D, int type) { return vectors * D * type_bytes(type) >= (int64_t)64 << 20; }
bool whole_lines(const HeadArgs &a) { return a.half == 0 || (!a.interleaved && 2 * a.half == a.D); }

constexpr int64_t kForwardWaves = 4096;
constexpr int64_t kBackwardWaves = 4096;

// Lanes that hold one piece of either half (place()): all if nothing is turned,
// those of the turned pairs, none with neighbours; 0 too where they are no power of
// two.
int split_lanes(const HeadArgs &a)
{
    const int n = a.half == 0 ? a.D / 8 : a.interleaved ? 0 : a.half / 4;
    return (n & (n - 1)) ? 0 : n;
}

// Groups of heads; the grid: how many waves share a token (y), as few as give
// every compute unit its waves, since each takes the token's cosines anew, and
// workgroups over the tokens (x), at most `most` in all.
dim3 split_heads(int (&groups)[3], const int (&heads)[3], int64_t T, int D, int64_t waves, int64_t most)
{
    const int per = 64 / lanes_of(D);
    int all = 0;
    for (int i = 0; i < 3; ++i) {
        groups[i] = (heads[i] + per - 1) / per;
        all += groups[i];
    }
    const int64_t parts = std::min<int64_t>(all, ceil_div(waves, T));
    return dim3((unsigned)std::min(ceil_div(T, kBlock / 64), std::max<int64_t>(1, most / parts)), (unsigned)parts);
}

dim3 backward_grid(int (&groups)[3], int q_heads, int k_heads, int64_t T, int D)
{
    const int heads[3] = {q_heads, k_heads, 0};
    return split_heads(groups, heads, T, D, kBackwardWaves, kBackwardWaves / (kBlock / 64));
}

// A wave for each portion of KvPlace.
dim3 kv_grid(const KvArgs &a)
{
    const int groups = 64 / lanes_of(a.cache.dim), all = 2 * a.cache.heads;
    const int64_t waves = all <= groups ? ceil_div(a.T, groups / all) : a.T;
    const unsigned parts = (unsigned)ceil_div(all, groups);
    const int64_t most = std::max<int64_t>(1, kMaxBlocks / parts);
    return dim3((unsigned)std::min(ceil_div(waves, kBlock / 64), most), parts);
}

}  // namespace

hipError_t launch_head_norm_rope(const HeadArgs &args, int x_type, hipStream_t stream)
{
    HeadArgs a = args;
    a.split = split_lanes(a);
    const dim3 grid = split_heads(a.groups, a.heads, a.T, a.D, kForwardWaves, kMaxBlocks);
    if (whole_lines(a) && large(a.T * (a.heads[0] + a.heads[1]), a.D, a.y_type))
        return by_type(
            x_type, a.D,
            [](auto t, auto l) { return &head_kernel<decltype(t), decltype(l)::value, false, false, true>; }, grid, a,
            stream);
    return by_type(
        x_type, a.D, [](auto t, auto l) { return &head_kernel<decltype(t), decltype(l)::value, false, false, false>; },
        grid, a, stream);
}

hipError_t launch_head_norm_rope_write(const HeadArgs &args, int x_type, hipStream_t stream)
{
    HeadArgs a = args;
    a.split = split_lanes(a);
    const dim3 grid = split_heads(a.groups, a.heads, a.T, a.D, kForwardWaves, kMaxBlocks);
    if (a.cache.type == QG_F8)
        return by_type(
            x_type, a.D,
            [](auto t, auto l) { return &head_kernel<decltype(t), decltype(l)::value, true, true, false>; }, grid, a,
            stream);
    return by_type(
        x_type, a.D, [](auto t, auto l) { return &head_kernel<decltype(t), decltype(l)::value, true, false, false>; },
        grid, a, stream);
}

size_t head_backward_workspace(int64_t T, int q_heads, int k_heads, int D)
{
    int groups[3];
    const dim3 grid = backward_grid(groups, q_heads, k_heads, T, D);
    return (size_t)grid.x * grid.y * 2 * D * sizeof(float);
}

template <bool kOnce>
hipError_t backward(const HeadGradArgs &a, int x_type, dim3 grid, hipStream_t stream)
{
    return by_type(
        x_type, a.h.D,
        [&](auto t, auto l) -> void (*)(HeadGradArgs) {
            using T = decltype(t);
            constexpr int L = decltype(l)::value;
            return a.h.y_type == QG_F32   ? &head_backward_kernel<T, float, L, kOnce>
                   : a.h.y_type == QG_F16 ? &head_backward_kernel<T, Fp16, L, kOnce>
                                          : &head_backward_kernel<T, Bf16, L, kOnce>;
        },
        grid, a, stream);
}

hipError_t launch_head_norm_rope_backward(const HeadGradArgs &args, int x_type, hipStream_t stream)
{
    HeadGradArgs a = args;
    const dim3 grid = backward_grid(a.h.groups, a.h.heads[0], a.h.heads[1], a.h.T, a.h.D);
    a.rows = (int)(grid.x * grid.y);
    const bool once = whole_lines(a.h) && large(a.h.T * (a.h.heads[0] + a.h.heads[1]), a.h.D, x_type);
    const hipError_t e = once ? backward<true>(a, x_type, grid, stream) : backward<false>(a, x_type, grid, stream);
    if (e != hipSuccess || !a.h.gain[0])
        return e;
    return launch_kernel(reinterpret_cast<const void *>(&gain_join_kernel), dim3((unsigned)(a.h.D / 8)), dim3(1024), 0,
                         stream, a);
}

hipError_t launch_kv_write(const KvArgs &a, int x_type, hipStream_t stream)
{
    return by_type(
        x_type, a.cache.dim, [](auto t, auto l) { return &kv_write_kernel<decltype(t), decltype(l)::value>; },
        kv_grid(a), a, stream);
}

hipError_t launch_kv_read(const KvArgs &a, int y_type, hipStream_t stream)
{
    if (large(a.T * 2 * a.cache.heads, a.cache.dim, y_type))
        return by_type(
            y_type, a.cache.dim, [](auto t, auto l) { return &kv_read_kernel<decltype(t), decltype(l)::value, true>; },
            kv_grid(a), a, stream);
    return by_type(
        y_type, a.cache.dim, [](auto t, auto l) { return &kv_read_kernel<decltype(t), decltype(l)::value, false>; },
        kv_grid(a), a, stream);
}

}  // namespace qg
