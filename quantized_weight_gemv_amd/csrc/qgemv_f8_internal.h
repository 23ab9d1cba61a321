// Shared by the f8 translation units: packed layouts, element types, the
// quantizer's rule and the operands' conversions (qgemv_f8.h states the
// formats).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "qgemv_f8.h"
#include "qgemv_internal.h"

namespace qg {

constexpr int64_t kF8MaxK = 1 << 20;
constexpr int64_t kF8MaxRows = 1 << 30;       // row numbers, a tile or a few steps on, fit 31 bits
constexpr int64_t kF8MaxGemvK = 16384;        // 128 KiB of codes in LDS
constexpr int64_t kRouteMaxTokens = 1 << 24;
constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 16;

__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Packed weights of an N x K matrix.
struct F8Weights {
    int cb;             // column blocks of 128
    int rt;             // row tiles of 16
    int ls;             // bytes of a row of scales
    int64_t scales;     // byte offset of the scale region
    int64_t bytes;
};

inline F8Weights f8_weights(int64_t N, int64_t K)
{
    F8Weights w;
    w.cb = (int)ceil_div(K, 128);
    w.rt = (int)ceil_div(N, 16);
    w.ls = (w.cb + 3) / 4 * 4;
    w.scales = (int64_t)w.rt * w.cb * 2048;
    w.bytes = ceil_div(w.scales + ceil_div(N, 128) * w.ls, 256) * 256;
    return w;
}

// Packed activations of M x K.
struct F8Acts {
    int cb, ls;
    int64_t scales, bytes;
};

inline F8Acts f8_acts(int64_t M, int64_t K)
{
    F8Acts a;
    a.cb = (int)ceil_div(K, 128);
    a.ls = (a.cb + 3) / 4 * 4;
    a.scales = ceil_div(M * a.cb * 128, 256) * 256;
    a.bytes = ceil_div(a.scales + M * a.ls, 256) * 256;
    return a;
}

inline int type_bytes(int t) { return t == QG_F32 ? 4 : 2; }
inline bool type_ok(int t) { return t == QG_F32 || t == QG_F16 || t == QG_BF16; }

typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
typedef float f4_t __attribute__((ext_vector_type(4)));
typedef float f16v_t __attribute__((ext_vector_type(16)));

// Element types as C++ types, for templates.
struct Bf16 {
    uint16_t u;
};
struct Fp16 {
    uint16_t u;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(Fp16 v) { return (float)__builtin_bit_cast(_Float16, v.u); }
__device__ __forceinline__ float to_f32(Bf16 v) { return __uint_as_float((uint32_t)v.u << 16); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ Fp16 from_f32<Fp16>(float v) { return Fp16{__builtin_bit_cast(uint16_t, (_Float16)v)}; }
template <>
__device__ __forceinline__ Bf16 from_f32<Bf16>(float v) { return Bf16{__builtin_bit_cast(uint16_t, (__bf16)v)}; }

// 16 bytes at any element's alignment (the hardware takes unaligned
// addresses; rows of an odd stride start anywhere).
struct __attribute__((packed, aligned(2))) Raw16 {
    uint32_t w[4];
};

// N consecutive elements as fp32; elements from `left` on are zero.
template <typename T, int N>
__device__ __forceinline__ void load_row(const T *p, int left, float (&v)[N])
{
    if (left >= N) {
        constexpr int kPer = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < N / kPer; ++i) {
            const Raw16 r = *reinterpret_cast<const Raw16 *>(p + i * kPer);
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                if constexpr (sizeof(T) == 4)
                    v[i * kPer + j] = __uint_as_float(r.w[j]);
                else
                    v[i * kPer + j] = to_f32(T{(uint16_t)(r.w[j / 2] >> (16 * (j & 1)))});
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = i < left ? to_f32(p[i]) : 0.0f;
    }
}

// Two values of a 16-bit type in one word (one instruction for bf16).
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<Fp16>(float a, float b)
{
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, h2{(_Float16)a, (_Float16)b});
}
template <>
__device__ __forceinline__ uint32_t pack2<Bf16>(float a, float b)
{
    return __builtin_bit_cast(uint32_t, bf2_t{(__bf16)a, (__bf16)b});
}

// Scale byte of a block whose largest finite magnitude has the fp32 bits
// `amax`: the smallest e >= -127 with amax <= 448 * 2^e, 448 = 1.75 * 2^8, as
// e + 127; 127 for an empty or zero block.  From the bits alone, so it is
// exact: with amax = 1.f * 2^x, e = x - 8, one more where 1.f > 1.75.
// Subnormal amax needs e < -127 at any rate.
__host__ __device__ __forceinline__ uint32_t f8_scale_byte(uint32_t amax)
{
    if (amax == 0)
        return 127;
    const int e = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // biased by 127
    return e < 0 ? 0u : (uint32_t)e;
}

// 2^(byte - 127); byte 0 is the subnormal 2^-127.
__device__ __forceinline__ float f8_scale(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 0x00400000u); }

// 2^(127 - byte).
__device__ __forceinline__ float f8_inverse(uint32_t byte) { return byte >= 254 ? 0x1p-127f : __uint_as_float((254u - byte) << 23); }

// Four values in the codes' range as one word, rounded to nearest even; a NaN
// becomes a NaN code.
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d)
{
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    return (uint32_t)w;
}

// Largest value over the eight lanes of a block (data-parallel-primitive
// moves: neighbours, pairs, halves).
__device__ __forceinline__ float max_of_8(float v)
{
    auto moved = [](float x, auto ctrl) {
        return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x),
                                                                     decltype(ctrl)::value, 0xF, 0xF, true));
    };
    v = fmaxf(v, moved(v, std::integral_constant<int, 0xB1>{}));
    v = fmaxf(v, moved(v, std::integral_constant<int, 0x4E>{}));
    return fmaxf(v, moved(v, std::integral_constant<int, 0x141>{}));
}

// One lane's 16 values of a block held by eight consecutive lanes: their codes
// and the block's scale byte.  The maximum passes over NaNs by itself and a
// NaN stays one through the product and the conversion; an infinity, which
// would become the scale and the largest code, sends the wave over its values
// once more with NaNs in the place of whatever is not finite.  Under the
// largest scale, 2^120, codes stop at 240: 256 would be 2^128.
__device__ __forceinline__ uint32_t f8_quantize16(float (&v)[16], uint32_t (&w)[4])
{
    auto largest = [&] {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i += 2)
            m = fmaxf(fmaxf(m, fabsf(v[i])), fabsf(v[i + 1]));
        return max_of_8(m);
    };
    float amax = largest();
    if (__any(amax == __builtin_inff())) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i] = fabsf(v[i]) < __builtin_inff() ? v[i] : __builtin_nanf("");
        amax = largest();
    }
    const uint32_t byte = f8_scale_byte(__float_as_uint(amax));
    if (__any(byte == 120 + 127)) {
        const float most = byte == 120 + 127 ? 0x1.ep127f : __builtin_inff();
#pragma unroll
        for (int i = 0; i < 16; ++i)   // (a NaN compares false)
            v[i] = fabsf(v[i]) > most ? copysignf(most, v[i]) : v[i];
    }
    const float inv = f8_inverse(byte);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = f8_pack4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
    return byte;
}

// The scale operand of the widening conversions: they read its exponent field
// alone, and take 0 as 2^-127.
__device__ __forceinline__ float f8_exponent(uint32_t byte) { return __uint_as_float(byte << 23); }

// Eight codes (two words) times a power of two (f8_exponent) as a bf16
// operand: exact (four significant bits, bf16's exponent range) down to
// multiples of 2^-133, its subnormal step.
__device__ __forceinline__ bf8_t f8_widen(uint32_t lo, uint32_t hi, float scale)
{
    const bf2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    bf8_t r;
    r[0] = a[0], r[1] = a[1], r[2] = b[0], r[3] = b[1], r[4] = c[0], r[5] = c[1], r[6] = d[0], r[7] = d[1];
    return r;
}

// Wait until at most N vector memory operations of this wave are in flight
// (gfx9 encoding of s_waitcnt: vmcnt in bits 3:0 and 15:14, lgkmcnt in 11:8).
template <int N>
__device__ __forceinline__ void wait_vm()
{
    static_assert(N >= 0 && N < 64, "vmcnt holds 6 bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// Wait for this wave's LDS operations alone.
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4)); }

// At most N vector memory operations, and no LDS operation.
template <int N>
__device__ __forceinline__ void wait_vm_lds()
{
    static_assert(N >= 0 && N < 64, "vmcnt holds 6 bits");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

// A barrier that waits for no memory operation (the fence of __syncthreads
// waits for all of them, copies in flight included); nothing is moved across.
__device__ __forceinline__ void bare_barrier()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// 16 bytes a lane from `at` + `off` of the buffer to consecutive LDS from `to`.
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t from, uint4 *to, uint32_t at, int off)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void *)to, 16, at, off, 0, 0);
}

// Sums of v over the lanes up to this one, the whole wave active, with
// data-parallel-primitive moves: one to eight lanes on inside rows of 16, then
// the rows' and the halves' totals (a step of a shuffle through LDS takes over
// a hundred cycles).
__device__ __forceinline__ int prefix_sum(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // lane 15 of a row into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // lane 31 into rows 2 and 3
    return v;
}

// Where a group's rows are: rows r0 .. r1 - 1 of `order` (or of Y and X, dense),
// at most `tile` of them, of expert e; e = P: slots without an expert.
struct F8Unit {
    int e;
    int64_t r0, r1;
    int first, tiles;   // the expert's first unit and how many it has
    int64_t begin, end; // all of its rows
};

// The unit-th tile of `tile` rows, counting expert by expert, each expert
// beginning a tile of its own; r0 = r1 past the last one.  Every wave finds it
// by itself: a lane counts the tiles of its share of the experts, a prefix sum
// over the lanes and one ballot find the share that holds the unit.  Offsets
// are device data: they are held to 0 .. rows and to their order, so a tile
// never leaves `order`.
template <int kPer>
__device__ __forceinline__ F8Unit f8_unit_of(const int32_t *offsets, int P, int64_t rows, int tile, int64_t unit)
{
    const int lane = threadIdx.x & 63;
    const int per = (P + 1 + 63) / 64;   // experts a lane, the last one: slots without an expert
    const int n = (int)rows;
    int at[kPer + 1];   // all loads first: one latency
#pragma unroll
    for (int j = 0; j <= kPer; ++j) {
        const int e = lane * per + j;
        at[j] = j <= per && e <= P ? offsets[e] : n;
    }
    int mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = lane * per + j;
        at[j] = min(max(at[j], 0), n);
        const int end = e < P ? max(at[j], min(max(at[j + 1], 0), n)) : n;
        mine += j < per && e <= P ? (end - at[j] + tile - 1) / tile : 0;
    }
    const int incl = prefix_sum(mine);
    const unsigned long long holds = __ballot((int64_t)incl > unit);
    if (holds == 0)
        return F8Unit{P, 0, 0, 0, 1, 0, 0};
    const int src = __ffsll(holds) - 1;
    int left = (int)unit - __builtin_amdgcn_readlane(incl - mine, src);
    F8Unit u{P, 0, 0, 0, 1, 0, 0};
    bool found = false;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = src * per + j;
        const int a = __builtin_amdgcn_readlane(at[j], src);
        const int next = min(max(__builtin_amdgcn_readlane(at[j + 1], src), 0), n);
        const int b = e < P ? max(a, next) : n;
        const int tiles = j < per && e <= P ? (b - a + tile - 1) / tile : 0;
        if (!found && left < tiles) {
            u = F8Unit{e, a + (int64_t)left * tile, min((int64_t)b, a + (int64_t)(left + 1) * tile), (int)unit - left,
                       tiles, a, b};
            found = true;
        }
        left -= found ? 0 : tiles;
    }
    return u;
}

__device__ __forceinline__ F8Unit f8_unit(const int32_t *offsets, int P, int64_t rows, int tile, int64_t unit)
{
    if (P < 64)
        return f8_unit_of<1>(offsets, P, rows, tile, unit);
    if (P < 192)
        return f8_unit_of<3>(offsets, P, rows, tile, unit);
    return f8_unit_of<(kMaxExperts + 1 + 63) / 64>(offsets, P, rows, tile, unit);
}

// Another tile of the same expert, the index-th of its tiles.
__device__ __forceinline__ void f8_tile_of(F8Unit &u, int index, int tile)
{
    u.r0 = u.begin + (int64_t)index * tile;
    u.r1 = min(u.end, u.r0 + tile);
}

// An upper bound of the tiles that f8_unit counts.
inline int64_t f8_units(int64_t rows, int P, int tile) { return rows / tile + (rows < P + 1 ? rows : P + 1); }

// Launchers (arguments validated by the callers in qgemv_f8_capi.hip).
hipError_t launch_act_quantize(const void *x, int type, int64_t ldx, int64_t M, int64_t K, uint8_t *xq,
                               hipStream_t stream);
hipError_t launch_act_dequant(const uint8_t *xq, int64_t M, int64_t K, int type, void *out, hipStream_t stream);
hipError_t launch_f8_dequant(const uint8_t *W, int64_t N, int64_t K, bool fp16, void *out, hipStream_t stream);
hipError_t launch_f8_transpose(const uint8_t *W, int64_t N, int64_t K, uint8_t *WT, hipStream_t stream);

// Rows of a product: all M of them, or the slots of one expert after the
// other (order, offsets), with row s of X being slot / k_slots.
struct F8Rows {
    int64_t rows;             // rows of Y
    int64_t x_rows;           // rows of X
    const int32_t *order;     // nullptr: dense
    const int32_t *offsets;   // [P + 1]
    int P;
    int k_slots;
    int64_t stride;           // bytes between pool matrices
};

// x (type QG_*) to be quantized in the launch, or nullptr and xq.
hipError_t launch_f8_skinny(const uint8_t *W, const uint8_t *xq, const void *x, int x_type, void *Y, int y_type,
                            const F8Rows &r, int64_t N, int64_t K, int cus, hipStream_t stream);
hipError_t launch_f8_gemm(const uint8_t *W, const uint8_t *xq, void *Y, int y_type, const F8Rows &r, int64_t N,
                          int64_t K, int cus, hipStream_t stream);

size_t f8_wgrad_workspace(int64_t M, int64_t N, int64_t K);
hipError_t launch_f8_wgrad(const uint16_t *dY, const uint8_t *xq, float *dW, bool accumulate, const F8Rows &r,
                           int64_t N, int64_t K, float *workspace, hipStream_t stream);

struct RouteArgs {
    const void *logits;
    int type;
    int64_t ldl;
    const uint8_t *mask;
    int64_t T;
    int E, k;
    bool renormalize;
    int32_t *idx;
    float *weight;
    int32_t *counts, *offsets, *order;
    float *loss;
    void *workspace;
    bool vec;   // set by the launcher
};
struct RouteGradArgs {
    const void *logits;
    int type;
    int64_t ldl;
    const uint8_t *mask;
    int64_t T;
    int E, k;
    bool renormalize;
    const int32_t *idx;
    const float *weight;
    const int32_t *counts;
    const float *grad_weight, *grad_loss;
    void *dlogits;
    bool vec, vec_out;   // set by the launcher
};
size_t route_workspace(int64_t T, int64_t E);
hipError_t launch_route(const RouteArgs &a, hipStream_t stream);
hipError_t launch_route_backward(const RouteGradArgs &a, int cus, hipStream_t stream);

}  // namespace qg
