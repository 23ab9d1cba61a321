// Shared by the translation units of the attention step: the cache's layout,
// cross-lane reductions, launcher declarations (qgemv_attn.h states the
// formats).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "qgemv_attn.h"
#include "qgemv_f8_internal.h"

namespace qg {

constexpr int64_t kAttnMaxTokens = 1 << 30;
constexpr int kAttnMaxHeads = 1024;
constexpr int kAttnMaxNew = 16;
constexpr int kAttnMaxBatch = 1 << 16;
constexpr int kMaxAxes = 4;
constexpr int64_t kAttnMaxPlaces = 1 << 30;   // of a sequence: a place, a few steps on, fits 31 bits
constexpr int64_t kAttnMaxTable = (int64_t)1 << 36;   // of all sequences: tiles of them are counted in 31 bits
constexpr int64_t kAttnMaxRows = 1 << 23;     // query heads of all new tokens: workgroups of a launch

inline bool cache_type_ok(int t) { return t == QG_F8 || t == QG_F16 || t == QG_BF16; }
inline bool page_ok(int page) { return page >= 16 && page <= 1024 && (page & (page - 1)) == 0; }
inline bool cache_dim_ok(int d) { return d == 64 || d == 128 || d == 192 || d == 256; }

// A page: codes [head][K, V][token][dim], then for f8 the scale bytes
// [head][K, V][token].
struct KvCache {
    uint8_t *data;
    int64_t page_bytes;
    int64_t scales;     // byte offset of the scale bytes in a page
    int pages, page;
    int log_page;
    int heads, dim, type;
};

inline KvCache kv_cache(void *data, int64_t pages, int page, int heads, int dim, int type)
{
    KvCache c;
    c.data = static_cast<uint8_t *>(data);
    c.scales = (int64_t)2 * heads * page * dim * (type == QG_F8 ? 1 : 2);
    c.page_bytes = ceil_div(c.scales + (type == QG_F8 ? 2 * heads * page : 0), 256) * 256;
    c.pages = (int)pages;
    c.page = page;
    c.log_page = __builtin_ctz((unsigned)page);
    c.heads = heads;
    c.dim = dim;
    c.type = type;
    return c;
}

// 8 bytes at any element's alignment.
struct __attribute__((packed, aligned(2))) Raw8 {
    uint32_t w[2];
};

typedef float f2_t __attribute__((ext_vector_type(2)));

// The two values of lanes 16 (32) apart, in both of them: with both operands
// the same the swap leaves a pair of rows' (halves') first value in one result
// and the second in the other.
__device__ __forceinline__ f2_t pair16(float v)
{
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return f2_t{__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ f2_t pair32(float v)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return f2_t{__uint_as_float(r[0]), __uint_as_float(r[1])};
}

template <int kCtrl>
__device__ __forceinline__ float dpp(float v)
{
    return __uint_as_float(
        (uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), kCtrl, 0xF, 0xF, true));
}

// Over the L consecutive lanes of a group (8, 16 or 32), in all of them:
// neighbours, pairs, halves of eight, halves of a row of 16, rows.
template <int L>
__device__ __forceinline__ float group_sum(float v)
{
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    if constexpr (L >= 16)
        v += dpp<0x140>(v);
    if constexpr (L >= 32) {
        const f2_t p = pair16(v);
        v = p[0] + p[1];
    }
    return v;
}
template <int L>
__device__ __forceinline__ float group_max(float v)
{
    v = fmaxf(v, dpp<0xB1>(v));
    v = fmaxf(v, dpp<0x4E>(v));
    v = fmaxf(v, dpp<0x141>(v));
    if constexpr (L >= 16)
        v = fmaxf(v, dpp<0x140>(v));
    if constexpr (L >= 32) {
        const f2_t p = pair16(v);
        v = fmaxf(p[0], p[1]);
    }
    return v;
}

// What a pass over head vectors does with them.
struct HeadArgs {
    const void *x[3];       // q, k, v
    int64_t ldx[3];
    int heads[3];
    int groups[3];          // groups of heads that a wave takes at once
    const void *gain[2];
    int gain_type;
    float eps;
    const int32_t *positions;
    const float *freq;
    int sections[kMaxAxes]; // where each axis' pairs end
    int axes;
    int half;               // pairs that are turned (rot / 2)
    bool interleaved;
    int split;              // lanes whose two pieces are of different halves (set by the launcher)
    int64_t T;
    int D;
    void *y[2];
    int64_t ldy[2];
    int y_type;
    const int32_t *slots;
    KvCache cache;
};

struct HeadGradArgs {
    HeadArgs h;             // y: the gradients of the outputs, read
    void *g[2];
    int64_t ldg[2];
    float *g_gain;          // [2][D]
    float *workspace;       // [workgroups][2][D]
    int rows;               // of it
};

hipError_t launch_head_norm_rope(const HeadArgs &a, int x_type, hipStream_t stream);
hipError_t launch_head_norm_rope_write(const HeadArgs &a, int x_type, hipStream_t stream);
size_t head_backward_workspace(int64_t T, int q_heads, int k_heads, int D);
hipError_t launch_head_norm_rope_backward(const HeadGradArgs &a, int x_type, hipStream_t stream);

struct KvArgs {
    const void *k, *v;
    int64_t ldk, ldv;
    void *yk, *yv;
    const int32_t *slots;
    int64_t T;
    KvCache cache;
};
hipError_t launch_kv_write(const KvArgs &a, int x_type, hipStream_t stream);
hipError_t launch_kv_read(const KvArgs &a, int y_type, hipStream_t stream);

struct AttendArgs {
    KvCache cache;
    const void *q;
    int64_t ldq;
    int B, M, q_heads, share;   // share: query heads a key head
    const int32_t *table;
    int width;
    const int32_t *lens;
    float scale;
    int window;
    float softcap;
    void *out;
    void *workspace;
};
size_t attend_workspace(int64_t B, int M, int q_heads, int kv_heads, int dim, int cache_type, int page,
                        int64_t width);
hipError_t launch_attend(const AttendArgs &a, int q_type, hipStream_t stream);

}  // namespace qg
