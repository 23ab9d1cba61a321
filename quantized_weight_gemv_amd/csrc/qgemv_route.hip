// Expert routing: top-k softmax, per-expert counts, the slots sorted by
// expert, the balance loss and its gradient (definitions in qgemv_f8.h).
//
// L lanes hold a token, a wave 64 / L of them: lane l has the logits of experts
// l J .. l J + J - 1.  Bound by instructions (forward: the k rounds of the
// selection), not by the logits' bytes: in each round a lane's J values cost a
// few instructions each, for all of the wave's tokens at once, the reduction over
// the lanes four to six (16384 x 256, 8 each: 18500 cycles of vector
// instructions a SIMD, forward as backward, about 9 us of 13).  Measured forward + backward (us, bf16; L 16 / 32 /
// 64): 16384 tokens of 256 experts, 8 each: 23 + 15 / 24 + 15 / 28 + 11; of
// 512, 10 each: 46 + 31 / 34 + 25 / 37 + 21; of 64, 6 each: 16 + 5 / 18 + 5 /
// 21 + 6; 4 tokens of 128, 10 each (one workgroup): 7 / 6 / 6 forward; 64
// tokens: 9 / 11 / 15 (all forms of the forward pass are 1 to 2 us faster
// since, by what they share).  So many tokens take L = 16, with 512 experts 32, the
// one workgroup of a decode step 32, the backward pass, which has no rounds
// and many values in registers, 32 and from 256 experts on 64.
// The forward pass reads each logit once.  Beyond one workgroup's tokens it is
// three launches, because the sorted order of a slot needs the counts of every
// expert:
//   1. tokens: each workgroup ("chunk") routes its tokens and leaves its
//      counts and its sums of p per expert;
//   2. experts: the counts of the chunks before each chunk, the totals;
//   3. slots: offsets from the totals, every slot to its place, the loss.
// 16384 x 256: 13, 4 and 5 us (the launches' own latencies in the last two),
// the backward pass 12; 8.4 MB of logits, read twice, and their gradient would
// take 5 us at the copy rate.  Up to kChunkTokens tokens one workgroup does all
// of it in one launch.
// All sums run in a fixed order (a lane's tokens, the wave's, the waves, the
// chunks), so results repeat bit for bit; only whole numbers are counted with
// atomics.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "qgemv_f8_internal.h"

namespace qg {
namespace {

constexpr int kChunkTokens = 64;   // tokens of a workgroup: the bits of a mask
constexpr int kWaves = 16;
constexpr int kThreads = 64 * kWaves;
constexpr int kBins = kMaxExperts + 1;   // the last: slots without an expert

// The order of logits as unsigned keys: larger logit, larger key; 0 for what
// is closed (-infinity, NaN).  -0 and +0 get one key.
__device__ __forceinline__ uint32_t key_of(float v)
{
    if (!(v > -__builtin_inff()))
        return 0;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// Reductions over a token's L lanes with data-parallel-primitive moves, every
// lane gets the result: neighbours, pairs, halves and whole rows of 16; a few
// cycles a step where a shuffle through LDS takes over a hundred.  Rows and
// halves of the wave are exchanged by register swaps.
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

template <int L, typename OP>
__device__ __forceinline__ uint32_t reduce(uint32_t v, OP op)
{
    v = op(v, moved<0xB1>(v));    // lanes 1 0 3 2 of each quad
    v = op(v, moved<0x4E>(v));    // lanes 2 3 0 1
    v = op(v, moved<0x141>(v));   // mirror of each half row
    v = op(v, moved<0x140>(v));   // mirror of each row
    if constexpr (L >= 32) {   // rows 0 0 2 2 and 1 1 3 3
        const auto rows = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = op(rows[0], rows[1]);
    }
    if constexpr (L == 64) {   // lower halves and upper halves
        const auto halves = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = op(halves[0], halves[1]);
    }
    return v;
}

template <int L>
__device__ __forceinline__ uint32_t max_of(uint32_t v)
{
    return reduce<L>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}

template <int L>
__device__ __forceinline__ uint32_t min_of(uint32_t v)
{
    return reduce<L>(v, [](uint32_t a, uint32_t b) { return min(a, b); });
}

template <int L>
__device__ __forceinline__ float sum_of(float v)
{
    return __uint_as_float(reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

// This lane's logits of a token; vec: a lane's J elements are aligned vectors,
// and E is a multiple of J.
template <int J, typename T>
__device__ __forceinline__ void load_logits(const T *row, int E, int lane, bool vec, T (&raw)[J])
{
    if (vec) {
        if (lane * J < E)
            __builtin_memcpy(raw, __builtin_assume_aligned(row + lane * J, sizeof(raw) < 16 ? sizeof(raw) : 16), sizeof(raw));
    } else {
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (lane * J + j < E)
                raw[j] = row[lane * J + j];
    }
}

template <int J, typename T>
__device__ __forceinline__ void open_logits(const T (&raw)[J], int E, int lane, bool routed, float (&x)[J])
{
#pragma unroll
    for (int j = 0; j < J; ++j)
        x[j] = routed && lane * J + j < E ? to_f32(raw[j]) : -__builtin_inff();
}

// e^x for x <= 0, within two units of the last place from 2^-125 up: 2^t for t =
// x log2(e), the rounding of t put right to first order.  Below, the correction
// is lost, and what is smaller than 2^-126 is zero (the instruction flushes it);
// the cut is for the NaN that the correction of -infinity is.
__device__ __forceinline__ float exp_of(float x)
{
    constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
    const float t = x * kLog2e;
    const float low = __builtin_fmaf(x, kRest, __builtin_fmaf(x, kLog2e, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return x < -104.0f ? 0.0f : __builtin_fmaf(e * kLn2, low, e);
}

// Softmax of a token: this lane's p of its J experts; returns whether the
// token is live.  A NaN or +infinity among its logits makes every p NaN (the
// sum is).
template <int L, int J>
__device__ __forceinline__ bool softmax(const float (&x)[J], float (&p)[J], float &top, float &inv)
{
    top = x[0];   // the maximum passes over NaNs by itself
#pragma unroll
    for (int j = 1; j < J; ++j)
        top = fmaxf(top, x[j]);
    top = __uint_as_float(reduce<L>(__float_as_uint(top), [](uint32_t a, uint32_t b) {
        return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
    }));
    const bool live = top > -__builtin_inff();
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        p[j] = live ? exp_of(x[j] - top) : 0.0f;
        s += p[j];
    }
    inv = 1.0f / sum_of<L>(s);
#pragma unroll
    for (int j = 0; j < J; ++j)
        p[j] = live ? p[j] * inv : 0.0f;
    return live;
}

// The k largest logits of a token, one after the other; lane q gets the q-th
// one's expert (-1: none is open any more) and its value.
//   16-bit logits: a word holds the logit's 16-bit key and below it the
//   expert's number, inverted, so the largest word is the choice, ties and all.
//   fp32: the largest key, then the lowest expert that has it.
template <int L, int J, typename T>
__device__ __forceinline__ void choose(const T (&raw)[J], const float (&x)[J], int l, int k, int &my_idx,
                                       float &my_value)
{
    constexpr bool kHalf = sizeof(T) == 2;
    uint32_t key[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        if constexpr (kHalf) {
            const uint32_t b = raw[j].u == 0x8000u ? 0u : raw[j].u;   // -0 as +0
            const uint32_t ordered = (b ^ (b & 0x8000u ? 0xFFFFu : 0x8000u)) << 16;
            const uint32_t word = ordered | (0xFFFFu - (uint32_t)(l * J + j));
            key[j] = x[j] > -__builtin_inff() ? word : 0u;
        } else {
            key[j] = key_of(x[j]);
        }
    }
    my_idx = -1;
    uint32_t my_key = 0;
    for (int q = 0; q < k; ++q) {
        uint32_t best = 0;
#pragma unroll
        for (int j = 0; j < J; ++j)
            best = max(best, key[j]);
        const uint32_t all = max_of<L>(best);
        uint32_t e;
        if constexpr (kHalf) {
            e = 0xFFFFu - (all & 0xFFFFu);
#pragma unroll
            for (int j = 0; j < J; ++j)
                key[j] = key[j] == all ? 0 : key[j];
        } else {
            uint32_t at = ~0u;
#pragma unroll
            for (int j = J - 1; j >= 0; --j)
                at = key[j] == all ? (uint32_t)(l * J + j) : at;
            e = min_of<L>(at);
#pragma unroll
            for (int j = 0; j < J; ++j)
                key[j] = (uint32_t)(l * J + j) == e ? 0 : key[j];
        }
        const bool mine = l == q && all != 0;
        my_idx = mine ? (int)e : my_idx;
        my_key = mine ? all : my_key;
    }
    if constexpr (kHalf) {
        const uint32_t b = my_key >> 16;
        my_value = to_f32(T{(uint16_t)(b & 0x8000u ? b & 0x7FFFu : ~b)});
    } else {
        my_value = value_of(my_key);
    }
}

struct Route {
    RouteArgs a;
    int chunks;
    int32_t *chunk_counts;   // [chunks][E + 2]: slots per expert, without one (E), live tokens (E + 1)
    float *chunk_sums;       // [chunks][E]: sums of p
    int32_t *totals;         // [E + 2]
    double *sums;            // [E]
};

struct Lds {
    unsigned long long tokens[kMaxExperts];   // bit t: token t of the chunk chose the expert
    int32_t dropped[kChunkTokens];            // slots of a token without an expert (always its last ones)
    int32_t live;
    float sums[kWaves][kMaxExperts];
};

__device__ __forceinline__ void clear(Lds &s, int E)
{
    for (int i = threadIdx.x; i < E; i += kThreads)
        s.tokens[i] = 0;
    if (threadIdx.x < kChunkTokens)
        s.dropped[threadIdx.x] = 0;
    if (threadIdx.x == 0)
        s.live = 0;
    __syncthreads();
}

// Marks a slot of token i of the chunk.
__device__ __forceinline__ void mark(Lds &s, int i, int idx)
{
    if (idx >= 0)
        atomicOr(&s.tokens[idx], 1ull << i);
    else
        atomicAdd(&s.dropped[i], 1);
}

// Slots of the chunk per expert, without one (E) and live tokens (E + 1).
__device__ __forceinline__ int count_of(const Lds &s, int e, int E)
{
    if (e < E)
        return __popcll(s.tokens[e]);
    if (e > E)
        return s.live;
    int n = 0;
    for (int t = 0; t < kChunkTokens; ++t)
        n += s.dropped[t];
    return n;
}

// Routes the tokens t0 .. t0 + n - 1 of a workgroup: idx and weight to memory,
// marks and the waves' sums of p to LDS.
template <int L, int J, typename T>
__device__ __forceinline__ void route_tokens(const RouteArgs &a, int64_t t0, int n, Lds &s)
{
    constexpr int kTokens = 64 / L;   // of a wave
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int l = lane % L, own = wave * kTokens + lane / L;
    const int E = a.E, k = a.k;
    const T *const logits = static_cast<const T *>(a.logits);
    float psum[J];
#pragma unroll
    for (int j = 0; j < J; ++j)
        psum[j] = 0.0f;
    for (int i0 = 0; i0 < n; i0 += kWaves * kTokens) {
        const bool any = i0 + wave * kTokens < n;   // uniform over the wave
        const int i = i0 + own;
        const int64_t t = t0 + min(i, n - 1);   // past the end: the last token, unrouted
        T raw[J];
        int routed = 0;
        if (any) {
            load_logits<J>(logits + t * a.ldl, E, l, a.vec, raw);
            routed = a.mask ? a.mask[t] : 1;
        }
        if (i0 == 0)
            clear(s, E);   // behind the first loads
        if (!any)
            break;
        float x[J], p[J];
        open_logits<J>(raw, E, l, routed != 0 && i < n, x);
        float top, inv;
        const bool live = softmax<L, J>(x, p, top, inv);
#pragma unroll
        for (int j = 0; j < J; ++j)
            psum[j] += p[j];
        int my_idx;
        float my_value;
        choose<L, J, T>(raw, x, l, k, my_idx, my_value);
        float my_w = my_idx >= 0 ? exp_of(my_value - top) * inv : 0.0f;
        if (a.renormalize) {
            const float total = sum_of<L>(my_w);
            my_w = my_idx >= 0 && total != 0.0f ? my_w / total : 0.0f;
        }
        if (l < k && i < n) {
            a.idx[t * k + l] = my_idx;
            a.weight[t * k + l] = my_w;
            mark(s, i, my_idx);
        }
        if (l == 0 && live)
            atomicAdd(&s.live, 1);
    }
    // the sums over a wave's tokens
#pragma unroll
    for (int j = 0; j < J; ++j) {
#pragma unroll
        for (int d = L; d < 64; d *= 2)
            psum[j] += __shfl_xor(psum[j], d);
        if (lane < L && lane * J + j < E)
            s.sums[wave][lane * J + j] = psum[j];
    }
    __syncthreads();
}

__device__ __forceinline__ float waves_sum(const Lds &s, int e)
{
    float v = 0.0f;
    for (int w = 0; w < kWaves; ++w)
        v += s.sums[w][e];
    return v;
}

// Exclusive prefix sums of E + 1 counts (counts[E]: slots without an expert)
// into base[0 .. E + 1], by the first wave; all threads wait for it.
__device__ __forceinline__ void bases(const int32_t *counts, int E, int32_t *base)
{
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        const int per = (E + 1 + 63) / 64;
        int mine = 0;
        for (int j = 0; j < per; ++j) {
            const int e = lane * per + j;
            mine += e <= E ? counts[e] : 0;
        }
        const int incl = prefix_sum(mine);
        int at = incl - mine;
        for (int j = 0; j < per; ++j) {
            const int e = lane * per + j;
            if (e <= E) {
                base[e] = at;
                at += counts[e];
            }
        }
        if (lane == 63)
            base[E + 1] = incl;
    }
    __syncthreads();
}

// counts, offsets and the loss, by one workgroup.
template <typename S>
__device__ __forceinline__ void write_totals(const RouteArgs &a, const int32_t *counts, const int32_t *base, S sum_of,
                                             double *scratch)
{
    const int E = a.E;
    const int live = counts[E + 1];
    double part = 0.0;
    for (int e = threadIdx.x; e <= E; e += kThreads) {
        a.offsets[e] = base[e];
        a.counts[e] = e < E ? counts[e] : live;
        if (e < E)
            part += (double)counts[e] * (double)sum_of(e);
    }
#pragma unroll
    for (int s = 1; s < 64; s *= 2)
        part += __shfl_xor(part, s);
    if ((threadIdx.x & 63) == 0)
        scratch[threadIdx.x >> 6] = part;
    __syncthreads();
    if (threadIdx.x == 0) {
        double total = 0.0;
        for (int w = 0; w < kWaves; ++w)
            total += scratch[w];
        const double n = live;
        *a.loss = live ? (float)(E * total / (n * n * a.k)) : 0.0f;
    }
}

// Places of a chunk's slots.  Tokens choose an expert at most once, so a slot
// comes after as many slots of its expert as earlier tokens have its bit set;
// the slots without an expert come after those of the earlier tokens and of
// their own.
__device__ __forceinline__ void place_slots(const RouteArgs &a, const Lds &s, const int32_t *base, int64_t t0, int n)
{
    const int k = a.k;
    for (int i = threadIdx.x; i < n * k; i += kThreads) {
        const int t = i / k;
        const int e = a.idx[t0 * k + i];
        int at;
        if (e >= 0)
            at = base[e] + __popcll(s.tokens[e] & ((1ull << t) - 1));
        else {
            at = base[a.E] + i - t * k - (k - s.dropped[t]);
            for (int u = 0; u < t; ++u)
                at += s.dropped[u];
        }
        a.order[at] = (int32_t)(t0 * k + i);
    }
}

template <int L, int J, typename T>
__global__ __launch_bounds__(kThreads) void route_one_kernel(Route r)
{
    __shared__ Lds s;
    __shared__ int32_t base[kBins + 1];
    __shared__ double scratch[kWaves];
    __shared__ int32_t counts[kBins + 1];
    const RouteArgs &a = r.a;
    route_tokens<L, J, T>(a, 0, (int)a.T, s);
    for (int e = threadIdx.x; e < a.E + 2; e += kThreads)
        counts[e] = count_of(s, e, a.E);
    __syncthreads();   // idx is read back below by other threads of this workgroup
    bases(counts, a.E, base);
    write_totals(a, counts, base, [&](int e) { return waves_sum(s, e); }, scratch);
    place_slots(a, s, base, 0, (int)a.T);
}

template <int L, int J, typename T>
__global__ __launch_bounds__(kThreads) void route_tokens_kernel(Route r)
{
    __shared__ Lds s;
    const RouteArgs &a = r.a;
    const int64_t t0 = (int64_t)blockIdx.x * kChunkTokens;
    route_tokens<L, J, T>(a, t0, (int)min((int64_t)kChunkTokens, a.T - t0), s);
    for (int e = threadIdx.x; e < a.E + 2; e += kThreads)
        r.chunk_counts[(int64_t)blockIdx.x * (a.E + 2) + e] = count_of(s, e, a.E);
    for (int e = threadIdx.x; e < a.E; e += kThreads)
        r.chunk_sums[(int64_t)blockIdx.x * a.E + e] = waves_sum(s, e);
}

// A wave per expert (and for the two counts behind the experts): the chunks'
// counts become the counts before each chunk, 64 chunks a step.
__global__ __launch_bounds__(256) void route_experts_kernel(Route r)
{
    const int lane = threadIdx.x & 63;
    const int E = r.a.E;
    const int e = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (e >= E + 2)
        return;
    int before = 0;
    double sum = 0.0;
    constexpr int kAt = 8;   // loads in flight
    for (int c0 = 0; c0 < r.chunks; c0 += 64 * kAt) {
        int v[kAt];
        float f[kAt];
#pragma unroll
        for (int q = 0; q < kAt; ++q) {
            const int c = c0 + 64 * q + lane;
            v[q] = c < r.chunks ? r.chunk_counts[(int64_t)c * (E + 2) + e] : 0;
            f[q] = c < r.chunks && e < E ? r.chunk_sums[(int64_t)c * E + e] : 0.0f;
        }
#pragma unroll
        for (int q = 0; q < kAt; ++q) {
            const int c = c0 + 64 * q + lane;
            if (c0 + 64 * q >= r.chunks)
                break;
            const int incl = prefix_sum(v[q]);
            if (c < r.chunks)
                r.chunk_counts[(int64_t)c * (E + 2) + e] = before + incl - v[q];
            sum += (double)f[q];
            before += __builtin_amdgcn_readlane(incl, 63);
        }
    }
#pragma unroll
    for (int s = 1; s < 64; s *= 2)
        sum += __shfl_xor(sum, s);
    if (lane == 0) {
        r.totals[e] = before;
        if (e < E)
            r.sums[e] = sum;
    }
}

__global__ __launch_bounds__(kThreads) void route_slots_kernel(Route r)
{
    __shared__ int32_t counts[kBins + 1];
    __shared__ int32_t base[kBins + 1];
    __shared__ Lds s;
    __shared__ double scratch[kWaves];
    const RouteArgs &a = r.a;
    const int E = a.E;
    const int64_t t0 = (int64_t)blockIdx.x * kChunkTokens;
    const int n = (int)min((int64_t)kChunkTokens, a.T - t0);
    for (int e = threadIdx.x; e < E + 2; e += kThreads)
        counts[e] = r.totals[e];
    clear(s, E);
    for (int i = threadIdx.x; i < n * a.k; i += kThreads)
        mark(s, i / a.k, a.idx[t0 * a.k + i]);
    __syncthreads();
    bases(counts, E, base);
    if (blockIdx.x == 0) {
        write_totals(a, counts, base, [&](int e) { return r.sums[e]; }, scratch);
        __syncthreads();
    }
    for (int e = threadIdx.x; e <= E; e += kThreads)
        base[e] += r.chunk_counts[(int64_t)blockIdx.x * (E + 2) + e];
    __syncthreads();
    place_slots(a, s, base, t0, n);
}

// dlogits of a token: p (dp - sum p dp) with dp[e] = grad_loss E counts[e] /
// (k n^2), and for the chosen experts the gradient through the weights: with
// renormalized weights w_j (g_j - sum_i g_i w_i); without, p_j g_j enters the
// sum and the product with p like dp.
template <int L, int J, typename T>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteGradArgs a)
{
    constexpr int kTokens = 64 / L;   // of a wave
    const int l = threadIdx.x % L;
    const int E = a.E, k = a.k;
    const double n = a.counts[E];
    const float unit = a.grad_loss && n > 0 ? (float)((double)*a.grad_loss * E / (n * n * k)) : 0.0f;
    float dp0[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int e = l * J + j;
        dp0[j] = e < E && a.grad_loss ? unit * (float)a.counts[e] : 0.0f;
    }
    __shared__ float given[256 / L][L * J];   // a row a token
    float *const mine = given[threadIdx.x / L];
#pragma unroll
    for (int j = 0; j < J; ++j)
        mine[l * J + j] = 0.0f;
    const T *const logits = static_cast<const T *>(a.logits);
    const int64_t first = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), stride = (int64_t)gridDim.x * 4;   // of waves
    const int own = (threadIdx.x & 63) / L;
    struct Row {
        T raw[J];
        int routed, idx;
        float w, g;
    };
    auto load = [&](int64_t t, Row &r) {
        t = min(t, a.T - 1);
        load_logits<J>(logits + t * a.ldl, E, l, a.vec, r.raw);
        r.routed = a.mask ? a.mask[t] : 1;
        r.idx = -1, r.w = r.g = 0.0f;
        if (l < k && a.grad_weight) {
            const int e = a.idx[t * k + l];
            r.idx = (uint32_t)e < (uint32_t)E ? e : -1;
            r.w = a.weight[t * k + l];
            r.g = a.grad_weight[t * k + l];
        }
    };
    Row row, next;
    load(first * kTokens + own, row);
    for (int64_t at = first; at * kTokens < a.T; at += stride) {
        const int64_t t = at * kTokens + own;
        if ((at + stride) * kTokens < a.T)
            load(t + stride * kTokens, next);   // in flight while these tokens are worked on
        float x[J], p[J], dp[J], own[J];
        open_logits<J>(row.raw, E, l, row.routed != 0, x);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            dp[j] = dp0[j];
            own[j] = 0.0f;
        }
        float top, inv;
        const bool live = softmax<L, J>(x, p, top, inv);
        if (a.grad_weight) {
            const float w = row.idx >= 0 ? row.w : 0.0f, g = row.idx >= 0 ? row.g : 0.0f;
            const float c = a.renormalize ? sum_of<L>(w * g) : 0.0f;
            const float d = a.renormalize ? w * (g - c) : g;
            // from the lanes of the k choices to the lanes of their experts,
            // through the token's row in LDS (zeros but for the choices)
            if (row.idx >= 0)
                mine[row.idx] = d;
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float v = mine[l * J + j];
                own[j] = a.renormalize ? v : 0.0f;
                dp[j] += a.renormalize ? 0.0f : v;
            }
            __builtin_amdgcn_wave_barrier();
            if (row.idx >= 0)
                mine[row.idx] = 0.0f;
            __builtin_amdgcn_wave_barrier();
        }
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j)
            s += p[j] * dp[j];
        s = sum_of<L>(s);
        T *out = static_cast<T *>(a.dlogits) + t * E;
        T res[J];
#pragma unroll
        for (int j = 0; j < J; ++j)
            res[j] = from_f32<T>(live && x[j] > -__builtin_inff() ? own[j] + p[j] * (dp[j] - s) : 0.0f);
        if (t >= a.T) {
            // past the end: nothing to store
        } else if (a.vec_out) {
            if (l * J < E)
                __builtin_memcpy(__builtin_assume_aligned(out + l * J, sizeof(res) < 16 ? sizeof(res) : 16), res, sizeof(res));
        } else {
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (l * J + j < E)
                    out[l * J + j] = res[j];
        }
        row = next;
    }
}

template <typename P>
hipError_t go(void (*fn)(P), dim3 grid, dim3 block, const P &a, hipStream_t stream)
{
    return launch_kernel(reinterpret_cast<const void *>(fn), grid, block, 0, stream, a);
}

// L lanes hold a token, J = 2^n experts each.
template <int L_, int J_>
struct Form {
    static constexpr int L = L_, J = J_;
};

// f for the form and the logits' type; a form each for up to 64, 128, 256 and
// 512 experts.
template <typename F64, typename F128, typename F256, typename F512, typename F>
hipError_t with_types(int E, int type, F f)
{
    static_assert(F64::L * F64::J == 64 && F128::L * F128::J == 128 && F256::L * F256::J == 256 &&
                      F512::L * F512::J == 512,
                  "");
    auto by_type = [&](auto form) {
        return type == QG_F32   ? f(form, float{})
               : type == QG_F16 ? f(form, Fp16{})
                                : f(form, Bf16{});
    };
    return E <= 64 ? by_type(F64{}) : E <= 128 ? by_type(F128{}) : E <= 256 ? by_type(F256{}) : by_type(F512{});
}

// Whether a lane's J elements of every row are one aligned vector.
inline bool whole_vectors(const void *p, int64_t ld, int E, int J, int type)
{
    const uintptr_t bytes = (uintptr_t)J * type_bytes(type);
    return E % J == 0 && ld % J == 0 && (reinterpret_cast<uintptr_t>(p) & (std::min<uintptr_t>(bytes, 16) - 1)) == 0;
}

inline int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

}  // namespace

size_t route_workspace(int64_t T, int64_t E)
{
    if (T <= kChunkTokens)
        return 0;
    const int64_t chunks = ceil_div(T, kChunkTokens);
    return (size_t)(round16(8 * E) + round16(4 * (E + 2)) + round16(chunks * (E + 2) * 4) + round16(chunks * E * 4));
}

hipError_t launch_route(const RouteArgs &a, hipStream_t stream)
{
    Route r{};
    r.a = a;
    if (a.T <= kChunkTokens) {
        return with_types<Form<32, 2>, Form<32, 4>, Form<32, 8>, Form<32, 16>>(a.E, a.type, [&](auto form, auto t) {
            using O = decltype(form);
            r.a.vec = whole_vectors(a.logits, a.ldl, a.E, O::J, a.type);
            return go(&route_one_kernel<O::L, O::J, decltype(t)>, dim3(1), dim3(kThreads), r, stream);
        });
    }
    const int64_t E = a.E;
    r.chunks = (int)ceil_div(a.T, kChunkTokens);
    uint8_t *w = static_cast<uint8_t *>(a.workspace);
    r.sums = reinterpret_cast<double *>(w);
    w += round16(8 * E);
    r.totals = reinterpret_cast<int32_t *>(w);
    w += round16(4 * (E + 2));
    r.chunk_counts = reinterpret_cast<int32_t *>(w);
    w += round16((int64_t)r.chunks * (E + 2) * 4);
    r.chunk_sums = reinterpret_cast<float *>(w);
    hipError_t e = with_types<Form<16, 4>, Form<16, 8>, Form<16, 16>, Form<32, 16>>(a.E, a.type, [&](auto form, auto t) {
        using O = decltype(form);
        r.a.vec = whole_vectors(a.logits, a.ldl, a.E, O::J, a.type);
        return go(&route_tokens_kernel<O::L, O::J, decltype(t)>, dim3(r.chunks), dim3(kThreads), r, stream);
    });
    if (e == hipSuccess)
        e = go(&route_experts_kernel, dim3((a.E + 2 + 3) / 4), dim3(256), r, stream);
    if (e == hipSuccess)
        e = go(&route_slots_kernel, dim3(r.chunks), dim3(kThreads), r, stream);
    return e;
}

hipError_t launch_route_backward(const RouteGradArgs &args, int cus, hipStream_t stream)
{
    RouteGradArgs a = args;
    return with_types<Form<32, 2>, Form<32, 4>, Form<64, 4>, Form<64, 8>>(a.E, a.type, [&](auto form, auto t) {
        using O = decltype(form);
        a.vec = whole_vectors(a.logits, a.ldl, a.E, O::J, a.type);
        a.vec_out = whole_vectors(a.dlogits, a.E, a.E, O::J, a.type);
        const unsigned wgs = (unsigned)std::min<int64_t>(ceil_div(a.T, 256 / O::L), 8LL * cus);
        return go(&route_backward_kernel<O::L, O::J, decltype(t)>, dim3(wgs), dim3(256), a, stream);
    });
}

}  // namespace qg
