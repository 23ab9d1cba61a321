// Expert routing: top-k softmax, per-expert counts, the slots sorted by
// expert, the balance loss and its gradient (definitions in qgemv_f8.h).
//
// A wave holds a token: lane l has the J = ceil(E / 64) logits of experts
// l J .. l J + J - 1, so that the lowest lane of a tie is the lowest expert.
// The forward pass reads each logit once.  Beyond one workgroup's tokens it
// is three launches, because the sorted order of a slot needs the counts of
// every expert:
//   1. tokens: each workgroup ("chunk") routes its tokens and leaves its
//      counts and its sums of p per expert;
//   2. experts: the counts of the chunks before each chunk, the totals;
//   3. slots: offsets from the totals, every slot to its place, the loss.
// Up to kOneChunk tokens one workgroup does all of it in one launch (a decode
// step is bound by launches, not by bytes).
// All sums run in a fixed order (a lane's tokens, the waves, the chunks), so
// results repeat bit for bit; only whole numbers are counted with atomics.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "qgemv_f8_internal.h"

namespace qg {
namespace {

constexpr int kChunkTokens = 64;   // tokens of a workgroup
constexpr int kWaves = 8;
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

__device__ __forceinline__ uint32_t wave_max(uint32_t v)
{
#pragma unroll
    for (int s = 1; s < 64; s *= 2)
        v = max(v, (uint32_t)__shfl_xor((int)v, s));
    return v;
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int s = 1; s < 64; s *= 2)
        v += __shfl_xor(v, s);
    return v;
}

// Softmax of a token: this lane's p of its J experts.  `any` = the token is
// live; a NaN or +infinity among its logits makes every p NaN (the sum is).
template <int J, typename T>
__device__ __forceinline__ void load_logits(const T *row, int E, int lane, bool routed, float (&x)[J])
{
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int e = lane * J + j;
        x[j] = routed && e < E ? to_f32(row[e]) : -__builtin_inff();
    }
}

template <int J>
__device__ __forceinline__ bool softmax(const float (&x)[J], const uint32_t (&key)[J], float (&p)[J], float &top,
                                        float &sum)
{
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < J; ++j)
        best = max(best, key[j]);
    best = wave_max(best);
    const bool live = best != 0;   // uniform
    top = value_of(best);
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        p[j] = live ? expf(x[j] - top) : 0.0f;
        s += p[j];
    }
    sum = wave_sum(s);
#pragma unroll
    for (int j = 0; j < J; ++j)
        p[j] = live ? p[j] / sum : 0.0f;
    return live;
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
    int32_t hist[kBins + 1];
    float sums[kWaves][kMaxExperts];
    int32_t expert[kChunkTokens * kMaxTopK];
};

// Routes the tokens t0 .. t0 + n - 1 of a workgroup: idx and weight to memory,
// the slots' experts (E: none), the counts and the waves' sums of p to LDS.
template <int J, typename T>
__device__ __forceinline__ void route_tokens(const RouteArgs &a, int64_t t0, int n, Lds &s)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int E = a.E, k = a.k;
    for (int i = threadIdx.x; i < E + 2; i += kThreads)
        s.hist[i] = 0;
    __syncthreads();
    float psum[J];
#pragma unroll
    for (int j = 0; j < J; ++j)
        psum[j] = 0.0f;
    for (int i = wave; i < n; i += kWaves) {
        const int64_t t = t0 + i;
        const bool routed = !a.mask || a.mask[t] != 0;
        float x[J], p[J];
        uint32_t key[J];
        load_logits<J>(static_cast<const T *>(a.logits) + t * a.ldl, E, lane, routed, x);
#pragma unroll
        for (int j = 0; j < J; ++j)
            key[j] = key_of(x[j]);
        float top, sum;
        const bool live = softmax<J>(x, key, p, top, sum);
#pragma unroll
        for (int j = 0; j < J; ++j)
            psum[j] += p[j];
        // the k largest, one after the other: the wave's largest key, the
        // first lane that holds it, that lane's first such expert
        int my_idx = -1;
        float my_w = 0.0f;
        for (int q = 0; q < k; ++q) {
            uint32_t best = 0;
#pragma unroll
            for (int j = 0; j < J; ++j)
                best = max(best, key[j]);
            const uint32_t all = wave_max(best);
            int e = -1;
            if (all != 0) {   // uniform
                const int src = __ffsll((unsigned long long)__ballot(best == all)) - 1;
                int at = 0;
#pragma unroll
                for (int j = J - 1; j >= 0; --j)
                    at = key[j] == all ? j : at;
                if (lane == src) {
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        key[j] = j == at ? 0 : key[j];
                }
                e = __shfl(lane * J + at, src);
            }
            if (lane == q) {
                my_idx = e;
                my_w = e >= 0 ? expf(value_of(all) - top) / sum : 0.0f;
            }
        }
        if (a.renormalize) {
            const float total = wave_sum(lane < k ? my_w : 0.0f);
            my_w = my_idx >= 0 && total != 0.0f ? my_w / total : 0.0f;
        }
        if (lane < k) {
            a.idx[t * k + lane] = my_idx;
            a.weight[t * k + lane] = my_w;
            const int e = my_idx < 0 ? E : my_idx;
            s.expert[i * k + lane] = e;
            atomicAdd(&s.hist[e], 1);
        }
        if (lane == 0 && live)
            atomicAdd(&s.hist[E + 1], 1);
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
        if (lane * J + j < E)
            s.sums[wave][lane * J + j] = psum[j];
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
        int incl = mine;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(incl, d);
            incl += lane >= d ? o : 0;
        }
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

// Places of a chunk's slots: the base of the expert plus the number of
// earlier slots of the chunk with the same expert (every thread counts for
// its own slots; the reads are the same for all lanes).
__device__ __forceinline__ void place_slots(const int32_t *expert, int slots, const int32_t *base, int64_t first,
                                            int32_t *order)
{
    for (int i = threadIdx.x; i < slots; i += kThreads) {
        const int e = expert[i];
        int rank = 0;
        for (int j = 0; j < i; ++j)
            rank += expert[j] == e ? 1 : 0;
        order[base[e] + rank] = (int32_t)(first + i);
    }
}

template <int J, typename T>
__global__ __launch_bounds__(kThreads) void route_one_kernel(Route r)
{
    __shared__ Lds s;
    __shared__ int32_t base[kBins + 1];
    __shared__ double scratch[kWaves];
    const RouteArgs &a = r.a;
    route_tokens<J, T>(a, 0, (int)a.T, s);
    bases(s.hist, a.E, base);
    write_totals(a, s.hist, base, [&](int e) { return waves_sum(s, e); }, scratch);
    place_slots(s.expert, (int)a.T * a.k, base, 0, a.order);
}

template <int J, typename T>
__global__ __launch_bounds__(kThreads) void route_tokens_kernel(Route r)
{
    __shared__ Lds s;
    const RouteArgs &a = r.a;
    const int64_t t0 = (int64_t)blockIdx.x * kChunkTokens;
    route_tokens<J, T>(a, t0, (int)min((int64_t)kChunkTokens, a.T - t0), s);
    for (int e = threadIdx.x; e < a.E + 2; e += kThreads)
        r.chunk_counts[(int64_t)blockIdx.x * (a.E + 2) + e] = s.hist[e];
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
    for (int c0 = 0; c0 < r.chunks; c0 += 64) {
        const int c = c0 + lane;
        int32_t *p = r.chunk_counts + (int64_t)c * (E + 2) + e;
        const int v = c < r.chunks ? *p : 0;
        int incl = v;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(incl, d);
            incl += lane >= d ? o : 0;
        }
        if (c < r.chunks) {
            *p = before + incl - v;
            if (e < E)
                sum += (double)r.chunk_sums[(int64_t)c * E + e];
        }
        before += __shfl(incl, 63);
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
    __shared__ int32_t expert[kChunkTokens * kMaxTopK];
    __shared__ double scratch[kWaves];
    const RouteArgs &a = r.a;
    const int E = a.E;
    const int64_t t0 = (int64_t)blockIdx.x * kChunkTokens;
    const int slots = (int)min((int64_t)kChunkTokens, a.T - t0) * a.k;
    for (int e = threadIdx.x; e < E + 2; e += kThreads)
        counts[e] = r.totals[e];
    for (int i = threadIdx.x; i < slots; i += kThreads) {
        const int e = a.idx[t0 * a.k + i];
        expert[i] = e < 0 ? E : e;
    }
    __syncthreads();
    bases(counts, E, base);
    if (blockIdx.x == 0) {
        write_totals(a, counts, base, [&](int e) { return r.sums[e]; }, scratch);
        __syncthreads();
    }
    for (int e = threadIdx.x; e <= E; e += kThreads)
        base[e] += r.chunk_counts[(int64_t)blockIdx.x * (E + 2) + e];
    __syncthreads();
    place_slots(expert, slots, base, t0 * a.k, a.order);
}

// dlogits of a token: p (dp - sum p dp) with dp[e] = grad_loss E counts[e] /
// (k n^2), and for the chosen experts the gradient through the weights: with
// renormalized weights w_j (g_j - sum_i g_i w_i); without, p_j g_j enters the
// sum and the product with p like dp.
template <int J, typename T>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteGradArgs a)
{
    const int lane = threadIdx.x & 63;
    const int E = a.E, k = a.k;
    const double n = a.counts[E];
    const float unit = a.grad_loss && n > 0 ? (float)((double)*a.grad_loss * E / (n * n * k)) : 0.0f;
    float dp0[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int e = lane * J + j;
        dp0[j] = e < E && a.grad_loss ? unit * (float)a.counts[e] : 0.0f;
    }
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.T; t += (int64_t)gridDim.x * 4) {
        const bool routed = !a.mask || a.mask[t] != 0;
        float x[J], p[J], dp[J], own[J];
        uint32_t key[J];
        load_logits<J>(static_cast<const T *>(a.logits) + t * a.ldl, E, lane, routed, x);
        int my_idx = -1;
        float w = 0.0f, g = 0.0f;
        if (lane < k && a.grad_weight) {
            my_idx = a.idx[t * k + lane];
            w = my_idx >= 0 ? a.weight[t * k + lane] : 0.0f;
            g = my_idx >= 0 ? a.grad_weight[t * k + lane] : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
            key[j] = key_of(x[j]);
            dp[j] = dp0[j];
            own[j] = 0.0f;
        }
        float top, sum;
        const bool live = softmax<J>(x, key, p, top, sum);
        if (a.grad_weight) {
            const float c = a.renormalize ? wave_sum(w * g) : 0.0f;
            const float d = a.renormalize ? w * (g - c) : g;
            for (int q = 0; q < k; ++q) {
                const int e = __shfl(my_idx, q);
                const float v = __shfl(d, q);
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (e == lane * J + j) {
                        if (a.renormalize)
                            own[j] += v;
                        else
                            dp[j] += v;
                    }
            }
        }
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < J; ++j)
            s += p[j] * dp[j];
        s = wave_sum(s);
        T *out = static_cast<T *>(a.dlogits) + t * E;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int e = lane * J + j;
            if (e < E)
                out[e] = from_f32<T>(live && key[j] ? own[j] + p[j] * (dp[j] - s) : 0.0f);
        }
    }
}

template <typename P>
hipError_t go(void (*fn)(P), dim3 grid, dim3 block, const P &a, hipStream_t stream)
{
    return launch_kernel(reinterpret_cast<const void *>(fn), grid, block, 0, stream, a);
}

// fn<J, T> for the experts per lane and the logits' type.
template <typename F>
hipError_t with_types(int E, int type, F f)
{
    const int J = (E + 63) / 64;
    auto by_type = [&](auto j) {
        return type == QG_F32   ? f(j, float{})
               : type == QG_F16 ? f(j, Fp16{})
                                : f(j, Bf16{});
    };
    if (J <= 1)
        return by_type(std::integral_constant<int, 1>{});
    if (J <= 2)
        return by_type(std::integral_constant<int, 2>{});
    if (J <= 4)
        return by_type(std::integral_constant<int, 4>{});
    return by_type(std::integral_constant<int, 8>{});
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
        return with_types(a.E, a.type, [&](auto j, auto t) {
            return go(&route_one_kernel<decltype(j)::value, decltype(t)>, dim3(1), dim3(kThreads), r, stream);
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
    hipError_t e = with_types(a.E, a.type, [&](auto j, auto t) {
        return go(&route_tokens_kernel<decltype(j)::value, decltype(t)>, dim3(r.chunks), dim3(kThreads), r, stream);
    });
    if (e == hipSuccess)
        e = go(&route_experts_kernel, dim3((a.E + 2 + 3) / 4), dim3(256), r, stream);
    if (e == hipSuccess)
        e = go(&route_slots_kernel, dim3(r.chunks), dim3(kThreads), r, stream);
    return e;
}

hipError_t launch_route_backward(const RouteGradArgs &a, int cus, hipStream_t stream)
{
    const unsigned wgs = (unsigned)std::min<int64_t>(ceil_div(a.T, 4), 8LL * cus);
    return with_types(a.E, a.type, [&](auto j, auto t) {
        return go(&route_backward_kernel<decltype(j)::value, decltype(t)>, dim3(wgs), dim3(256), a, stream);
    });
}

}  // namespace qg
