// ns_route.hip -- gfx950 kernels of the experts' router (include/ns.h, ns_route_*):
// softmax, the top experts of each token, their weights, the experts' counts, the
// balance loss, and the logits' gradient.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "ns.h"
#include "ns_device.h"
#include "ns_route.h"

namespace ns {
namespace {

constexpr int kThreads = kRouteThreads, kJoinThreads = 256;

// An expert's key: a double whose high word is its logit, low word its index, so that
// keys order as the choice does and no two are alike. (Doubles compare by sign, then
// magnitude: among equal positive logits the index counts down, among negative ones up.
// No logit's bits make a NaN of a double but an fp32 NaN's, which becomes the quiet one,
// above Inf.) -0 is 0; the key of -Inf, of an expert that is not to be had, is kNone.
constexpr uint32_t kNone = 0xFF800000u;
__device__ __forceinline__ double key_of(float x, int expert)
{
    const uint32_t b = x != x ? 0x7FC00000u : __float_as_uint(x + 0.f);
    return __hiloint2double((int)b, b == kNone ? 0 : (int)(b >> 31) ? expert : ~expert);
}
__device__ __forceinline__ double no_key() { return __hiloint2double((int)kNone, 0); }
__device__ __forceinline__ bool is_none(double k) { return (uint32_t)__double2hiint(k) == kNone; }
__device__ __forceinline__ float logit_of(double k) { return __int_as_float(__double2hiint(k)); }
__device__ __forceinline__ int expert_of(double k)
{
    const int lo = __double2loint(k);
    return __double2hiint(k) < 0 ? lo : ~lo;
}

// op over a group of G lanes, in all of them: within 16 lanes by row rotations, beyond
// by exchange. (Every lane adds in an order of its own, but 16 lanes' sums by rotations
// of 8, 4, 2 and 1 pair the same values: all lanes get the same bits.)
template <int G, typename Op>
__device__ __forceinline__ int32_t reduce(int32_t v, Op&& op)
{
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x128, 0xF, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x124, 0xF, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x122, 0xF, 0xF, false));
    v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x121, 0xF, 0xF, false));
    if constexpr (G == 64) {
        v = op(v, __shfl_xor(v, 16, 64));
        v = op(v, __shfl_xor(v, 32, 64));
    }
    return v;
}
template <int CTRL>
__device__ __forceinline__ double rotated(double v)
{
    return __hiloint2double(__builtin_amdgcn_update_dpp(0, __double2hiint(v), CTRL, 0xF, 0xF, false),
                            __builtin_amdgcn_update_dpp(0, __double2loint(v), CTRL, 0xF, 0xF, false));
}
template <int G>
__device__ __forceinline__ double max_of(double v)
{
    v = fmax(v, rotated<0x128>(v));
    v = fmax(v, rotated<0x124>(v));
    v = fmax(v, rotated<0x122>(v));
    v = fmax(v, rotated<0x121>(v));
    if constexpr (G == 64) {
        v = fmax(v, __shfl_xor(v, 16, 64));
        v = fmax(v, __shfl_xor(v, 32, 64));
    }
    return v;
}
template <int G>
__device__ __forceinline__ float fmax_of(float v)
{
    return __int_as_float(reduce<G>(__float_as_int(v), [](int32_t a, int32_t b) {
        return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b)));
    }));
}
template <int G>
__device__ __forceinline__ float sum_of(float v)
{
    return __int_as_float(reduce<G>(__float_as_int(v), [](int32_t a, int32_t b) {
        return __float_as_int(__int_as_float(a) + __int_as_float(b));
    }));
}
template <int G>
__device__ __forceinline__ int32_t count_of(int32_t v)
{
    return reduce<G>(v, [](int32_t a, int32_t b) { return a + b; });
}

// exp(x - m) of the row's largest m: off by two roundings of the distance, which are as
// much of the result, and one of its own. (The difference comes first: the products of
// large logits pass fp32's range, and round by more than the distance is.)
__device__ __forceinline__ float exp_of(float x, float m)
{
    return __builtin_amdgcn_exp2f((x - m) * 1.44269504f);
}

// N logits of a row from expert e on, -Inf past the end.
template <int N, typename T>
__device__ __forceinline__ void load_logits(const T* row, int e, int experts, float* x)
{
    constexpr int kVec = 16 / sizeof(T);   // values a load
    if constexpr (N % kVec == 0) {
        if (e + N <= experts) {
#pragma unroll
            for (int i = 0; i < N / kVec; ++i) {
                const u32x4 w = load16_any(row + e + i * kVec);
#pragma unroll
                for (int j = 0; j < kVec; ++j)
                    x[i * kVec + j] = sizeof(T) == 4 ? __uint_as_float(w[j % 4])
                                                     : __uint_as_float(j & 1 ? w[j / 2 % 4] & 0xFFFF0000u : w[j / 2 % 4] << 16);
            }
            return;
        }
    }
#pragma unroll
    for (int v = 0; v < N; ++v)
        x[v] = e + v < experts ? to_f32(gbl(row)[e + v]) : -__builtin_inff();
}

// What the workgroups' sums come to: of c P, of c (below 2^29: at most 16 of 2^24 tokens) and
// of n.
struct Totals {
    float cp;
    int32_t c, n;
};
__device__ __forceinline__ Totals add(const Totals& a, const Totals& b)
{
    return {a.cp + b.cp, a.c + b.c, a.n + b.n};
}
// The sum over N threads, in thread 0; red: LDS for one a wavefront.
template <int N>
__device__ __forceinline__ Totals block_sum(Totals v, Totals* red)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1)
        v = add(v, {__shfl_xor(v.cp, off, 64), __shfl_xor(v.c, off, 64), __shfl_xor(v.n, off, 64)});
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < N / 64; ++w)
        v = add(v, red[w]);
    return v;
}
__device__ __forceinline__ void add_expert(Totals& v, float p, int32_t c)
{
    v.cp = fmaf((float)c, p, v.cp);
    v.c += c;
}
__device__ __forceinline__ void put_loss(const RouteArgs& a, const Totals& v)
{
    a.routed[0] = v.n;
    a.loss[0] = v.n > 0 ? a.experts * (v.cp / (float)v.c) / (float)v.n : 0.f;
}

// A value of the 16 neighbouring lanes, R lanes before this one (cyclic).
template <int R>
__device__ __forceinline__ float before(float v)
{
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + R, 0xF, 0xF, false));
}
template <typename F, int... R>
__device__ __forceinline__ void rotations_of(F&& f, std::integer_sequence<int, R...>)
{
    (f(std::integral_constant<int, R + 1>{}), ...);
}
// f(1) .. f(15) with the numbers as constants
template <typename F>
__device__ __forceinline__ void rotations(F&& f)
{
    rotations_of(f, std::make_integer_sequence<int, 15>{});
}

// One of a token's candidates.
struct Candidate { float x; int32_t expert; };

// The top experts of the four tokens of a wavefront, 16 lanes each, at once. The k-th
// largest of the lanes' own largest logits bounds the k-th largest of all from below, so
// the few that reach it (10 or 11 of 256 for k = 8, as a rule) are all that need ordering:
// they move to LDS, one to a lane in the experts' order, and each counts those before it.
// Returns false, for all lanes, where some token has more than 16 of them, or logits that
// do not compare (a NaN): true with the expert of a lane's own, if it has one, and its rank
// (lanes without one rank behind the others, so that all ranks are different).
template <int V>
__device__ __forceinline__ bool rank_few(const float (&x)[V], float own, int top_k, bool sound, Candidate* list,
                                         Candidate& mine, int& rank)
{
    const int l = threadIdx.x & 15;
    int least = 1;   // lanes whose largest is at least this one's
    rotations([&](auto r) __attribute__((always_inline)) { least += before<decltype(r)::value>(own) >= own; });
    const float bound = fmax_of<16>(least >= top_k ? own : -__builtin_inff());
    int n = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
        n += x[v] >= bound;
    int upto = n;   // candidates of the lanes up to this one
    upto += __builtin_amdgcn_update_dpp(0, upto, 0x111, 0xF, 0xF, true);   // row_shr:1
    upto += __builtin_amdgcn_update_dpp(0, upto, 0x112, 0xF, 0xF, true);
    upto += __builtin_amdgcn_update_dpp(0, upto, 0x114, 0xF, 0xF, true);
    upto += __builtin_amdgcn_update_dpp(0, upto, 0x118, 0xF, 0xF, true);
    if (__ballot(!sound || upto > 16 || bound == -__builtin_inff()))
        return false;
    const int total = count_of<16>(n);
    int at = upto - n;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (x[v] >= bound)
            list[at++] = {x[v], l * V + v};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const Candidate read = list[l];
    mine = l < total ? read : Candidate{-__builtin_inff(), -1};
    rank = 0;
    rotations([&](auto r) __attribute__((always_inline)) {
        const float y = before<decltype(r)::value>(mine.x);
        rank += y > mine.x || (y == mine.x && l >= decltype(r)::value);
    });
    return true;
}

// G lanes take a token, lane i the experts V i .. V i + V - 1; a workgroup 512 / G tokens at
// a time, kRouteGroups workgroups in all. Half bound by vector operations, which keep the
// SIMDs busy 60% of the time (32768 tokens of 256 fp32 logits, top 8: 16 us); for the rest all
// wavefronts wait for their round's logits, which they load at its start. Ordering the few
// candidates of a token (rank_few) saves about 3 us there over taking the top experts one
// after the other from all of them. That way remains for the tokens that the other refuses,
// for few experts a lane, where it is no longer, and for more than 256 experts (512: 58 us,
// 1024: 86). Sums of p stay in the lanes' registers over a workgroup's tokens, counts in LDS.
template <int DT, int G, int V>
__global__ __launch_bounds__(kThreads, 4) void k_route(const RouteArgs a)
{
    using T = typename Elt<DT>::type;
    constexpr int kPer = kThreads / G;   // tokens at a time
    constexpr bool kFew = G == 16 && V >= 4;
    __shared__ float sums[kPer][G * V];
    __shared__ int32_t hist[G * V];
    __shared__ Totals red[kThreads / 64];
    __shared__ Candidate list[kFew ? kPer : 1][16];
    const int t = threadIdx.x, l = t % G, grp = t / G;
    for (int e = t; e < G * V; e += kThreads)
        hist[e] = 0;
    __syncthreads();
    float acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        acc[v] = 0.f;
    int n = 0;
    for (int t0 = blockIdx.x * kPer; t0 < a.tokens; t0 += gridDim.x * kPer) {
        const int token = t0 + grp;
        const bool in = token < a.tokens;
        float x[V], e[V];
        load_logits<V>(reinterpret_cast<const T*>(a.logits) + (in ? token : 0) * a.ld, l * V, a.experts, x);
        // p: with a NaN or +Inf among the logits, or with none, the sum is NaN
        float own = -__builtin_inff();
#pragma unroll
        for (int v = 0; v < V; ++v)
            own = fmaxf(own, x[v]);
        const float mx = fmax_of<G>(own);
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            e[v] = exp_of(x[v], mx);
            sum += e[v];
        }
        sum = sum_of<G>(sum);
        const float inv = 1.f / sum;
        bool live = in && (!a.mask || gbl(a.mask)[token]);
        Candidate mine = {0.f, -1};   // a chosen expert, of lane i or of any lane
        int rank = l;                 // which one, top_k or more for none
        bool done = false;
        if constexpr (kFew)
            done = rank_few<V>(x, own, a.top_k, sum == sum, list[grp], mine, rank);
        if (!done) {
            // (with a NaN, top is one, and the largest of all)
            double key[V], best = no_key();
#pragma unroll
            for (int v = 0; v < V; ++v) {
                key[v] = key_of(x[v], l * V + v);
                best = fmax(best, key[v]);
            }
            double top = max_of<G>(best), mykey = no_key();
            live = live && !is_none(top);
            for (int i = 0; i < a.top_k; ++i) {
                if (l == i)
                    mykey = top;
                best = no_key();
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    key[v] = key[v] == top ? no_key() : key[v];
                    best = fmax(best, key[v]);
                }
                top = max_of<G>(best);
            }
            mine = {logit_of(mykey), is_none(mykey) ? -1 : expert_of(mykey)};
            rank = l;
        }
        if (live)
#pragma unroll
            for (int v = 0; v < V; ++v)
                acc[v] = fmaf(e[v], inv, acc[v]);
        n += live;
        const bool chosen = live && rank < a.top_k && mine.expert >= 0;
        if (chosen)
            atomicAdd(&hist[mine.expert], 1);
        float w = chosen ? exp_of(mine.x, mx) * inv : 0.f;
        if (a.normalize) {
            // (added in the order of the ranks, which is the lanes' own where experts are taken
            // one after the other: a token's weights do not depend on which way its neighbours
            // send it)
            const float all = sum_of<G>(
                !kFew ? w : __int_as_float(__builtin_amdgcn_ds_permute(((int)(threadIdx.x & 48) + rank) * 4, __float_as_int(w))));
            w = chosen ? w / all : 0.f;
        }
        if (in && rank < a.top_k) {
            gbl(a.chosen)[(int64_t)token * a.top_k + rank] = chosen ? mine.expert : -1;
            gbl(a.weights)[(int64_t)token * a.top_k + rank] = w;
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        sums[grp][l * V + v] = acc[v];
    __syncthreads();
    const bool alone = gridDim.x == 1;
    Totals all = {0.f, 0, l == 0 ? n : 0};   // (all lanes of a group count its tokens)
    for (int k = t; k < a.experts; k += kThreads) {
        float p = 0.f;
#pragma unroll
        for (int g = 0; g < kPer; ++g)
            p += sums[g][k];
        const int32_t c = hist[k];
        if (alone) {
            gbl(a.probs)[k] = p;
            gbl(a.counts)[k] = c;
            add_expert(all, p, c);
        } else {
            // (16 experts of all workgroups side by side, as the join reads them)
            const int64_t at = ((int64_t)(k / kRouteJoin) * gridDim.x + blockIdx.x) * kRouteJoin + k % kRouteJoin;
            gbl(a.part_probs)[at] = p;
            gbl(a.part_counts)[at] = c;
        }
    }
    all = block_sum<kThreads>(all, red);
    if (t > 0)
        return;
    if (alone) {
        put_loss(a, all);
        return;
    }
    gbl(a.part_routed)[blockIdx.x] = all.n;
    if (blockIdx.x == 0)
        *gbl(a.arrived) = 0;
}

// Adds up the workgroups' sums, 16 experts a workgroup: thread t four of them (t % 4) of
// every 64th workgroup from t / 4 on, all loads in flight at once. The last one to arrive
// has all experts' and writes the loss. (The counter is cleared by the launch before.)
// Latency bounds it: 6 us for 512 workgroups' sums of 256 experts.
__global__ __launch_bounds__(kJoinThreads) void k_route_join(const RouteArgs a, int parts)
{
    __shared__ float sp[kJoinThreads / 64][kRouteJoin];
    __shared__ int32_t sc[kJoinThreads / 64][kRouteJoin];
    __shared__ Totals red[kJoinThreads / 64];
    __shared__ uint32_t order;
    constexpr int kEach = (int)kRouteGroups * kRouteJoin / 4 / kJoinThreads;
    const int t = threadIdx.x, wave = t >> 6;
    const int64_t base = (int64_t)blockIdx.x * parts * kRouteJoin;
    f32x4 p[kEach];
    i32x4 c[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int b = t / 4 + kJoinThreads / 4 * i;
        const bool in = b < parts;
        const int64_t at = base + (int64_t)(in ? b : 0) * kRouteJoin + 4 * (t % 4);
        p[i] = *(const NS_GLOBAL f32x4*)(gbl(a.part_probs) + at);
        c[i] = *(const NS_GLOBAL i32x4*)(gbl(a.part_counts) + at);
        if (!in) {
            p[i] = f32x4{0.f, 0.f, 0.f, 0.f};
            c[i] = i32x4{0, 0, 0, 0};
        }
    }
#pragma unroll
    for (int i = 1; i < kEach; ++i) {
        p[0] += p[i];
        c[0] += c[i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float pj = p[0][j];
        int32_t cj = c[0][j];
#pragma unroll
        for (int off = 4; off < 64; off <<= 1) {
            pj += __shfl_xor(pj, off, 64);
            cj += __shfl_xor(cj, off, 64);
        }
        if ((t & 63) < 4) {
            sp[wave][4 * (t & 3) + j] = pj;
            sc[wave][4 * (t & 3) + j] = cj;
        }
    }
    __syncthreads();
    const int e = blockIdx.x * kRouteJoin + t;
    if (t < kRouteJoin && e < a.experts) {
        float ps = 0.f;
        int32_t cs = 0;
#pragma unroll
        for (int w = 0; w < kJoinThreads / 64; ++w) {
            ps += sp[w][t];
            cs += sc[w][t];
        }
        __hip_atomic_store(a.probs + e, ps, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(a.counts + e, cs, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __threadfence();
    __syncthreads();
    if (t == 0)
        order = __hip_atomic_fetch_add(a.arrived, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (order != gridDim.x - 1)
        return;
    __threadfence();
    Totals all = {0.f, 0, 0};
    for (int b = t; b < parts; b += kJoinThreads)
        all.n += gbl(a.part_routed)[b];
    for (int k = t; k < a.experts; k += kJoinThreads)
        add_expert(all, __hip_atomic_load(a.probs + k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT),
                   __hip_atomic_load(a.counts + k, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
    all = block_sum<kJoinThreads>(all, red);
    if (t == 0)
        put_loss(a, all);
}

// G lanes take a token, in pieces of 16 bytes a lane one after the other, so that each
// load and store of them covers whole lines (16 experts a lane side by side store
// quarters of lines: 29 us for 32768 tokens of 256 fp32 logits instead of 16, 4.3 TB/s).
template <int DT, int G, int V>
__global__ __launch_bounds__(kThreads) void k_route_grad(const RouteGradArgs a)
{
    using T = typename Elt<DT>::type;
    constexpr int kPer = kThreads / G, kVec = 16 / (int)sizeof(T), P = V < kVec ? V : kVec;
    // h of a token's chosen experts, 0 but while its lanes are at it: one row a group of
    // lanes, who are of one wavefront
    __shared__ __attribute__((aligned(16))) float chosen[kPer][G * V];
    const int t = threadIdx.x, l = t % G, grp = t / G, first = (t & 63) / G * G;
    auto expert = [&](int v) { return v / P * (G * P) + l * P + v % P; };
#pragma unroll
    for (int v = 0; v < V; ++v)
        chosen[grp][expert(v)] = 0.f;
    // the loss's part of g, the same for all tokens
    float base[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        base[v] = 0.f;
    if (a.dloss) {
        int32_t c[V], own = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            c[v] = expert(v) < a.experts ? gbl(a.counts)[expert(v)] : 0;
            own += c[v];
        }
        const int32_t all = count_of<G>(own), n = gbl(a.routed)[0];
        const float f = all > 0 && n > 0 ? gbl(a.dloss)[0] * (float)a.experts / (float)n : 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
            base[v] = all > 0 ? f * ((float)c[v] / (float)all) : 0.f;
    }
    for (int t0 = blockIdx.x * kPer; t0 < a.tokens; t0 += gridDim.x * kPer) {
        const int token = t0 + grp;
        const bool in = token < a.tokens;
        const T* row = reinterpret_cast<const T*>(a.logits) + (in ? token : 0) * a.ld;
        float x[V];
#pragma unroll
        for (int v = 0; v < V; v += P)
            load_logits<P>(row, expert(v), a.experts, x + v);
        int32_t mine = -1;
        float h = 0.f;
        bool live = false;   // (of a token's first lane: its own, which all take)
        if (in && l < a.top_k) {
            mine = gbl(a.chosen)[(int64_t)token * a.top_k + l];
            live = mine != -1;
            if (mine >= a.experts)
                mine = -1;
            if (a.dweights && mine >= 0)
                h = gbl(a.dweights)[(int64_t)token * a.top_k + l];
        }
        const float picked = mine >= 0 ? to_f32(gbl(row)[mine]) : -__builtin_inff();
        live = __shfl((int)live, first, 64) != 0;
        // (a NaN is not the largest here, but makes a NaN of the sum)
        float mx = -__builtin_inff();
#pragma unroll
        for (int v = 0; v < V; ++v)
            mx = fmaxf(mx, x[v]);
        mx = fmax_of<G>(mx);
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] = exp_of(x[v], mx);
            sum += x[v];
        }
        const float inv = 1.f / sum_of<G>(sum);
        if (a.normalize && a.dweights) {
            const float p = mine >= 0 ? exp_of(picked, mx) * inv : 0.f;
            const float s = sum_of<G>(p);
            const float dot = sum_of<G>(h * (p / s));
            h = mine >= 0 ? (h - dot) / s : 0.f;
        }
        float g[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            g[v] = base[v];
        if (a.dweights) {
            // (an index twice: its lanes add in their order, within one instruction)
            __builtin_amdgcn_wave_barrier();
            if (mine >= 0)
                atomicAdd(&chosen[grp][mine], h);
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int v = 0; v < V; ++v)
                g[v] += chosen[grp][expert(v)];
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            if (mine >= 0)
                chosen[grp][mine] = 0.f;
        }
        float dot = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            x[v] *= inv;
            dot = fmaf(g[v], x[v], dot);
        }
        dot = sum_of<G>(dot);
        if (!in)
            continue;
        float d[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            d[v] = live ? x[v] * (g[v] - dot) : 0.f;
        T* out = reinterpret_cast<T*>(a.out) + token * a.ldo;
#pragma unroll
        for (int v = 0; v < V; v += P) {
            if constexpr (P == kVec) {
                if (expert(v) + P <= a.experts) {
                    u32x4 w;
                    if constexpr (sizeof(T) == 4) {
                        w = __builtin_bit_cast(u32x4, f32x4{d[v], d[v + 1], d[v + 2], d[v + 3]});
                    } else {
                        bf16x8 b;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            b[j] = (bf16)d[v + j % P];
                        w = __builtin_bit_cast(u32x4, b);
                    }
                    store16_any(out + expert(v), w);
                    continue;
                }
            }
#pragma unroll
            for (int j = 0; j < P; ++j)
                if (expert(v) + j < a.experts)
                    gbl(out)[expert(v) + j] = from_f32<T>(d[v + j]);
        }
    }
}

// go(lanes a token, values a lane) for a number of experts
template <typename F>
void by_experts(int experts, F&& go)
{
    const std::integral_constant<int, 16> g16{};
    const std::integral_constant<int, 64> g64{};
    if (experts <= 16)
        go(g16, std::integral_constant<int, 1>{});
    else if (experts <= 32)
        go(g16, std::integral_constant<int, 2>{});
    else if (experts <= 64)
        go(g16, std::integral_constant<int, 4>{});
    else if (experts <= 128)
        go(g16, std::integral_constant<int, 8>{});
    else if (experts <= 256)
        go(g16, std::integral_constant<int, 16>{});
    else if (experts <= 512)
        go(g64, std::integral_constant<int, 8>{});
    else
        go(g64, std::integral_constant<int, 16>{});
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, int nwg, int dtype, hipStream_t stream)
{
    by_experts(a.experts, [&](auto g, auto v) {
        if (dtype == 0)
            hipLaunchKernelGGL((k_route<0, decltype(g)::value, decltype(v)::value>), dim3(nwg), dim3(kThreads), 0,
                               stream, a);
        else
            hipLaunchKernelGGL((k_route<1, decltype(g)::value, decltype(v)::value>), dim3(nwg), dim3(kThreads), 0,
                               stream, a);
    });
    return hipGetLastError();
}

hipError_t launch_route_join(const RouteArgs& a, int nwg, hipStream_t stream)
{
    hipLaunchKernelGGL(k_route_join, dim3((a.experts + kRouteJoin - 1) / kRouteJoin), dim3(kJoinThreads), 0,
                       stream, a, nwg);
    return hipGetLastError();
}

hipError_t launch_route_grad(const RouteGradArgs& a, int nwg, int dtype, hipStream_t stream)
{
    by_experts(a.experts, [&](auto g, auto v) {
        if (dtype == 0)
            hipLaunchKernelGGL((k_route_grad<0, decltype(g)::value, decltype(v)::value>), dim3(nwg), dim3(kThreads), 0,
                               stream, a);
        else
            hipLaunchKernelGGL((k_route_grad<1, decltype(g)::value, decltype(v)::value>), dim3(nwg), dim3(kThreads), 0,
                               stream, a);
    });
    return hipGetLastError();
}

}  // namespace ns
