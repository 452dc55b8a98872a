// k_logprobs.cu - log probabilities of given tokens, entropy and the most probable tokens of each row of logits
// (sm_103a).
//
// With z = x / T and m the row's maximum, one pass keeps s = sum e^(z - m) and w = sum (x - m) e^(z - m) with a running
// maximum: log p(t) = (x_t - m) / T - log s, entropy = log s - (w / s) / T.  Powers are of 2 (the factor log2(e) joins the
// scaling); differences to the maximum are taken in the logits' own units, where they are exact or nearly so.  The sums
// are kept in pairs (f32x2 instructions): the formula costs an element its conversion, a comparison, a power and half of five
// others.  The power is the fast one, off by about as much (2^-22) as the rounding of its argument moves it: the results are
// within 7e-8 of 64-bit ones (root mean square; elementary fp32 operations come within 1.6e-7).
// Logits below -1e37, masked ones above all, count as -1e37: no infinity meets a zero in the sums.  A row whose maximum is
// not above -1e36, that holds a NaN or +inf (which make s a NaN), or whose w is past the range (a difference to a maximum above
// 3.3e38 is) is summed again by an exact path, with w in the scaled units; so is every row at temperatures above 7e34.
//
// A row is the work of a cluster of CTAs (one for many rows, up to eight for few), each on a slice; the leader joins the
// slices' sums and candidates through distributed shared memory in a fixed order.
//
// Top tokens in the same pass: from the maxima of the threads over the slice's first eighth comes a bound that at least n
// of its logits reach.  Groups of four loads that hold a logit at or above it are noted with their maximum, some n of each
// further eighth of an ordinary row.  The threads' final maxima give a closer bound; the groups that reach it are looked
// through and their logits at or above it listed.  Each listed logit's rank is the number of larger keys (logit order above
// the complement of the index, so equal logits go by the lower index).
// A slice in which fewer than n logits are not masked lists all of these.  Where too many reach the bound (many equal
// logits), in a row with a NaN or an infinity, and where a row has fewer than n unmasked logits, rounds of an exact maximum
// find the rest.
//
// Bound by memory for long rows: 256 rows of 128256 fp32 with the top 5 take 29 us (4.5 TB/s), 2047 rows of 32064 bf16
// without top tokens 27.9 (4.7 TB/s; the issue slots are 69 % busy: 10.2 warp instructions for 32 elements, 14.7 in fp32, where
// selects at the end of a slice, moves into pairs and the double buffer join the formula's), with the top 20 58, of which the
// lists and ranks of 2047 rows are the half.  1 row of 128256 with the top 20 takes 10.4 us: the launch,
// one pass over 16032 logits by each of eight CTAs and four joins.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "f32x2.cuh"
#include "launch.cuh"
#include "uw_internal.h"

namespace cg = cooperative_groups;
using namespace uw;
using namespace uw::dev;

namespace {

constexpr int kMaxTop = 32;
constexpr int kCand = 1024;            // logits listed for the top tokens
constexpr int kGroups = 1024;          // groups of loads that hold one
constexpr int kUnroll = 4;             // 16-byte loads of a thread on their way
constexpr float kLow = -1e37f;         // masked logits count as this, or in bf16 as the next value below it
constexpr float kLeastScale = 2e-35f;  // below, what counts as kLow would keep a probability beside a maximum of -1e36
constexpr int kMaxCluster = 8;

struct LpArgs {
    const void *logits;
    int64_t rows, vocab, ld;
    float scale, inv_t;  // log2(e) / T, 1 / T
    const int32_t *targets;
    float *logprob, *entropy;
    int n_top;
    int32_t *top_ids;
    float *top_lp;
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// running maximum m, s = sum 2^(d scale), w = sum d 2^(d scale) with d = x - m; m is finite unless a logit is +inf
struct Sums {
    float m, s, w;
};

__device__ __forceinline__ Sums join(const Sums &a, const Sums &b, float scale)
{
    Sums r;
    r.m = fmaxf(a.m, b.m);
    const float da = a.m - r.m, db = b.m - r.m;
    const float ea = exp2_fast(da * scale), eb = exp2_fast(db * scale);
    r.s = a.s * ea + b.s * eb;
    // a factor of 0 ends the term: its difference times its sum may be past the range
    r.w = (ea == 0.f ? 0.f : ea * fmaf(da, a.s, a.w)) + (eb == 0.f ? 0.f : eb * fmaf(db, b.s, b.w));
    return r;
}

// a thread's sums in pairs
struct PairSums {
    float m;
    Pair s, w;
    __device__ __forceinline__ PairSums() : m(kLow), s(pair(0.f, 0.f)), w(pair(0.f, 0.f)) {}
    // the maximum becomes at least v
    __device__ __forceinline__ void raise(float v, float scale)
    {
        if (v > m) {
            const float d = m - v, e = exp2_fast(d * scale);
            if (e == 0.f) {
                s = w = pair(0.f, 0.f);
            } else {
                w = mul2(fma2(pair(d, d), s, w), pair(e, e));
                s = mul2(s, pair(e, e));
            }
            m = v;
        }
    }
    // x: raised logits, none above m
    template <int N>
    __device__ __forceinline__ void add(const float (&x)[N], float scale)
    {
        const Pair nm = pair(-m, -m), sc = pair(scale, scale);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const Pair d = add2(pair(x[i], x[i + 1]), nm);
            float z0, z1;
            unpair(mul2(d, sc), z0, z1);
            const Pair e = pair(exp2_fast(z0), exp2_fast(z1));
            s = add2(s, e);
            w = fma2(d, e, w);
        }
    }
    __device__ __forceinline__ void add1(float x, float scale)
    {
        raise(x, scale);
        const float d = x - m, e = exp2_fast(d * scale);
        s = add2(s, pair(e, 0.f));
        w = fma2(pair(d, 0.f), pair(e, 0.f), w);
    }
    __device__ __forceinline__ Sums total() const
    {
        float s0, s1, w0, w1;
        unpair(s, s0, s1);
        unpair(w, w0, w1);
        return Sums{m, s0 + s1, w0 + w1};
    }
};

// max(x, kLow) that keeps a NaN
__device__ __forceinline__ float clamp_low(float x)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(kLow));
    return y;
}

// The exact path: m may be -inf (nothing but masked tokens so far), and w is the sum of z 2^z with z = d scale, which ends
// where 2^z does.  Halves keep the difference of two finite logits within the range.
__device__ __forceinline__ Sums join_exact(const Sums &a, const Sums &b, float scale)
{
    if (a.m == -INFINITY && a.s == 0.f) return b;
    if (b.m == -INFINITY && b.s == 0.f) return a;
    Sums r;
    r.m = fmaxf(a.m, b.m);
    const float za = 2.f * ((0.5f * a.m - 0.5f * r.m) * scale), zb = 2.f * ((0.5f * b.m - 0.5f * r.m) * scale);
    const float ea = exp2_fast(za), eb = exp2_fast(zb);
    r.s = a.s * ea + b.s * eb;
    r.w = (ea == 0.f ? 0.f : ea * fmaf(za, a.s, a.w)) + (eb == 0.f ? 0.f : eb * fmaf(zb, b.s, b.w));
    return r;
}

__device__ __forceinline__ unsigned long long key_of(float x, uint32_t i)
{
    x += 0.f;
    const uint32_t b = __float_as_uint(x);
    const uint32_t k = x != x ? 0xFFFFFFFEu : (b & 0x80000000u) ? ~b : b | 0x80000000u;
    return ((unsigned long long)k << 32) | (uint32_t)~i;
}

template <bool BF16>
struct Row {
    static constexpr int V = BF16 ? 8 : 4;  // elements of a 16-byte load
    const void *p;
    __device__ __forceinline__ float at(int i) const
    {
        return BF16 ? __bfloat162float(((const __nv_bfloat16 *)p)[i]) : ((const float *)p)[i];
    }
    __device__ __forceinline__ uint4 load(int i) const  // i: 16-byte aligned element
    {
        return *(const uint4 *)((const uint8_t *)p + (uint32_t)i * (16u / V));
    }
    // a load with its masked logits raised to kLow or the next value below it
    static __device__ __forceinline__ uint4 raised(const uint4 &v)
    {
        return make_uint4(raised1(v.x), raised1(v.y), raised1(v.z), raised1(v.w));
    }
    static __device__ __forceinline__ uint32_t raised1(uint32_t w)
    {
        uint32_t u;
        if constexpr (BF16) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(u) : "r"(w), "r"(0xFCF1FCF1u));
        else asm("max.NaN.f32 %0, %1, %2;" : "=r"(u) : "r"(w), "r"(__float_as_uint(kLow)));
        return u;
    }
    // the largest element of N loads
    template <int N>
    static __device__ __forceinline__ float largest(const uint4 (&v)[N])
    {
        auto max1 = [](uint32_t a, uint32_t b) {
            uint32_t u;
            if constexpr (BF16) asm("max.bf16x2 %0, %1, %2;" : "=r"(u) : "r"(a), "r"(b));
            else asm("max.f32 %0, %1, %2;" : "=r"(u) : "r"(a), "r"(b));
            return u;
        };
        uint32_t m = max1(max1(v[0].x, v[0].y), max1(v[0].z, v[0].w));
#pragma unroll
        for (int i = 1; i < N; i++) m = max1(m, max1(max1(v[i].x, v[i].y), max1(v[i].z, v[i].w)));
        if constexpr (BF16) return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
        else return __uint_as_float(m);
    }
    static __device__ __forceinline__ void split(const uint4 &v, float (&f)[V])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; q++) {
            if constexpr (BF16) {
                f[2 * q] = __uint_as_float(w[q] << 16);
                f[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
            } else {
                f[q] = __uint_as_float(w[q]);
            }
        }
    }
};

// a CTA's slice of a row: whole 16-byte vectors [v0, v1) from element `head` on, and single elements (the row's
// unaligned head for the first CTA, its tail for the last) that threads take one each; a row has at most 2^24 elements
struct Slice {
    int head, v0, v1, s1;  // singles: [0, s1)
    int t0, t1;            // and [t0, t1)
};

// CTA c of 1 << cs
template <bool BF16>
__device__ __forceinline__ Slice slice_of(const Row<BF16> &r, int vocab, int c, int cs)
{
    constexpr int V = Row<BF16>::V;
    Slice s;
    const int mis = (int)((uint32_t)(uintptr_t)r.p & 15u) / (16 / V);
    s.head = min((V - mis) % V, vocab);
    const int nv = (vocab - s.head) / V;
    s.v0 = (nv * c) >> cs;  // at most 2^22 vectors by 8
    s.v1 = (nv * (c + 1)) >> cs;
    s.s1 = c == 0 ? s.head : 0;
    s.t0 = s.head + nv * V;
    s.t1 = c == (1 << cs) - 1 ? vocab : s.t0;
    return s;
}

// f(x, index) on each of this thread's elements
template <bool BF16, int THREADS, typename F>
__device__ __forceinline__ void each(const Row<BF16> &r, const Slice &s, F f)
{
    constexpr int V = Row<BF16>::V;
    for (int v = s.v0 + threadIdx.x; v < s.v1; v += THREADS) {
        float x[V];
        Row<BF16>::split(r.load(s.head + v * V), x);
#pragma unroll
        for (int i = 0; i < V; i++) f(x[i], (uint32_t)(s.head + v * V + i));
    }
    for (int i = threadIdx.x; i < s.s1; i += THREADS) f(r.at(i), (uint32_t)i);
    for (int i = s.t0 + threadIdx.x; i < s.t1; i += THREADS) f(r.at(i), (uint32_t)i);
}

__device__ __forceinline__ unsigned long long warp_max(unsigned long long k)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        const unsigned long long o = __shfl_xor_sync(0xFFFFFFFFu, k, d);
        k = o > k ? o : k;
    }
    return k;
}

// What few threads come to stays out of line: the kernel's own code has to fit the instruction cache (with these inline,
// waits for instructions were a third of its time on short rows).

// this thread's largest key below `last`
template <bool BF16, int THREADS>
__device__ __noinline__ unsigned long long largest_below(const Row<BF16> r, const Slice s, unsigned long long last)
{
    unsigned long long k = 0ull;
    each<BF16, THREADS>(r, s, [&](float x, uint32_t i) {
        const unsigned long long o = key_of(x, i);
        if (o < last && o > k) k = o;
    });
    return k;
}

// this thread's sums, exactly: a NaN for an infinity, nothing for a masked token
template <bool BF16, int THREADS>
__device__ __noinline__ Sums exact_sums(const Row<BF16> r, const Slice s, float scale)
{
    Sums t{-INFINITY, 0.f, 0.f};
    each<BF16, THREADS>(r, s, [&](float x, uint32_t) {
        if (x != -INFINITY) t = join_exact(t, Sums{x, (x - x) + 1.f, 0.f}, scale);
    });
    return t;
}

// A bound that at least n of the values behind the threads' maxima reach, and few more: the warps whose lanes all have
// one (the first `full`) bring a few of their largest each, and the n-th largest of these is it; -inf without such a warp.
template <int kWarps>
__device__ __forceinline__ float bound_of(float m, int full, int n, float *top)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (full == 0) return -INFINITY;
    const int q = min(32, (n + full - 1) / full + 1);  // full q <= 63 values, at least n
    if (warp < full) {
        const uint32_t b = __float_as_uint(m + 0.f);
        uint32_t k = (b & 0x80000000u) ? ~b : b | 0x80000000u;  // in the order of the values, above 0
        for (int i = 0; i < q; i++) {
            const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, k);
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, k == best);
            if (lane == __ffs(who) - 1) {
                k = 0u;
                top[warp * q + i] = __uint_as_float((best & 0x80000000u) ? best & 0x7FFFFFFFu : ~best);
            }
        }
    }
    __syncthreads();
    const int k = full * q;
    const float v0 = lane < k ? top[lane] : -INFINITY, v1 = lane + 32 < k ? top[lane + 32] : -INFINITY;
    int g0 = 0, g1 = 0;  // larger values
    for (int i = 0; i < k; i++) {
        const float v = top[i];
        g0 += v > v0;
        g1 += v > v1;
    }
    float b = fminf(lane < k && g0 < n ? v0 : INFINITY, lane + 32 < k && g1 < n ? v1 : INFINITY);
#pragma unroll
    for (int d = 16; d; d >>= 1) b = fminf(b, __shfl_xor_sync(0xFFFFFFFFu, b, d));
    __syncthreads();
    return b;
}

template <bool BF16, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) logprob_kernel(const LpArgs a, int cs)
{
    constexpr int kWarps = kThreads / 32;
    constexpr int V = Row<BF16>::V;
    __shared__ Sums warp_sums[kWarps];
    __shared__ float bounds[64];
    __shared__ unsigned long long cand[kCand], best[kMaxTop], merged[kMaxTop];
    __shared__ int groups[kGroups], n_groups, n_cand;
    __shared__ float group_max[kGroups];
    // written by the row's CTAs: their sums and counts in each, their top tokens in the leader
    __shared__ Sums row_parts[kMaxCluster];
    __shared__ int row_have[kMaxCluster];
    __shared__ unsigned long long row_tops[kMaxCluster * kMaxTop];
    cg::cluster_group cluster = cg::this_cluster();
    const int C = 1 << cs, c = (int)(blockIdx.x & (C - 1));  // the cluster's CTAs are a row's
    const int64_t row = blockIdx.x >> cs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Row<BF16> r{BF16 ? (const void *)((const uint16_t *)a.logits + row * a.ld) : (const void *)((const float *)a.logits + row * a.ld)};
    const int vocab = (int)a.vocab;
    const Slice sl = slice_of<BF16>(r, vocab, c, cs);
    const int n = a.n_top;
    const float scale = a.scale;

    if (threadIdx.x == 0) n_groups = n_cand = 0;
    // The row's CTAs write into each other's shared memory: each has to be known to run first.  The arrival is here and the wait
    // before the first of those writes, so that it costs nothing.
    if (C > 1) cluster.barrier_arrive();
    pdl_trigger();
    __syncthreads();
    pdl_wait();

    auto lanes_join = [&](Sums u, auto join_fn) {
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            // both lanes join in the same order: the result is the same in each
            const Sums o{__shfl_xor_sync(0xFFFFFFFFu, u.m, d), __shfl_xor_sync(0xFFFFFFFFu, u.s, d), __shfl_xor_sync(0xFFFFFFFFu, u.w, d)};
            u = (lane & d) ? join_fn(o, u, scale) : join_fn(u, o, scale);
        }
        return u;
    };
    // the CTA's sums, in every thread (lowest: the maximum of none)
    auto cta_join = [&](Sums t, float lowest, auto join_fn) {
        t = lanes_join(t, join_fn);
        if (lane == 0) warp_sums[warp] = t;
        __syncthreads();
        return lanes_join(lane < kWarps ? warp_sums[lane] : Sums{lowest, 0.f, 0.f}, join_fn);
    };
    // to every CTA of the row, and to the leader
    auto publish = [&](const Sums &t, int have) {
        if (threadIdx.x < C) {
            *cluster.map_shared_rank(&row_parts[c], threadIdx.x) = t;
            *cluster.map_shared_rank(&row_have[c], threadIdx.x) = have;
        }
        if ((int)threadIdx.x < n) cluster.map_shared_rank(row_tops, 0)[c * n + threadIdx.x] = best[threadIdx.x];
    };
    auto row_sync = [&] {
        if (C > 1) cluster.sync();
        else __syncthreads();
    };
    static_assert(kUnroll * V <= 32, "a group's elements");
    static_assert(kWarps <= 32, "the join of the warps' sums");

    PairSums sums;
    float bound = INFINITY;
    // a thread's group of loads, from vector v, holds a logit that reaches the bound; none is above mx
    auto note = [&](int v, float mx) {
        const int at = atomicAdd(&n_groups, 1);
        if (at < kGroups) groups[at] = v, group_max[at] = mx;
    };
    auto list = [&](float x, int i) {
        const int at = atomicAdd(&n_cand, 1);
        if (at < kCand) cand[at] = key_of(x, (uint32_t)i);
    };
    constexpr uint32_t kPad = BF16 ? 0xFCF1FCF1u : 0xFCF0BDC2u;  // kLow, as raised: adds nothing and is not listed
    // the sums over vectors [v, v1), kThreads apart, in groups
    auto sweep = [&](int v, int v1) {
        uint4 next[kUnroll];
        auto load = [&](int at) {
#pragma unroll
            for (int u = 0; u < kUnroll; u++)
                next[u] = at + u * kThreads < v1 ? r.load(sl.head + (at + u * kThreads) * V) : make_uint4(kPad, kPad, kPad, kPad);
        };
        if (v < v1) load(v);
        for (; v < v1; v += kUnroll * kThreads) {
            uint4 x[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; u++) x[u] = Row<BF16>::raised(next[u]);
            if (v + kUnroll * kThreads < v1) load(v + kUnroll * kThreads);  // on their way during the sums
            const float mx = Row<BF16>::largest(x);
            sums.raise(mx, scale);
#pragma unroll
            for (int u = 0; u < kUnroll; u++) {
                float f[V];
                Row<BF16>::split(x[u], f);
                sums.add(f, scale);
            }
            if (mx >= bound) note(v, mx);
        }
    };
    const int nv = sl.v1 - sl.v0;
    const float unmasked = BF16 ? __uint_as_float(0xFCF00000u) : __uint_as_float(__float_as_uint(kLow) - 1);  // the lowest such logit
    int done = sl.v0;
    if (n) {
        constexpr int kStep = kUnroll * kThreads;
        const int first = min(nv, (nv / 8 + kStep - 1) / kStep * kStep);
        done = sl.v0 + first;
        sweep(sl.v0 + threadIdx.x, done);
        bound = bound_of<kWarps>(sums.m, min(kWarps, first / 32), n, bounds);
        // no bound above the masked logits: every logit above them is listed
        bound = fmaxf(bound, unmasked);
        if (sums.m >= bound)
            for (int v = sl.v0 + threadIdx.x; v < done; v += kStep) note(v, sums.m);
    }
    sweep(done + threadIdx.x, sl.v1);
    const float vec_max = sums.m;  // over whole vectors alone
    auto single = [&](int i) {
        const float x = r.at(i);
        sums.add1(clamp_low(x), scale);
        if (x >= bound) list(x, i);
    };
    for (int i = threadIdx.x; i < sl.s1; i += kThreads) single(i);
    for (int i = sl.t0 + threadIdx.x; i < sl.t1; i += kThreads) single(i);
    auto plain_join = [](const Sums &p, const Sums &q, float s) { return join(p, q, s); };
    auto exact_join = [](const Sums &p, const Sums &q, float s) { return join_exact(p, q, s); };
    Sums row_sums = cta_join(sums.total(), kLow, plain_join);
    int have = 0;

    // the slice's top: complete (n, or all it has), or all of its unmasked logits
    auto rounds = [&](int from) {
        unsigned long long last = from ? best[from - 1] : ~0ull;
        for (int j = from; j < n; j++) {
            unsigned long long k = warp_max(largest_below<BF16, kThreads>(r, sl, last));
            __syncthreads();  // cand is free
            if (lane == 0) cand[warp] = k;
            __syncthreads();
            k = 0ull;
            for (int w = 0; w < kWarps; w++) k = cand[w] > k ? cand[w] : k;
            if (threadIdx.x == 0) best[j] = k;
            last = k;
            if (!k) break;  // the slice has no more
        }
        __syncthreads();
    };
    if (n) {
        if ((int)threadIdx.x < kMaxTop) best[threadIdx.x] = 0ull;
        const int ng = n_groups;
        // the closer bound, where it saves more than it costs (0.8 us of latency)
        const float lim = ng <= 64 || done == sl.v1 ? bound : fmaxf(bound, bound_of<kWarps>(vec_max, min(kWarps, nv / 32), n, bounds));
        bool listed = row_sums.s == row_sums.s && ng <= kGroups;  // no NaN, no +inf
        if (listed) {
            // a thread takes an element of every kThreads, four on their way
            constexpr int kElems = kUnroll * V;
            for (int e0 = threadIdx.x; e0 < ng * kElems; e0 += 4 * kThreads) {
                float x[4];
                int at[4];
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const int e = e0 + u * kThreads, g = e / kElems, k = e % kElems;
                    const int v = g < ng && group_max[g] >= lim ? groups[g] + k / V * kThreads : sl.v1;
                    at[u] = sl.head + v * V + k % V;
                    x[u] = v < sl.v1 ? r.at(at[u]) : -INFINITY;  // below any bound
                }
#pragma unroll
                for (int u = 0; u < 4; u++)
                    if (x[u] >= lim) list(x[u], at[u]);
            }
            __syncthreads();
        }
        const int nc = n_cand;
        listed = listed && nc <= kCand;
        if (listed) {
            for (int i = threadIdx.x; i < nc; i += kThreads) {
                const unsigned long long k = cand[i];
                int rank = 0;
                for (int j = 0; j < nc; j++) rank += cand[j] > k;
                if (rank < n) best[rank] = k;
            }
            have = min(nc, n);
            __syncthreads();
        } else {
            // a NaN or +inf, or a list that is too long
            __syncthreads();
            rounds(0);
            // Of these the unmasked count, as in a list: which masked ones are among the row's top is up to all its slices.
            const unsigned long long least = key_of(unmasked, ~0u);
            for (int j = 0; j < n; j++) have += best[j] >= least;
        }
    }
    if (C > 1) cluster.barrier_wait();
    publish(row_sums, have);
    row_sync();

    // every CTA of the row comes to the same view of it
    int row_n = have;
    if (C > 1) {
        row_sums = lanes_join(lane < C ? row_parts[lane] : Sums{kLow, 0.f, 0.f}, plain_join);
        row_n = 0;
        for (int i = 0; i < C; i++) row_n += row_have[i];
    }
    const bool again = !(row_sums.m > -1e36f) || row_sums.s != row_sums.s || !isfinite(row_sums.w) || scale < kLeastScale;
    const bool lack = n && row_n < n;
    if (again || lack) {
        if (lack) rounds(have);
        if (again) {
            const Sums t = exact_sums<BF16, kThreads>(r, sl, scale);
            row_sync();  // warp_sums is free, and the others have read what was published
            row_sums = cta_join(t, -INFINITY, exact_join);
        } else {
            row_sync();
        }
        publish(row_sums, n);
        row_sync();
        if (again && C > 1) row_sums = lanes_join(lane < C ? row_parts[lane] : Sums{-INFINITY, 0.f, 0.f}, exact_join);
    }

    if (c == 0) {
        const bool none = row_sums.s == 0.f;  // nothing but masked tokens
        const float log_s = logf(row_sums.s);
        auto lp_of = [&](float x) {
            const float d = x - row_sums.m;
            const float z = isinf(d) ? 2.f * ((0.5f * x - 0.5f * row_sums.m) * a.inv_t) : d * a.inv_t;  // past the range as a difference alone
            return none ? -INFINITY : z - log_s;
        };
        const float unit = again ? 0.69314718f : a.inv_t;  // of w
        if (threadIdx.x == 0) {
            if (a.logprob) {
                const int32_t tg = a.targets[row];
                a.logprob[row] = tg < 0 ? 0.f : tg >= vocab ? __int_as_float(0x7FC00000) : lp_of(r.at(tg));
            }
            if (a.entropy) a.entropy[row] = none ? 0.f : log_s - row_sums.w / row_sums.s * unit;
        }
        if (n) {
            for (int i = threadIdx.x; i < C * n; i += kThreads) {
                const unsigned long long k = row_tops[i];
                int rank = 0;
                for (int j = 0; j < C * n; j++) rank += row_tops[j] > k;
                if (k && rank < n) merged[rank] = k;
            }
            __syncthreads();
            if ((int)threadIdx.x < n) {
                const uint32_t id = ~(uint32_t)merged[threadIdx.x];
                a.top_ids[row * n + threadIdx.x] = (int32_t)id;
                a.top_lp[row * n + threadIdx.x] = lp_of(r.at(id));
            }
        }
    }
}

}  // namespace

extern "C" uw_status uw_token_logprobs(const void *logits, uw_out_dtype dtype, int64_t rows, int64_t vocab, int64_t ld, float temperature,
                                       const int32_t *targets, float *logprob, float *entropy, int n_top, int32_t *top_ids,
                                       float *top_logprobs, uw_stream stream)
{
    clear_error();
    if (ld == 0) ld = vocab;
    if (rows < 0 || rows > ((int64_t)1 << 31) / kMaxCluster - 1 || vocab < 1 || vocab > (1 << 24) || ld < vocab)
        return fail(UW_ERR_SHAPE, "uw_token_logprobs: rows=%lld vocab=%lld ld=%lld", (long long)rows, (long long)vocab, (long long)ld);
    if (dtype != UW_OUT_F32 && dtype != UW_OUT_BF16) return fail(UW_ERR_INVALID_ARG, "uw_token_logprobs: bad dtype");
    if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(1.4426950408889634f / temperature))
        return fail(UW_ERR_INVALID_ARG, "uw_token_logprobs: temperature %g", (double)temperature);
    if (n_top < 0 || n_top > kMaxTop || n_top > vocab) return fail(UW_ERR_INVALID_ARG, "uw_token_logprobs: n_top %d", n_top);
    if (!targets != !logprob) return fail(UW_ERR_INVALID_ARG, "uw_token_logprobs: targets and logprob go together");
    if (n_top && (!top_ids || !top_logprobs)) return fail(UW_ERR_INVALID_ARG, "uw_token_logprobs: n_top without its outputs");
    if (((uintptr_t)logits & (dtype == UW_OUT_F32 ? 3 : 1)) || (((uintptr_t)targets | (uintptr_t)logprob | (uintptr_t)entropy |
                                                                 (uintptr_t)top_ids | (uintptr_t)top_logprobs) & 3))
        return fail(UW_ERR_INVALID_ARG, "uw_token_logprobs: a pointer is not aligned to its elements");
    if (rows == 0 || (!logprob && !entropy && !n_top)) return UW_OK;
    if (!logits) return fail(UW_ERR_INVALID_ARG, "uw_token_logprobs: logits NULL");
    const LpArgs a{logits, rows, vocab, ld, 1.4426950408889634f / temperature, 1.f / temperature, targets, logprob, entropy, n_top, top_ids, top_logprobs};
    // Few rows: a cluster of CTAs a row, while the rows fill the GPU at most and a slice keeps 4096 logits (1 row of 128256:
    // 20 us alone, 11 with eight).  Many rows: smaller CTAs, whose fixed part costs less, as soon as their number fills the
    // SMs' 1024 threads (2047 rows of 32064 bf16: 42 us with 512 threads, 31 with 256, 27 with 128).
    int cs = 0;
    while ((1 << cs) < kMaxCluster && (rows << (cs + 1)) <= 2 * num_sms() && (vocab >> (cs + 1)) >= 4096) cs++;
    const int threads = (rows << cs) <= 2 * num_sms() ? 512 : rows <= 4 * num_sms() ? 256 : 128;
    auto go = [&](auto kernel, int t) { return launch_dependent(kernel, dim3((unsigned)(rows << cs)), (unsigned)t, 0, 1u << cs, (cudaStream_t)stream, a, cs); };
    const bool bf16 = dtype == UW_OUT_BF16;
    const cudaError_t e = threads == 128 ? go(bf16 ? logprob_kernel<true, 128> : logprob_kernel<false, 128>, 128)
                        : threads == 256 ? go(bf16 ? logprob_kernel<true, 256> : logprob_kernel<false, 256>, 256)
                                         : go(bf16 ? logprob_kernel<true, 512> : logprob_kernel<false, 512>, 512);
    return e == cudaSuccess ? UW_OK : fail(UW_ERR_CUDA, "uw_token_logprobs: launch: %s", cudaGetErrorString(e));
}
