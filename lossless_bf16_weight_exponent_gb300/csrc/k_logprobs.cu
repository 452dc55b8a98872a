// k_logprobs.cu - log probabilities of given tokens, entropy and the most probable tokens of each row of logits
// (sm_103a).
//
// With z = x / T and m the row's maximum, one pass keeps s = sum e^(z - m) and w = sum (x - m) e^(z - m) with a running
// maximum: log p(t) = (x_t - m) / T - log s, entropy = log s - (w / s) / T.  Powers are of 2 (the factor log2(e) joins the
// scaling); differences to the maximum are taken in the logits' own units, where they are exact or nearly so.  The sums
// are kept in pairs (f32x2 instructions): an element costs its conversion, a comparison, a power and half of five others.
// Logits below -1e37, masked ones above all, count as -1e37: no infinity meets a zero in the sums.  A row whose maximum is
// not above -1e36, or that holds a NaN or +inf (which make s a NaN), is summed again by an exact path.
//
// A row is the work of a cluster of CTAs (one for many rows, up to eight for few), each on a slice; the leader joins the
// slices' sums and candidates through distributed shared memory in a fixed order.
//
// Top tokens in the same pass: from the maxima of the threads over the slice's first eighth comes a bound that at least n
// of its logits reach; logits at or above it are listed (those of the first eighth in a second look at it), a few
// hundred of an ordinary row.  The threads' final maxima give a closer bound, and each remaining one's rank is the number
// of larger keys (logit order above the complement of the index, so equal logits go by the lower index).  A slice in
// which fewer than n logits are not masked lists all of these.  Where too many reach the bound (many equal logits), in a
// row with a NaN or an infinity, and where a row has fewer than n unmasked logits, rounds of an exact maximum find the rest.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "launch.cuh"
#include "uw_internal.h"

namespace cg = cooperative_groups;
using namespace uw;

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kCand = 2048;
constexpr int kUnroll = 4;             // 16-byte loads of a thread on their way
constexpr float kLow = -1e37f;         // masked logits count as this, or in bf16 as the next value below it
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

// f32x2 arithmetic
struct Pair {
    unsigned long long v;
};
__device__ __forceinline__ Pair pair(float a, float b)
{
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(a), "f"(b));
    return p;
}
__device__ __forceinline__ void unpair(Pair p, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v)); }
__device__ __forceinline__ Pair add2(Pair a, Pair b)
{
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b)
{
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c)
{
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
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
    // x: clamped logits, v: their maximum
    template <int N>
    __device__ __forceinline__ void add(const float (&x)[N], float v, float scale)
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
        if (x > m) {
            const float d = m - x, e = exp2_fast(d * scale);
            if (e == 0.f) {
                s = w = pair(0.f, 0.f);
            } else {
                w = mul2(fma2(pair(d, d), s, w), pair(e, e));
                s = mul2(s, pair(e, e));
            }
            m = x;
        }
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

// the exact path: m may be -inf (nothing but masked tokens so far)
__device__ __forceinline__ Sums join_exact(const Sums &a, const Sums &b, float scale)
{
    if (a.m == -INFINITY && a.s == 0.f) return b;
    if (b.m == -INFINITY && b.s == 0.f) return a;
    return join(a, b, scale);
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
    __device__ __forceinline__ float at(int64_t i) const
    {
        return BF16 ? __bfloat162float(((const __nv_bfloat16 *)p)[i]) : ((const float *)p)[i];
    }
    __device__ __forceinline__ uint4 load(int64_t i) const  // i: 16-byte aligned element
    {
        return __ldg((const uint4 *)((const uint8_t *)p + i * (16 / V)));
    }
    // the elements of a load; CLAMP: with clamp_low
    template <bool CLAMP>
    static __device__ __forceinline__ void split(const uint4 &v, float (&f)[V])
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int q = 0; q < 4; q++) {
            if constexpr (BF16) {
                uint32_t u = w[q];
                // -1e37 in bf16 twice
                if (CLAMP) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(u) : "r"(u), "r"(0xFCF1FCF1u));
                f[2 * q] = __uint_as_float(u << 16);
                f[2 * q + 1] = __uint_as_float(u & 0xFFFF0000u);
            } else {
                f[q] = CLAMP ? clamp_low(__uint_as_float(w[q])) : __uint_as_float(w[q]);
            }
        }
    }
};

// a CTA's slice of a row: whole 16-byte vectors [v0, v1) from element `head` on, and single elements (the row's
// unaligned head for the first CTA, its tail for the last) that threads take one each
template <int V>
struct Slice {
    int64_t head, v0, v1, s0, s1;  // singles: [s0, s1)
    int64_t t0, t1;                // and [t0, t1)
};

template <bool BF16>
__device__ __forceinline__ Slice<Row<BF16>::V> slice_of(const Row<BF16> &r, int64_t vocab, int c, int C)
{
    constexpr int V = Row<BF16>::V;
    Slice<V> s;
    const int mis = (int)(((uintptr_t)r.p & 15) / (16 / V));
    s.head = min((int64_t)((V - mis) % V), vocab);
    const int64_t nv = (vocab - s.head) / V;
    s.v0 = nv * c / C;
    s.v1 = nv * (c + 1) / C;
    s.s0 = 0;
    s.s1 = c == 0 ? s.head : 0;
    s.t0 = s.head + nv * V;
    s.t1 = c == C - 1 ? vocab : s.t0;
    return s;
}

// f(x, index) on each of this thread's elements
template <bool BF16, typename F>
__device__ __forceinline__ void each(const Row<BF16> &r, const Slice<Row<BF16>::V> &s, F f)
{
    constexpr int V = Row<BF16>::V;
    for (int64_t v = s.v0 + threadIdx.x; v < s.v1; v += kThreads) {
        float x[V];
        Row<BF16>::template split<false>(r.load(s.head + v * V), x);
#pragma unroll
        for (int i = 0; i < V; i++) f(x[i], (uint32_t)(s.head + v * V + i));
    }
    for (int64_t i = s.s0 + threadIdx.x; i < s.s1; i += kThreads) f(r.at(i), (uint32_t)i);
    for (int64_t i = s.t0 + threadIdx.x; i < s.t1; i += kThreads) f(r.at(i), (uint32_t)i);
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

// a bound that at least n of the values behind the threads' maxima reach: the warps whose lanes all have one (the first
// `full`) bring q of their lanes' maxima each, n in all, and the least of those is it; -inf without such a warp
__device__ __forceinline__ float bound_of(float m, int full, int n, float *warp_bounds)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float bound = INFINITY;
    if (warp < full) {
        const int q = (n + full - 1) / full;
        for (int i = 0; i < q; i++) {
            bound = m;
#pragma unroll
            for (int d = 16; d; d >>= 1) bound = fmaxf(bound, __shfl_xor_sync(0xFFFFFFFFu, bound, d));
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, m == bound);
            if (who && lane == __ffs(who) - 1) m = -INFINITY;
        }
    }
    __syncthreads();
    if (lane == 0) warp_bounds[warp] = bound;
    __syncthreads();
    if (full == 0) return -INFINITY;
    float b = warp_bounds[0];
#pragma unroll
    for (int w = 1; w < kWarps; w++) b = fminf(b, warp_bounds[w]);
    return b;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) logprob_kernel(const LpArgs a)
{
    constexpr int V = Row<BF16>::V;
    __shared__ Sums warp_sums[kWarps], cta_sums;
    __shared__ float bounds[kWarps];
    __shared__ unsigned long long cand[kCand], best[kMaxTop], merged[kMaxTop];
    __shared__ uint16_t kept[kCand];
    __shared__ int n_cand, n_kept, n_best;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), c = (int)cluster.block_rank();
    const int64_t row = blockIdx.x / C;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Row<BF16> r{BF16 ? (const void *)((const uint16_t *)a.logits + row * a.ld) : (const void *)((const float *)a.logits + row * a.ld)};
    const Slice<V> sl = slice_of<BF16>(r, a.vocab, c, C);
    const int n = a.n_top;
    const float scale = a.scale;

    if (threadIdx.x == 0) n_cand = n_kept = 0;
    pdl_trigger();
    pdl_wait();

    // joins the threads' sums; the CTA's in cta_sums after the last barrier
    auto cta_join = [&](Sums t, auto join_fn) {
        auto lanes = [&](Sums u) {
#pragma unroll
            for (int d = 16; d; d >>= 1) {
                // both lanes join in the same order: the result is the same in each
                const Sums o{__shfl_xor_sync(0xFFFFFFFFu, u.m, d), __shfl_xor_sync(0xFFFFFFFFu, u.s, d), __shfl_xor_sync(0xFFFFFFFFu, u.w, d)};
                u = (lane & d) ? join_fn(o, u, scale) : join_fn(u, o, scale);
            }
            return u;
        };
        t = lanes(t);
        __syncthreads();
        if (lane == 0) warp_sums[warp] = t;
        __syncthreads();
        if (warp == 0) {
            t = lanes(lane < kWarps ? warp_sums[lane] : Sums{-INFINITY, 0.f, 0.f});
            if (lane == 0) cta_sums = t;
        }
        __syncthreads();
    };
    static_assert(kWarps <= 32, "the join of the warps' sums");

    PairSums sums;
    float bound = INFINITY;
    // the sums over vectors [v, v1), kThreads apart, and the list of those that reach the bound
    auto sweep = [&](int64_t v, int64_t v1, auto collect) {
        for (; v < v1; v += kUnroll * kThreads) {
            uint4 raw[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; u++)
                if (v + u * kThreads < v1) raw[u] = r.load(sl.head + (v + u * kThreads) * V);
#pragma unroll
            for (int u = 0; u < kUnroll; u++) {
                if (v + u * kThreads >= v1) break;
                float x[V];
                Row<BF16>::template split<true>(raw[u], x);
                float mx = x[0];
#pragma unroll
                for (int i = 1; i < V; i++) mx = fmaxf(mx, x[i]);
                sums.add(x, mx, scale);
                if (decltype(collect)::value && mx >= bound) {
#pragma unroll
                    for (int i = 0; i < V; i++)
                        if (x[i] >= bound) {
                            const int k = atomicAdd(&n_cand, 1);
                            if (k < kCand) cand[k] = key_of(x[i], (uint32_t)(sl.head + (v + u * kThreads) * V + i));
                        }
                }
            }
        }
    };
    const int64_t nv = sl.v1 - sl.v0;
    int64_t done = sl.v0;
    if (n) {
        constexpr int64_t kStep = kUnroll * kThreads;
        const int64_t first = min(nv, (nv / 8 + kStep - 1) / kStep * kStep);
        done = sl.v0 + first;
        sweep(sl.v0 + threadIdx.x, done, std::false_type());
        bound = bound_of(sums.m, (int)min((int64_t)kWarps, first / 32), n, bounds);
        // no bound above the masked logits: every logit above them is listed
        const float above = BF16 ? __uint_as_float(0xFCF00000u) : __uint_as_float(__float_as_uint(kLow) - 1);
        bound = fmaxf(bound, above);
        for (int64_t v = sl.v0 + threadIdx.x; v < done; v += kThreads) {
            float x[V];
            Row<BF16>::template split<false>(r.load(sl.head + v * V), x);
#pragma unroll
            for (int i = 0; i < V; i++)
                if (x[i] >= bound) {
                    const int k = atomicAdd(&n_cand, 1);
                    if (k < kCand) cand[k] = key_of(x[i], (uint32_t)(sl.head + v * V + i));
                }
        }
        sweep(done + threadIdx.x, sl.v1, std::true_type());
    } else {
        sweep(done + threadIdx.x, sl.v1, std::false_type());
    }
    const float vec_max = sums.m;  // over whole vectors alone
    auto single = [&](int64_t i) {
        const float x = r.at(i);
        sums.add1(clamp_low(x), scale);
        if (n && x >= bound) {
            const int k = atomicAdd(&n_cand, 1);
            if (k < kCand) cand[k] = key_of(x, (uint32_t)i);
        }
    };
    for (int64_t i = sl.s0 + threadIdx.x; i < sl.s1; i += kThreads) single(i);
    for (int64_t i = sl.t0 + threadIdx.x; i < sl.t1; i += kThreads) single(i);
    cta_join(sums.total(), [](const Sums &p, const Sums &q, float s) { return join(p, q, s); });

    // the slice's top: complete (n, or all it has), or all of its unmasked logits
    auto rounds = [&](int from) {
        unsigned long long last = from ? best[from - 1] : ~0ull;
        for (int j = from; j < n; j++) {
            unsigned long long k = 0ull;
            each<BF16>(r, sl, [&](float x, uint32_t i) {
                const unsigned long long o = key_of(x, i);
                if (o < last && o > k) k = o;
            });
            k = warp_max(k);
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
        const int nc = n_cand;
        const bool odd = cta_sums.s != cta_sums.s;  // a NaN or +inf
        if (!odd && nc <= kCand) {
            // the closer bound
            const float b2 = bound_of(vec_max, (int)min((int64_t)kWarps, nv / 32), n, bounds);
            const unsigned long long kb = b2 > bound ? key_of(b2, 0xFFFFFFFFu) : 0ull;
            for (int i = threadIdx.x; i < nc; i += kThreads)
                if (cand[i] >= kb) kept[atomicAdd(&n_kept, 1)] = (uint16_t)i;
            __syncthreads();
            const int nk = n_kept;
            for (int i = threadIdx.x; i < nk; i += kThreads) {
                const unsigned long long k = cand[kept[i]];
                int rank = 0;
                for (int j = 0; j < nk; j++) rank += cand[kept[j]] > k;
                if (rank < n) best[rank] = k;
            }
            if (threadIdx.x == 0) n_best = min(nk, n);
            __syncthreads();
        } else {
            __syncthreads();
            rounds(0);
            if (threadIdx.x == 0) n_best = n;
        }
    }
    if (C > 1) cluster.sync();
    else __syncthreads();

    // every CTA of the row comes to the same view of it
    Sums row_sums = cta_sums;
    int have = n_best;
    if (C > 1) {
        row_sums = *cluster.map_shared_rank(&cta_sums, 0);
        have = n ? *cluster.map_shared_rank(&n_best, 0) : 0;
        for (int i = 1; i < C; i++) {
            row_sums = join(row_sums, *cluster.map_shared_rank(&cta_sums, i), scale);
            if (n) have += *cluster.map_shared_rank(&n_best, i);
        }
    }
    const bool again = !(row_sums.m > -1e36f) || row_sums.s != row_sums.s;
    const bool lack = n && have < n;
    if (again || lack) {
        if (C > 1) cluster.sync();  // the others have read cta_sums and n_best
        else __syncthreads();
        if (lack) rounds(n_best);
        if (again) {
            Sums t{-INFINITY, 0.f, 0.f};
            each<BF16>(r, sl, [&](float x, uint32_t) {
                t = x == -INFINITY ? t : join_exact(t, Sums{x, (x - x) + 1.f, 0.f}, scale);  // a NaN for an infinity
            });
            cta_join(t, [](const Sums &p, const Sums &q, float s) { return join_exact(p, q, s); });
        }
        if (C > 1) cluster.sync();
        else __syncthreads();
        if (again) {
            row_sums = *cluster.map_shared_rank(&cta_sums, 0);
            for (int i = 1; i < C; i++) row_sums = join_exact(row_sums, *cluster.map_shared_rank(&cta_sums, i), scale);
        }
    }

    if (c == 0) {
        const bool none = row_sums.s == 0.f;  // nothing but masked tokens
        const float log_s = logf(row_sums.s);
        auto lp_of = [&](float x) { return none ? -INFINITY : (x - row_sums.m) * a.inv_t - log_s; };
        if (threadIdx.x == 0) {
            if (a.logprob) {
                const int32_t tg = a.targets[row];
                a.logprob[row] = tg < 0 ? 0.f : tg >= a.vocab ? __int_as_float(0x7FC00000) : lp_of(r.at(tg));
            }
            if (a.entropy) a.entropy[row] = none ? 0.f : log_s - row_sums.w / row_sums.s * a.inv_t;
        }
        if (n) {
            for (int i = threadIdx.x; i < C * n; i += kThreads) cand[i] = cluster.map_shared_rank(best, i / n)[i % n];
            __syncthreads();
            for (int i = threadIdx.x; i < C * n; i += kThreads) {
                const unsigned long long k = cand[i];
                int rank = 0;
                for (int j = 0; j < C * n; j++) rank += cand[j] > k;
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
    if (C > 1) cluster.sync();  // the leader reads the others' shared memory
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
    // few rows: several CTAs a row, while a slice keeps 4096 logits
    int C = 1;
    while (C < kMaxCluster && rows * C * 2 <= 2 * num_sms() && vocab / (C * 2) >= 4096) C *= 2;
    const cudaError_t e = launch_dependent(dtype == UW_OUT_BF16 ? logprob_kernel<true> : logprob_kernel<false>, dim3((unsigned)(rows * C)), kThreads, 0,
                                           (unsigned)C, (cudaStream_t)stream, a);
    return e == cudaSuccess ? UW_OK : fail(UW_ERR_CUDA, "uw_token_logprobs: launch: %s", cudaGetErrorString(e));
}
