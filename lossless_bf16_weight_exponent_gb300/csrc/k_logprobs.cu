// k_logprobs.cu - log probabilities of given tokens, entropy and the most probable tokens of each row of logits
// (sm_103a).
//
// With z = x / T and m the row's maximum, one pass keeps s = sum e^(z - m) and w = sum (z - m) e^(z - m) with a running
// maximum: log p(t) = z_t - m - log s, entropy = log s - w / s.  Powers are of 2 (the factor log2(e) / T joins the
// scaling); differences to the maximum are taken in the logits' own units, where they are exact or nearly so.
//
// A row is the work of a cluster of CTAs (one for many rows, up to eight for few), each on a slice; the leader joins the
// slices' sums and candidates through distributed shared memory in a fixed order.
//
// Top tokens: from the first pass's maxima of the threads comes a bound that at least n of the slice's logits reach; a
// second pass (over data that is in L2) lists the logits at or above it, a few dozen of ordinary rows, and each one's
// rank is the number of larger keys (logit order above the complement of the index, so equal logits go by the lower
// index).  Where too many reach the bound (many equal logits), or a row holds a NaN or an infinity, n rounds of an exact
// maximum take its place.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "launch.cuh"
#include "uw_internal.h"

namespace cg = cooperative_groups;
using namespace uw;

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kCand = 1024;
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

// running maximum m, s = sum 2^(z'), w = sum z' 2^(z') with z' = (x - m) scale
struct Sums {
    float m, s, w;
};

// terms below 2^-200 are 0; the bound keeps 0 * inf out of w
constexpr float kFloor = -200.f;

__device__ __forceinline__ Sums join(const Sums &a, const Sums &b, float scale)
{
    Sums r;
    r.m = fmaxf(a.m, b.m);
    if (r.m == -INFINITY) {
        r.s = a.s + b.s;
        r.w = a.w + b.w;
        return r;
    }
    const float da = fmaxf((a.m - r.m) * scale, kFloor), db = fmaxf((b.m - r.m) * scale, kFloor);
    const float ea = exp2_fast(da), eb = exp2_fast(db);
    r.s = a.s * ea + b.s * eb;
    r.w = ea * fmaf(da, a.s, a.w) + eb * fmaf(db, b.s, b.w);
    return r;
}

template <int N>
__device__ __forceinline__ void add(Sums &t, const float (&x)[N], float scale)
{
    float v = x[0];
#pragma unroll
    for (int i = 1; i < N; i++) v = fmaxf(v, x[i]);
    if (v > t.m) {
        const float d = fmaxf((t.m - v) * scale, kFloor), e = exp2_fast(d);
        t.w = e * fmaf(d, t.s, t.w);
        t.s *= e;
        t.m = v;
    }
    if (t.m == -INFINITY) {
        // masked tokens only so far; a NaN still counts
#pragma unroll
        for (int i = 0; i < N; i++)
            if (x[i] != x[i]) t.s = x[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < N; i++) {
        const float z = (x[i] - t.m) * scale, e = exp2_fast(z);
        t.s += e;
        t.w = fmaf(fmaxf(z, kFloor), e, t.w);
    }
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
    __device__ __forceinline__ void vec(int64_t i, float (&f)[V]) const  // i: 16-byte aligned element
    {
        if constexpr (BF16) {
            const uint4 v = __ldg((const uint4 *)((const uint16_t *)p + i));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; q++) {
                f[2 * q] = __uint_as_float(w[q] << 16);
                f[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
            }
        } else {
            const float4 v = __ldg((const float4 *)((const float *)p + i));
            f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
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
        r.vec(s.head + v * V, x);
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

template <bool BF16>
__global__ void __launch_bounds__(kThreads) logprob_kernel(const LpArgs a)
{
    constexpr int V = Row<BF16>::V;
    __shared__ Sums warp_sums[kWarps], cta_sums;
    __shared__ float bounds[kWarps];
    __shared__ unsigned long long cand[kCand], best[kMaxTop], merged[kMaxTop];
    __shared__ int n_cand;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), c = (int)cluster.block_rank();
    const int64_t row = blockIdx.x / C;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Row<BF16> r{BF16 ? (const void *)((const uint16_t *)a.logits + row * a.ld) : (const void *)((const float *)a.logits + row * a.ld)};
    const Slice<V> sl = slice_of<BF16>(r, a.vocab, c, C);
    const int n = a.n_top;

    pdl_trigger();
    pdl_wait();
    Sums t{-INFINITY, 0.f, 0.f};
    for (int64_t v = sl.v0 + threadIdx.x; v < sl.v1; v += kThreads) {
        float x[V];
        r.vec(sl.head + v * V, x);
        add(t, x, a.scale);
    }
    const float vec_max = t.m;  // over whole vectors alone
    for (int64_t i = sl.s0 + threadIdx.x; i < sl.s1; i += kThreads) {
        const float x[1] = {r.at(i)};
        add(t, x, a.scale);
    }
    for (int64_t i = sl.t0 + threadIdx.x; i < sl.t1; i += kThreads) {
        const float x[1] = {r.at(i)};
        add(t, x, a.scale);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) {
        // both lanes join in the same order: the result is the same in each
        const Sums o{__shfl_xor_sync(0xFFFFFFFFu, t.m, d), __shfl_xor_sync(0xFFFFFFFFu, t.s, d), __shfl_xor_sync(0xFFFFFFFFu, t.w, d)};
        t = (lane & d) ? join(o, t, a.scale) : join(t, o, a.scale);
    }
    if (lane == 0) warp_sums[warp] = t;

    if (n) {
        // the warps that have a vector for each lane bring q of their lanes' maxima each, n in all: the least of those
        // is a bound that at least n logits of the slice reach
        const int full = (int)min((int64_t)kWarps, (sl.v1 - sl.v0) / 32);
        float bound = INFINITY;
        if (warp < full) {
            const int q = (n + full - 1) / full;
            float m = vec_max;
            for (int i = 0; i < q; i++) {
                bound = m;
#pragma unroll
                for (int d = 16; d; d >>= 1) bound = fmaxf(bound, __shfl_xor_sync(0xFFFFFFFFu, bound, d));
                const uint32_t who = __ballot_sync(0xFFFFFFFFu, m == bound);
                if (who && lane == __ffs(who) - 1) m = -INFINITY;
            }
        }
        if (lane == 0) bounds[warp] = full ? bound : -INFINITY;
        if (threadIdx.x == 0) n_cand = 0;
    }
    __syncthreads();
    if (warp == 0) {
        Sums u = lane < kWarps ? warp_sums[lane] : Sums{-INFINITY, 0.f, 0.f};
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const Sums o{__shfl_xor_sync(0xFFFFFFFFu, u.m, d), __shfl_xor_sync(0xFFFFFFFFu, u.s, d), __shfl_xor_sync(0xFFFFFFFFu, u.w, d)};
            u = (lane & d) ? join(o, u, a.scale) : join(u, o, a.scale);
        }
        if (lane == 0) cta_sums = u;
    }
    if (n) {
        float bound = bounds[0];
        for (int w = 1; w < kWarps; w++) bound = fminf(bound, bounds[w]);
        if ((int)threadIdx.x < kMaxTop) best[threadIdx.x] = 0ull;
        // NaN and infinities have no place in the bound; NaN sums tell of them
        __syncthreads();
        const bool odd = cta_sums.s != cta_sums.s;
        if (!odd) {
            each<BF16>(r, sl, [&](float x, uint32_t i) {
                if (x >= bound) {
                    const int at = atomicAdd(&n_cand, 1);
                    if (at < kCand) cand[at] = key_of(x, i);
                }
            });
        }
        __syncthreads();
        const int nc = n_cand;
        if (!odd && nc <= kCand) {
            for (int i = threadIdx.x; i < nc; i += kThreads) {
                const unsigned long long k = cand[i];
                int rank = 0;
                for (int j = 0; j < nc; j++) rank += cand[j] > k;
                if (rank < n) best[rank] = k;
            }
        } else {
            unsigned long long last = ~0ull;
            for (int j = 0; j < n; j++) {
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
        }
    }
    if (C > 1) cluster.sync();
    else __syncthreads();

    if (c == 0) {
        Sums u = cta_sums;
        for (int i = 1; i < C; i++) u = join(u, *cluster.map_shared_rank(&cta_sums, i), a.scale);
        const bool none = u.s == 0.f;  // nothing but masked tokens
        const float log_s = logf(u.s);
        auto lp_of = [&](float x) { return none ? -INFINITY : (x - u.m) * a.inv_t - log_s; };
        if (threadIdx.x == 0) {
            if (a.logprob) {
                const int32_t tg = a.targets[row];
                a.logprob[row] = tg < 0 ? 0.f : tg >= a.vocab ? __int_as_float(0x7FC00000) : lp_of(r.at(tg));
            }
            if (a.entropy) a.entropy[row] = none ? 0.f : log_s - u.w / u.s * 0.69314718055994531f;
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
