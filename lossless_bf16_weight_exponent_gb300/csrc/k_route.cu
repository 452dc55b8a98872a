// k_route.cu - the router of a mixture of experts: each token's top-k experts, their weights, and the order of the
// grouped products' rows (sm_103a).
//
// A warp takes a token.  An expert's sort key is its (logit + bias), or (score + bias), mapped to an unsigned integer of the same
// order.  Up to 64
// experts a round of the choice is a warp-wide maximum of the keys left and a warp-wide minimum of the experts that hold
// it, one instruction each, so equal logits go to the lower index.  With more experts the lanes' largest keys give a bound
// that at least k keys reach; those that do, few unless many are equal, take a lane each and are ranked.
//
// Rows are ordered by (expert, token) without counters whose order could change: a CTA sets, for each expert, one bit per
// token in shared memory (a token takes an expert at most once), so a token's rank within the CTA is a population count
// and the CTA's rows per expert are another.  The second kernel adds up the counts of the CTAs before its own and the
// offsets; for many CTAs a scan between the two does.  Up to 128 tokens one CTA does everything in one launch; beyond, a CTA
// takes 64.
//
// Bound by latency: 16 tokens of 64 experts (top 8) take 5.4 us, 8192 of 64 11.4, 4096 of 256 14.0, 16384 of 256 26.8.  The
// bytes of the second and the last would take 0.4 and 2.8 us: a token's loads, exponentials and rounds follow on each
// other, and the order needs every choice.  Rounds over all keys took 20.4 us for 4096 of 256, ranks behind a bound 17.8,
// the next token's logits asked for during a choice 16.0, the order kernel's CTAs kept off the SMs until the choices are
// made 14.0.  Beyond 256 experts a lane holds 32 keys, which spill: 4096 tokens of 384, 512 and 1024 experts take 30, 32 and
// 37 us where 256 take 15 (other logits at each call).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "launch.cuh"
#include "uw_internal.h"

using namespace uw;

namespace {

constexpr int kThreads = 1024;
constexpr int kTokOne = 128;     // tokens that one CTA takes alone
constexpr int kTokMany = 64;     // and when there are more
constexpr int kMaxE = 1024, kMaxTop = 16;

struct RouteArgs {
    uw_router r;  // score without UW_SCORE_CHOOSES
    const void *logits;
    int bf16;
    int64_t tokens, ld;
    int32_t *ids;
    float *weights;
    int32_t *offsets, *row_src, *pos;
    int32_t *counts;  // [CTAs][experts], with a scan [CTAs + 1][experts]
};

__device__ __forceinline__ uint32_t order_key(float f)
{
    f += 0.f;  // -0 and +0 are equal
    const uint32_t b = __float_as_uint(f);
    if (f != f) return 0xFFFFFFFFu;
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float logit_at(const RouteArgs &a, int64_t t, int e)
{
    return a.bf16 ? __bfloat162float(((const __nv_bfloat16 *)a.logits)[t * a.ld + e]) : ((const float *)a.logits)[t * a.ld + e];
}

struct Choice {
    uint32_t key;
    int expert;
    float z;
};

// token t's logits, a warp's lanes side by side
template <int PER>  // PER: experts per lane
__device__ __forceinline__ void load_logits(const RouteArgs &a, int64_t t, int lane, float (&z)[PER])
{
#pragma unroll
    for (int i = 0; i < PER; i++) z[i] = lane + 32 * i < a.r.experts ? logit_at(a, t, lane + 32 * i) : -INFINITY;
}

// the choice of token t by one warp, BY_SCORE by the scores in place of the logits; sets the token's bits (WORDS per expert); few:
// the warp's 32
template <int PER, int WORDS, bool BY_SCORE>
__device__ __forceinline__ void choose(const RouteArgs &a, int64_t t, int lane, const float (&z)[PER], uint32_t *bits, int tl, Choice *few)
{
    const int E = a.r.experts, k = a.r.topk;
    uint32_t key[PER];  // 0: none, or taken
    auto keys = [&](auto value) {
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const int e = lane + 32 * i;
            key[i] = e < E ? order_key(a.r.bias ? value(z[i]) + a.r.bias[e] : value(z[i])) : 0u;
        }
    };
    if constexpr (!BY_SCORE) keys([](float x) { return x; });
    float m = -INFINITY, total = 1.f;
    if (a.r.score == UW_SCORE_SOFTMAX) {
#pragma unroll
        for (int i = 0; i < PER; i++) m = fmaxf(m, z[i]);
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
        total = 0.f;
#pragma unroll
        for (int i = 0; i < PER; i++)
            if (lane + 32 * i < E) total += m == -INFINITY ? (z[i] != z[i] ? z[i] : 0.f) : expf(z[i] - m);
#pragma unroll
        for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
    }
    auto score_of = [&](float x) {
        if (a.r.score == UW_SCORE_SOFTMAX) return total == 0.f ? 0.f : expf(x - m) / total;
        return 1.f / (1.f + expf(-x));
    };
    if constexpr (BY_SCORE) keys(score_of);
    int my_e = 0, place = lane < k ? lane : -1;
    float my_z = 0.f;
    bool chosen = false;
    if constexpr (PER >= 4) {
        // Every lane has an expert, so at least k keys reach the k-th of the lanes' largest.  They are few unless many are
        // equal: each takes a lane, and its rank is the number of keys before it.
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < PER; i++) best = max(best, key[i]);
        uint32_t bound = 0u;
        for (int j = 0; j < k; j++) {
            bound = __reduce_max_sync(0xFFFFFFFFu, best);
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, best == bound);
            if (lane == __ffs(who) - 1) best = 0u;
        }
        int n = 0;
#pragma unroll
        for (int i = 0; i < PER; i++) {
            const uint32_t who = __ballot_sync(0xFFFFFFFFu, key[i] >= bound);
            if (key[i] >= bound) {
                const int at = n + __popc(who & ((1u << lane) - 1u));
                if (at < 32) few[at] = Choice{key[i], lane + 32 * i, z[i]};
            }
            n += __popc(who);
        }
        __syncwarp();
        chosen = n <= 32;
        if (chosen) {
            const Choice mine = lane < n ? few[lane] : Choice{0u, 0, 0.f};
            int rank = 0;
            for (int i = 0; i < n; i++) rank += few[i].key > mine.key || (few[i].key == mine.key && few[i].expert < mine.expert);
            place = lane < n && rank < k ? rank : -1;
            my_e = mine.expert;
            my_z = mine.z;
        }
        __syncwarp();  // before the warp's next token
    }
    for (int j = 0; !chosen && j < k; j++) {
        uint32_t best = 0u;
        int first = 0;
#pragma unroll
        for (int i = PER - 1; i >= 0; i--)
            if (key[i] >= best) {
                best = key[i];
                first = i;
            }
        const uint32_t all = __reduce_max_sync(0xFFFFFFFFu, best);
        const int e = (int)__reduce_min_sync(0xFFFFFFFFu, best == all ? (uint32_t)(lane + 32 * first) : 0xFFFFFFFFu);
        float ze = 0.f;
#pragma unroll
        for (int i = 0; i < PER; i++)
            if (lane + 32 * i == e) {
                ze = z[i];
                key[i] = 0u;
            }
        ze = __shfl_sync(0xFFFFFFFFu, ze, e & 31);
        if (lane == j) {
            my_e = e;
            my_z = ze;
        }
    }
    float w = place >= 0 ? score_of(my_z) : 0.f;
    if (a.r.renormalize) {
        float s = w;
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        w = s == 0.f ? 0.f : w / s;
    }
    if (place >= 0) {
        a.ids[t * k + place] = my_e;
        a.weights[t * k + place] = w * a.r.scale;
        atomicOr(&bits[my_e * WORDS + (tl >> 5)], 1u << (tl & 31));
    }
}

template <int WORDS>
__device__ __forceinline__ int bits_count(const uint32_t *b)
{
    int n = 0;
#pragma unroll
    for (int i = 0; i < WORDS; i++) n += __popc(b[i]);
    return n;
}

// rank of token tl among the CTA's tokens that took the expert
__device__ __forceinline__ int bits_rank(const uint32_t *b, int tl)
{
    int n = __popc(b[tl >> 5] & ((1u << (tl & 31)) - 1u));
    for (int i = 0; i < (tl >> 5); i++) n += __popc(b[i]);
    return n;
}

// v[0..E) in shared memory becomes its exclusive sum; returns the total.  Begins and ends with a barrier.
__device__ __forceinline__ int exclusive_sum(int *v, int E, int *wsum)
{
    constexpr int Q = kMaxE / kThreads;  // consecutive values of a thread
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    int x[Q], s = 0;
#pragma unroll
    for (int i = 0; i < Q; i++) {
        x[i] = Q * (int)threadIdx.x + i < E ? v[Q * threadIdx.x + i] : 0;
        s += x[i];
    }
    int sum = s;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += o;
    }
    if (lane == 31) wsum[warp] = sum;
    __syncthreads();
    int w = lane < kThreads / 32 ? wsum[lane] : 0;
    const int mine = lane < warp ? w : 0;
    int at = sum - s + __reduce_add_sync(0xFFFFFFFFu, mine);
    const int total = __reduce_add_sync(0xFFFFFFFFu, w);
#pragma unroll
    for (int i = 0; i < Q; i++) {
        if (Q * (int)threadIdx.x + i < E) v[Q * threadIdx.x + i] = at;
        at += x[i];
    }
    __syncthreads();
    return total;
}

template <int PER, int TOK, bool BY_SCORE>
__global__ void __launch_bounds__(kThreads, PER <= 2 ? 2 : 1) route_choose_kernel(const RouteArgs a)
{
    constexpr int WORDS = TOK / 32;
    extern __shared__ uint32_t bits[];  // [experts][WORDS]
    __shared__ Choice few[PER >= 4 ? kThreads / 32 : 1][32];
    const int E = a.r.experts, k = a.r.topk;
    const int64_t t0 = (int64_t)blockIdx.x * TOK;
    const int nt = (int)min((int64_t)TOK, a.tokens - t0);
    for (int i = threadIdx.x; i < E * WORDS; i += kThreads) bits[i] = 0u;
    pdl_wait();
    __syncthreads();
    const int lane = threadIdx.x & 31;
    constexpr bool kAhead = PER <= 8;  // the next token's logits on their way during a choice, where registers allow
    float z[PER], next[PER];
    int tl = threadIdx.x >> 5;
    if (tl < nt) load_logits<PER>(a, t0 + tl, lane, z);
    for (; tl < nt; tl += kThreads / 32) {
        const bool more = tl + kThreads / 32 < nt;
        if (kAhead && more) load_logits<PER>(a, t0 + tl + kThreads / 32, lane, next);
        choose<PER, WORDS, BY_SCORE>(a, t0 + tl, lane, z, bits, tl, few[PER >= 4 ? threadIdx.x >> 5 : 0]);
        if (kAhead && more) {
#pragma unroll
            for (int i = 0; i < PER; i++) z[i] = next[i];
        } else if (more) {
            load_logits<PER>(a, t0 + tl + kThreads / 32, lane, z);
        }
    }
    pdl_trigger();
    __syncthreads();
    if (gridDim.x > 1) {
        for (int e = threadIdx.x; e < E; e += kThreads) a.counts[(int64_t)blockIdx.x * E + e] = bits_count<WORDS>(bits + e * WORDS);
        return;
    }
    // all tokens are here: the order too
    __shared__ int wsum[32], base[kMaxE];
    for (int e = threadIdx.x; e < E; e += kThreads) base[e] = bits_count<WORDS>(bits + e * WORDS);
    const int total = exclusive_sum(base, E, wsum);
    for (int e = threadIdx.x; e < E; e += kThreads) a.offsets[e] = base[e];
    if (threadIdx.x == 0) a.offsets[E] = total;
    for (int i = threadIdx.x; i < nt * k; i += kThreads) {
        const int tl = i / k, e = a.ids[i];
        const int r = base[e] + bits_rank(bits + e * WORDS, tl);
        a.pos[i] = r;
        a.row_src[r] = tl;
    }
}

// Many CTAs: each expert's counts become the exclusive sums over the CTAs, with the total after the last.  A CTA takes 32
// experts, lane = expert, a warp a run of consecutive CTAs.
__global__ void __launch_bounds__(kThreads) route_scan_kernel(const RouteArgs a, int ctas)
{
    __shared__ int sums[kThreads / 32][32];
    const int E = a.r.experts, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    const int per = (ctas + kThreads / 32 - 1) / (kThreads / 32), c0 = min(ctas, warp * per), c1 = min(ctas, c0 + per);
    pdl_trigger();
    pdl_wait();
    int32_t *const p = a.counts + e;
    int n = 0;
    if (e < E)
#pragma unroll 16
        for (int c = c0; c < c1; c++) n += p[(int64_t)c * E];
    sums[warp][lane] = n;
    __syncthreads();
    if (e >= E) return;
    int at = 0;
    for (int w = 0; w < warp; w++) at += sums[w][lane];
    for (int c = c0; c < c1; c += 8) {
        int v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = c + i < c1 ? p[(int64_t)(c + i) * E] : 0;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            if (c + i < c1) p[(int64_t)(c + i) * E] = at;
            at += v[i];
        }
    }
    if (warp == kThreads / 32 - 1) p[(int64_t)ctas * E] = at;
}

template <bool SCANNED>
__global__ void __launch_bounds__(kThreads) route_order_kernel(const RouteArgs a, int ctas)
{
    constexpr int WORDS = kTokMany / 32;
    extern __shared__ uint32_t bits[];  // [experts][WORDS]
    __shared__ int wsum[32], base[kMaxE], before[kMaxE];
    const int E = a.r.experts, k = a.r.topk;
    const int64_t t0 = (int64_t)blockIdx.x * kTokMany;
    const int nt = (int)min((int64_t)kTokMany, a.tokens - t0);
    for (int i = threadIdx.x; i < E * WORDS; i += kThreads) bits[i] = 0u;
    if constexpr (!SCANNED)
        for (int e = threadIdx.x; e < E; e += kThreads) base[e] = before[e] = 0;
    pdl_trigger();
    __syncthreads();
    pdl_wait();
    // this CTA's choices; few enough that each thread keeps its first
    const int first = (int)threadIdx.x < nt * k ? a.ids[t0 * k + threadIdx.x] : 0;
    // rows of each expert in all CTAs, and in those before this one: the threads beyond one for each expert share the CTAs
    const int parts = max(1, kThreads / E);
    if constexpr (SCANNED) {
        for (int e = threadIdx.x; e < E; e += kThreads) {
            base[e] = a.counts[(int64_t)ctas * E + e];
            before[e] = a.counts[(int64_t)blockIdx.x * E + e];
        }
    } else for (int i = threadIdx.x; i < E * parts; i += kThreads) {
        const int e = i % E, part = i / E;
        int all = 0, mine = 0;
#pragma unroll 16
        for (int c = part; c < ctas; c += parts) {
            const int n = a.counts[(int64_t)c * E + e];
            all += n;
            mine += c < (int)blockIdx.x ? n : 0;
        }
        if (all) atomicAdd(&base[e], all);
        if (mine) atomicAdd(&before[e], mine);
    }
    for (int i = threadIdx.x; i < nt * k; i += kThreads) {
        const int tl = i / k, e = i == (int)threadIdx.x ? first : a.ids[t0 * k + i];
        atomicOr(&bits[e * WORDS + (tl >> 5)], 1u << (tl & 31));
    }
    const int total = exclusive_sum(base, E, wsum);
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e < E; e += kThreads) a.offsets[e] = base[e];
        if (threadIdx.x == 0) a.offsets[E] = total;
    }
    for (int i = threadIdx.x; i < nt * k; i += kThreads) {
        const int tl = i / k, e = i == (int)threadIdx.x ? first : a.ids[t0 * k + i];
        const int r = base[e] + before[e] + bits_rank(bits + e * WORDS, tl);
        a.pos[t0 * k + i] = r;
        a.row_src[r] = (int32_t)(t0 + tl);
    }
}

// Up to a CTA for each SM no two share one: what they ask of shared memory sees to it, since behind another kernel's last
// CTAs they would (8192 tokens of 8 experts: 11.3 us sharing, 9.0 not; 131072: 84 and 95).
template <int PER, int TOK, bool BY_SCORE>
cudaError_t launch_choose_per(const RouteArgs &a, int64_t ctas, cudaStream_t st)
{
    constexpr int kAlone = 120 * 1024;
    auto kernel = route_choose_kernel<PER, TOK, BY_SCORE>;
    static OncePerDevice once;
    const cudaError_t e = allow_shared(once, kernel, kAlone);
    if (e != cudaSuccess) return e;
    const size_t smem = PER <= 2 && ctas > 1 && ctas <= num_sms() ? kAlone : (size_t)a.r.experts * (TOK / 8);
    return launch_dependent(kernel, dim3((unsigned)ctas), kThreads, smem, 0, st, a);
}

template <int TOK, bool BY_SCORE>
cudaError_t launch_choose_by(const RouteArgs &a, int64_t ctas, cudaStream_t st)
{
    const int E = a.r.experts;
    return E <= 32    ? launch_choose_per<1, TOK, BY_SCORE>(a, ctas, st)
           : E <= 64  ? launch_choose_per<2, TOK, BY_SCORE>(a, ctas, st)
           : E <= 128 ? launch_choose_per<4, TOK, BY_SCORE>(a, ctas, st)
           : E <= 256 ? launch_choose_per<8, TOK, BY_SCORE>(a, ctas, st)
                      : launch_choose_per<32, TOK, BY_SCORE>(a, ctas, st);
}

template <int TOK>
cudaError_t launch_choose(const RouteArgs &a, bool by_score, int64_t ctas, cudaStream_t st)
{
    return by_score ? launch_choose_by<TOK, true>(a, ctas, st) : launch_choose_by<TOK, false>(a, ctas, st);
}

uw_status check_router(const uw_router *r, const char *who)
{
    if (!r) return fail(UW_ERR_INVALID_ARG, "%s: NULL router", who);
    if (r->experts < 1 || r->experts > kMaxE || r->topk < 1 || r->topk > kMaxTop || r->topk > r->experts)
        return fail(UW_ERR_INVALID_ARG, "%s: %d of %d experts (1..%d of 1..%d)", who, r->topk, r->experts, kMaxTop, kMaxE);
    const int score = r->score & ~UW_SCORE_CHOOSES;
    if (score != UW_SCORE_SOFTMAX && score != UW_SCORE_SIGMOID) return fail(UW_ERR_INVALID_ARG, "%s: score %d", who, r->score);
    return UW_OK;
}

int64_t route_ctas(int64_t tokens) { return tokens <= kTokOne ? 1 : (tokens + kTokMany - 1) / kTokMany; }

// Each CTA of the order kernel reads all counts, ctas^2 experts words in all, or a scan adds them up first: 16384
// tokens of 64 experts take 16.6 us without the scan, 18.6 with it; 8192 of 256 17.9 and 16.3; 32768 of 256 73 and 47.
bool route_scans(const uw_router *r, int64_t ctas) { return ctas * r->experts >= 32768; }

size_t workspace_bytes(const uw_router *r, int64_t tokens)
{
    const int64_t ctas = route_ctas(tokens);
    return ctas == 1 ? 0 : (size_t)(ctas + route_scans(r, ctas)) * (size_t)r->experts * 4;
}

}  // namespace

extern "C" uw_status uw_route_workspace_size(const uw_router *r, int64_t tokens, size_t *bytes)
{
    clear_error();
    if (!bytes) return fail(UW_ERR_INVALID_ARG, "uw_route_workspace_size: NULL argument");
    const uw_status s = check_router(r, "uw_route_workspace_size");
    if (s != UW_OK) return s;
    if (tokens < 0 || tokens > (((int64_t)1 << 31) - 1024) / r->topk)
        return fail(UW_ERR_SHAPE, "uw_route_workspace_size: tokens=%lld", (long long)tokens);
    *bytes = workspace_bytes(r, tokens);
    return UW_OK;
}

extern "C" uw_status uw_route(const uw_router *r, const void *logits, uw_out_dtype dtype, int64_t tokens, int64_t ld, int32_t *ids,
                              float *weights, int32_t *offsets, int32_t *row_src, int32_t *pos, void *ws, size_t ws_bytes,
                              uw_stream stream)
{
    clear_error();
    const uw_status s = check_router(r, "uw_route");
    if (s != UW_OK) return s;
    if (ld == 0) ld = r->experts;
    if (tokens < 0 || tokens > (((int64_t)1 << 31) - 1024) / r->topk || ld < r->experts)
        return fail(UW_ERR_SHAPE, "uw_route: tokens=%lld ld=%lld", (long long)tokens, (long long)ld);
    if (dtype != UW_OUT_F32 && dtype != UW_OUT_BF16) return fail(UW_ERR_INVALID_ARG, "uw_route: bad dtype");
    if (!offsets || (tokens && (!logits || !ids || !weights || !row_src || !pos)))
        return fail(UW_ERR_INVALID_ARG, "uw_route: NULL argument");
    if (((uintptr_t)offsets | (uintptr_t)ids | (uintptr_t)weights | (uintptr_t)row_src | (uintptr_t)pos | (uintptr_t)r->bias) & 3 ||
        ((uintptr_t)logits & (dtype == UW_OUT_F32 ? 3 : 1)))
        return fail(UW_ERR_INVALID_ARG, "uw_route: a pointer is not aligned to its elements");
    const int64_t ctas = route_ctas(tokens);
    const size_t need = workspace_bytes(r, tokens);
    if (ws_bytes < need || (need && !ws)) return fail(UW_ERR_WORKSPACE, "uw_route: workspace %zu bytes, need %zu", ws_bytes, need);
    if ((uintptr_t)ws & 15) return fail(UW_ERR_INVALID_ARG, "uw_route: workspace not 16-byte aligned");
    RouteArgs a{*r, logits, dtype == UW_OUT_BF16, tokens, ld, ids, weights, offsets, row_src, pos, (int32_t *)ws};
    const bool by_score = r->score & UW_SCORE_CHOOSES;
    a.r.score &= ~UW_SCORE_CHOOSES;
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (tokens == 0) {
        e = cudaMemsetAsync(offsets, 0, ((size_t)r->experts + 1) * 4, st);
    } else {
        e = ctas == 1 ? launch_choose<kTokOne>(a, by_score, 1, st) : launch_choose<kTokMany>(a, by_score, ctas, st);
        const size_t smem = (size_t)r->experts * (kTokMany / 8);
        if (e == cudaSuccess && route_scans(r, ctas)) {
            e = launch_dependent(route_scan_kernel, dim3((unsigned)(r->experts + 31) / 32), kThreads, 0, 0, st, a, (int)ctas);
            if (e == cudaSuccess) e = launch_dependent(route_order_kernel<true>, dim3((unsigned)ctas), kThreads, smem, 0, st, a, (int)ctas);
        } else if (e == cudaSuccess && ctas > 1) {
            e = launch_dependent(route_order_kernel<false>, dim3((unsigned)ctas), kThreads, smem, 0, st, a, (int)ctas);
        }
    }
    return e == cudaSuccess ? UW_OK : fail(UW_ERR_CUDA, "uw_route: launch: %s", cudaGetErrorString(e));
}
