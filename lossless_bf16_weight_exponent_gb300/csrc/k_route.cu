// k_route.cu - the router of a mixture of experts: each token's top-k experts, their weights, and the order of the
// grouped products' rows (sm_103a).
//
// A warp takes a token.  A logit's sort key is its (logit + bias) mapped to an unsigned integer of the same order, above
// the complement of its index, so that the k largest 64-bit keys are the k experts in the wanted order with ties to the
// lower index; k rounds of a warp-wide maximum find them.
//
// Rows are ordered by (expert, token) without atomics on counters: a CTA of 128 tokens sets, for each expert, one bit
// per token in shared memory (a token takes an expert at most once), so a token's rank within the CTA is a population
// count and the CTA's rows per expert are another.  The second kernel adds up the counts of the CTAs before its own and
// the offsets.  Up to 128 tokens one CTA does everything in one launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "launch.cuh"
#include "uw_internal.h"

using namespace uw;

namespace {

constexpr int kTok = 128;        // tokens per CTA
constexpr int kThreads = 1024;
constexpr int kMaxE = 1024, kMaxTop = 16;

struct RouteArgs {
    uw_router r;
    const void *logits;
    int bf16;
    int64_t tokens, ld;
    int32_t *ids;
    float *weights;
    int32_t *offsets, *row_src, *pos;
    int32_t *counts;  // [CTAs][experts]
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

// the choice of token t by one warp; chosen[j] in lane j; sets the token's bits
template <int PER>  // experts per lane
__device__ __forceinline__ void choose(const RouteArgs &a, int64_t t, int lane, uint32_t (*bits)[kTok / 32], int tl)
{
    const int E = a.r.experts, k = a.r.topk;
    float z[PER];
    unsigned long long key[PER];
#pragma unroll
    for (int i = 0; i < PER; i++) {
        const int e = lane + 32 * i;
        z[i] = e < E ? logit_at(a, t, e) : -INFINITY;
        const float s = e < E && a.r.bias ? z[i] + __ldg(a.r.bias + e) : z[i];
        key[i] = e < E ? ((unsigned long long)order_key(s) << 32) | (uint32_t)~e : 0ull;
    }
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
    int my_e = 0;
    float my_z = 0.f;
    for (int j = 0; j < k; j++) {
        unsigned long long best = 0ull;
#pragma unroll
        for (int i = 0; i < PER; i++) best = key[i] > best ? key[i] : best;
        unsigned long long all = best;
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const unsigned long long o = __shfl_xor_sync(0xFFFFFFFFu, all, d);
            all = o > all ? o : all;
        }
        const int e = (int)~(uint32_t)all;
        float ze = 0.f;
#pragma unroll
        for (int i = 0; i < PER; i++)
            if (key[i] == all) {
                ze = z[i];
                key[i] = 0ull;
            }
        ze = __shfl_sync(0xFFFFFFFFu, ze, e & 31);
        if (lane == j) {
            my_e = e;
            my_z = ze;
        }
    }
    float w = 0.f;
    if (lane < k) {
        if (a.r.score == UW_SCORE_SOFTMAX) w = total == 0.f ? 0.f : expf(my_z - m) / total;
        else w = 1.f / (1.f + expf(-my_z));
    }
    if (a.r.renormalize) {
        float s = w;
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
        w = s == 0.f ? 0.f : w / s;
    }
    if (lane < k) {
        a.ids[t * k + lane] = my_e;
        a.weights[t * k + lane] = w * a.r.scale;
        atomicOr(&bits[my_e][tl >> 5], 1u << (tl & 31));
    }
}

__device__ __forceinline__ void choose_any(const RouteArgs &a, int64_t t, int lane, uint32_t (*bits)[kTok / 32], int tl)
{
    const int E = a.r.experts;
    if (E <= 32) choose<1>(a, t, lane, bits, tl);
    else if (E <= 64) choose<2>(a, t, lane, bits, tl);
    else if (E <= 128) choose<4>(a, t, lane, bits, tl);
    else if (E <= 256) choose<8>(a, t, lane, bits, tl);
    else choose<32>(a, t, lane, bits, tl);
}

__device__ __forceinline__ int bits_count(const uint32_t *b)
{
    int n = 0;
#pragma unroll
    for (int i = 0; i < kTok / 32; i++) n += __popc(b[i]);
    return n;
}

// rank of token tl among the CTA's tokens that took the expert
__device__ __forceinline__ int bits_rank(const uint32_t *b, int tl)
{
    int n = __popc(b[tl >> 5] & ((1u << (tl & 31)) - 1u));
    for (int i = 0; i < (tl >> 5); i++) n += __popc(b[i]);
    return n;
}

// exclusive scan of v over the CTA's 1024 threads; returns the total
__device__ __forceinline__ int block_scan(int &v, int *wsum)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, s, d);
        if (lane >= d) s += o;
    }
    if (lane == 31) wsum[warp] = s;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < kThreads / 32; w++) {
        if (w < warp) before += wsum[w];
        all += wsum[w];
    }
    v = before + s - v;
    return all;
}

__global__ void __launch_bounds__(kThreads) route_choose_kernel(const RouteArgs a)
{
    __shared__ uint32_t bits[kMaxE][kTok / 32];
    const int E = a.r.experts, k = a.r.topk;
    const int64_t t0 = (int64_t)blockIdx.x * kTok;
    const int nt = (int)min((int64_t)kTok, a.tokens - t0);
    for (int i = threadIdx.x; i < E * (kTok / 32); i += kThreads) (&bits[0][0])[i] = 0u;
    pdl_trigger();
    pdl_wait();
    __syncthreads();
    for (int tl = threadIdx.x >> 5; tl < nt; tl += kThreads / 32) choose_any(a, t0 + tl, threadIdx.x & 31, bits, tl);
    __syncthreads();
    if (gridDim.x > 1) {
        if ((int)threadIdx.x < E) a.counts[(int64_t)blockIdx.x * E + threadIdx.x] = bits_count(bits[threadIdx.x]);
        return;
    }
    // all tokens are here: the order too
    __shared__ int wsum[kThreads / 32], base[kMaxE];
    int v = (int)threadIdx.x < E ? bits_count(bits[threadIdx.x]) : 0;
    const int total = block_scan(v, wsum);
    if ((int)threadIdx.x < E) {
        base[threadIdx.x] = v;
        a.offsets[threadIdx.x] = v;
    }
    if (threadIdx.x == 0) a.offsets[E] = total;
    __syncthreads();
    for (int i = threadIdx.x; i < nt * k; i += kThreads) {
        const int tl = i / k, e = a.ids[i];
        const int r = base[e] + bits_rank(bits[e], tl);
        a.pos[i] = r;
        a.row_src[r] = tl;
    }
}

__global__ void __launch_bounds__(kThreads) route_order_kernel(const RouteArgs a, int ctas)
{
    __shared__ uint32_t bits[kMaxE][kTok / 32];
    __shared__ int wsum[kThreads / 32], base[kMaxE];
    const int E = a.r.experts, k = a.r.topk;
    const int64_t t0 = (int64_t)blockIdx.x * kTok;
    const int nt = (int)min((int64_t)kTok, a.tokens - t0);
    for (int i = threadIdx.x; i < E * (kTok / 32); i += kThreads) (&bits[0][0])[i] = 0u;
    pdl_trigger();
    pdl_wait();
    // rows of each expert in all CTAs, and in those before this one
    int all = 0, before = 0;
    if ((int)threadIdx.x < E)
        for (int c = 0; c < ctas; c++) {
            const int n = __ldg(a.counts + (int64_t)c * E + threadIdx.x);
            all += n;
            if (c < (int)blockIdx.x) before += n;
        }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * k; i += kThreads) {
        const int tl = i / k;
        atomicOr(&bits[a.ids[t0 * k + i]][tl >> 5], 1u << (tl & 31));
    }
    int v = all;
    const int total = block_scan(v, wsum);
    if ((int)threadIdx.x < E) {
        base[threadIdx.x] = v + before;
        if (blockIdx.x == 0) a.offsets[threadIdx.x] = v;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[E] = total;
    __syncthreads();
    for (int i = threadIdx.x; i < nt * k; i += kThreads) {
        const int tl = i / k, e = a.ids[t0 * k + i];
        const int r = base[e] + bits_rank(bits[e], tl);
        a.pos[t0 * k + i] = r;
        a.row_src[r] = (int32_t)(t0 + tl);
    }
}

uw_status check_router(const uw_router *r, const char *who)
{
    if (!r) return fail(UW_ERR_INVALID_ARG, "%s: NULL router", who);
    if (r->experts < 1 || r->experts > kMaxE || r->topk < 1 || r->topk > kMaxTop || r->topk > r->experts)
        return fail(UW_ERR_INVALID_ARG, "%s: %d of %d experts (1..%d of 1..%d)", who, r->topk, r->experts, kMaxTop, kMaxE);
    if (r->score != UW_SCORE_SOFTMAX && r->score != UW_SCORE_SIGMOID) return fail(UW_ERR_INVALID_ARG, "%s: score %d", who, r->score);
    return UW_OK;
}

int64_t route_ctas(int64_t tokens) { return (tokens + kTok - 1) / kTok; }

}  // namespace

extern "C" uw_status uw_route_workspace_size(const uw_router *r, int64_t tokens, size_t *bytes)
{
    clear_error();
    if (!bytes) return fail(UW_ERR_INVALID_ARG, "uw_route_workspace_size: NULL argument");
    const uw_status s = check_router(r, "uw_route_workspace_size");
    if (s != UW_OK) return s;
    if (tokens < 0 || tokens > (((int64_t)1 << 31) - 1024) / r->topk)
        return fail(UW_ERR_SHAPE, "uw_route_workspace_size: tokens=%lld", (long long)tokens);
    *bytes = tokens <= kTok ? 0 : (size_t)route_ctas(tokens) * (size_t)r->experts * 4;
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
    const size_t need = tokens <= kTok ? 0 : (size_t)ctas * (size_t)r->experts * 4;
    if (ws_bytes < need || (need && !ws)) return fail(UW_ERR_WORKSPACE, "uw_route: workspace %zu bytes, need %zu", ws_bytes, need);
    if ((uintptr_t)ws & 15) return fail(UW_ERR_INVALID_ARG, "uw_route: workspace not 16-byte aligned");
    const RouteArgs a{*r, logits, dtype == UW_OUT_BF16, tokens, ld, ids, weights, offsets, row_src, pos, (int32_t *)ws};
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e;
    if (tokens == 0) {
        e = cudaMemsetAsync(offsets, 0, ((size_t)r->experts + 1) * 4, st);
    } else {
        e = launch_dependent(route_choose_kernel, dim3((unsigned)ctas), kThreads, 0, 0, st, a);
        if (e == cudaSuccess && ctas > 1) e = launch_dependent(route_order_kernel, dim3((unsigned)ctas), kThreads, 0, 0, st, a, (int)ctas);
    }
    return e == cudaSuccess ? UW_OK : fail(UW_ERR_CUDA, "uw_route: launch: %s", cudaGetErrorString(e));
}
