// k_group.cu - groups of compressed expert matrices: their form, made on the device, and the entry points.
//
// Making a group reads each matrix twice: once for the histogram of its exponents (from which the 16 consecutive
// exponents that cover the most weights are chosen) and the masks of the runs that hold another exponent, once to
// pack it.  In between a scan numbers the verbatim runs, whose count sizes the group's memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <new>
#include <vector>

#include "group.cuh"
#include "uw_internal.h"

using namespace uw;

struct uw_group {
    GroupView v{};
    uint64_t n_verb = 0, bytes = 0;
    void *dev = nullptr;   // steps with their records, bases, status
    void *verb = nullptr;  // verbatim runs
    int device = 0;
};

namespace {

using namespace dev;

// one matrix's place among the virtual granules: its granule i is virtual granule i * stride + first
struct MatPlace {
    const uint16_t *w;  // [N, K] bf16
    int64_t N, K;
    int tiles, ksteps, stride, first;
    uint8_t *steps;     // the expert's steps
    uint8_t *verb;
    uint32_t *base;     // the matrix's entry
};

__global__ void __launch_bounds__(256) histogram_kernel(const uint16_t *w, uint64_t n8, unsigned long long *hist)
{
    __shared__ uint32_t h[256];
    h[threadIdx.x] = 0;
    __syncthreads();
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < n8; i += gridDim.x * 256ull) {
        const uint4 v = __ldg((const uint4 *)w + i);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            atomicAdd(&h[(word_of(v, j) >> 7) & 255u], 1u);
            atomicAdd(&h[(word_of(v, j) >> 23) & 255u], 1u);
        }
    }
    __syncthreads();
    if (h[threadIdx.x]) atomicAdd(hist + threadIdx.x, (unsigned long long)h[threadIdx.x]);
}

// the first of the 16 consecutive exponents that cover the most weights (the lowest of equals)
__global__ void __launch_bounds__(256) base_kernel(const unsigned long long *hist, uint32_t *base)
{
    __shared__ unsigned long long cover[256];
    unsigned long long s = 0;
    if (threadIdx.x <= 240)
        for (int i = 0; i < 16; i++) s += hist[threadIdx.x + i];
    cover[threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        uint32_t b = 0;
        for (uint32_t i = 1; i <= 240; i++)
            if (cover[i] > cover[b]) b = i;
        *base = (b << 7) | (b << 23);
    }
}

// rows' runs with an exponent outside the 16: one warp per (granule, step), two lanes per row
__global__ void __launch_bounds__(256) mask_kernel(MatPlace m, int64_t warps)
{
    const int64_t wi = (blockIdx.x * 256ll + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (wi >= warps) return;
    const int64_t gr = wi / m.ksteps;
    const int ks = (int)(wi % m.ksteps);
    const int64_t row = gr * kGran + (lane >> 1);
    const uint32_t b0 = (*m.base >> 7) & 255u;
    bool out = false;
    if (row < m.N) {
        const uint4 *p = (const uint4 *)(m.w + row * m.K + (int64_t)ks * kStepW + 32 * (lane & 1));
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint4 v = __ldg(p + i);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint32_t x = word_of(v, j);
                out |= ((x >> 7) & 255u) - b0 > 15u || ((x >> 23) & 255u) - b0 > 15u;
            }
        }
    }
    uint32_t bal = __ballot_sync(0xFFFFFFFFu, out);
    bal = (bal | (bal >> 1)) & 0x55555555u;  // bit 2r: row r
    uint32_t bits = 0;
#pragma unroll
    for (int r = 0; r < 16; r++) bits |= ((bal >> (2 * r)) & 1u) << r;
    if (lane == 0) {
        const int64_t vg = gr * m.stride + m.first;
        ((uint16_t *)((StepRec *)step_rec(m.steps, (vg / 8) * m.ksteps + ks))->mask)[vg % 8] = (uint16_t)bits;
    }
}

// numbers the verbatim runs: one CTA, an exclusive scan over all records; total in *total
__global__ void __launch_bounds__(1024) scan_kernel(uint8_t *steps, int64_t n, unsigned long long *total)
{
    __shared__ uint32_t wsum[32];
    unsigned long long carry = 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t i0 = 0; i0 < n; i0 += 1024) {
        const int64_t i = i0 + threadIdx.x;
        StepRec *rec = (StepRec *)step_rec(steps, i);
        uint32_t c = 0;
        if (i < n) c = __popc(rec->mask[0]) + __popc(rec->mask[1]) + __popc(rec->mask[2]) + __popc(rec->mask[3]);
        uint32_t s = c;
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t o = __shfl_up_sync(0xFFFFFFFFu, s, d);
            if (lane >= d) s += o;
        }
        if (lane == 31) wsum[warp] = s;
        __syncthreads();
        uint32_t before = 0, all = 0;
        for (int w = 0; w < 32; w++) {
            if (w < warp) before += wsum[w];
            all += wsum[w];
        }
        if (i < n) {
            rec->first = (uint32_t)(carry + before + s - c);
            rec->count = c;
        }
        carry += all;
        __syncthreads();
    }
    if (threadIdx.x == 0) *total = carry;
}

// one warp per (granule, step), lane 4 g + t chunk t of rows g and g + 8
__global__ void __launch_bounds__(256) pack_kernel(MatPlace m, int64_t warps)
{
    const int64_t wi = (blockIdx.x * 256ll + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (wi >= warps) return;
    const int64_t gr = wi / m.ksteps;
    const int ks = (int)(wi % m.ksteps);
    const int64_t vg = gr * m.stride + m.first;
    const int64_t step = (vg / 8) * m.ksteps + ks;
    const int gi = (int)(vg % 8);
    const StepRec &rec = *step_rec(m.steps, step);
    const uint32_t b0 = (*m.base >> 7) & 255u;
    uint8_t *st = m.steps + step * kStepBytes;
    uint32_t codes[4];
#pragma unroll
    for (int half = 0; half < 2; half++) {
        const int rg = 8 * half + g;
        const int64_t row = gr * kGran + rg;
        uint32_t P[8], D[8], E[4] = {0, 0, 0, 0};
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (row < m.N) {
            const uint4 *p = (const uint4 *)(m.w + row * m.K + (int64_t)ks * kStepW + 16 * t);
            a = __ldg(p);
            b = __ldg(p + 1);
        }
        const int rt = 16 * gi + rg;
        const bool verb = (rec.mask[rt >> 5] >> (rt & 31)) & 1u;
#pragma unroll
        for (int q = 0; q < 8; q++) {
            const uint32_t x = q < 4 ? word_of(a, q) : word_of(b, q - 4);
            const uint32_t e0 = (x >> 7) & 255u, e1 = (x >> 23) & 255u;
            P[q] = x & 0x807F807Fu;
            // rows past the matrix hold zeros that a distance cannot name; their products are never stored
            D[q] = verb || row >= m.N ? 0u : ((e0 - b0) << 7) | ((e1 - b0) << 23);
            E[q >> 1] |= (e0 | (e1 << 8)) << (16 * (q & 1));
        }
        uint32_t s[4];
#pragma unroll
        for (int j = 0; j < 4; j++) s[j] = P[2 * j] | prmt(P[2 * j + 1], 0u, 0x2301u);
        *(uint4 *)(st + gi * 1024 + half * 512 + chunk_at(g, t)) = make_uint4(s[0], s[1], s[2], s[3]);
#pragma unroll
        for (int i = 0; i < 2; i++)
            codes[2 * half + i] = D[4 * i] | (D[4 * i + 1] << 4) | (D[4 * i + 2] >> 4) | __funnelshift_r(D[4 * i + 3], D[4 * i + 3], 8);
        if (verb)
            *(uint4 *)(m.verb + ((uint64_t)rec.first + verbatim_rank(rec.mask, rt)) * 64 + 16 * t) = make_uint4(E[0], E[1], E[2], E[3]);
    }
    *(uint4 *)(st + kStepSm + gi * 512 + chunk_at(g, t)) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
}

// the inverse of pack_kernel
__global__ void __launch_bounds__(256) unpack_kernel(MatPlace m, uint16_t *out, int64_t warps)
{
    const int64_t wi = (blockIdx.x * 256ll + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (wi >= warps) return;
    const int64_t gr = wi / m.ksteps;
    const int ks = (int)(wi % m.ksteps);
    const int64_t vg = gr * m.stride + m.first;
    const int64_t step = (vg / 8) * m.ksteps + ks;
    const int gi = (int)(vg % 8);
    const StepRec &rec = *step_rec(m.steps, step);
    const uint8_t *st = m.steps + step * kStepBytes;
    const uint4 codes = *(const uint4 *)(st + kStepSm + gi * 512 + chunk_at(g, t));
#pragma unroll
    for (int half = 0; half < 2; half++) {
        const int rg = 8 * half + g;
        const int64_t row = gr * kGran + rg;
        if (row >= m.N) continue;
        const int rt = 16 * gi + rg;
        const uint4 S = *(const uint4 *)(st + gi * 1024 + half * 512 + chunk_at(g, t));
        uint32_t p[8];
        if ((rec.mask[rt >> 5] >> (rt & 31)) & 1u)
            rebuild_chunk_verbatim(S, *(const uint4 *)(m.verb + ((uint64_t)rec.first + verbatim_rank(rec.mask, rt)) * 64 + 16 * t), p);
        else
            rebuild_chunk(S, half ? make_uint2(codes.z, codes.w) : make_uint2(codes.x, codes.y), *m.base, p);
        uint4 *o = (uint4 *)(out + row * m.K + (int64_t)ks * kStepW + 16 * t);
        o[0] = make_uint4(p[0], p[1], p[2], p[3]);
        o[1] = make_uint4(p[4], p[5], p[6], p[7]);
    }
}

uw_status cuda_fail(cudaError_t e, const char *what) { return fail(UW_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e)); }

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// memory that cannot be had leaves no error behind for the next launch's check
template <typename T>
cudaError_t device_alloc(T **p, uint64_t bytes)
{
    const cudaError_t e = cudaMalloc(p, bytes);
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

MatPlace place_of(const uw_group *g, int expert, int up)
{
    const GroupView &v = g->v;
    MatPlace m{};
    m.N = v.N;
    m.K = v.K;
    m.tiles = v.tiles;
    m.ksteps = v.ksteps;
    m.stride = v.gated ? 2 : 1;
    m.first = up;
    const int64_t s0 = (int64_t)expert * v.tiles * v.ksteps;
    m.steps = const_cast<uint8_t *>(v.steps) + s0 * kStepBytes;
    m.verb = const_cast<uint8_t *>(v.verb);
    m.base = const_cast<uint32_t *>(v.base) + (int64_t)expert * m.stride + up;
    return m;
}

// a group's memory is its device's, and so is the stream of a call on it
uw_status check_device(const uw_group *g, const char *who)
{
    int device = 0;
    const cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return cuda_fail(e, who);
    return device == g->device ? UW_OK : fail(UW_ERR_INVALID_ARG, "%s: the group is on device %d, the current one is %d", who, g->device, device);
}

int64_t place_warps(const MatPlace &m) { return (m.N + kGran - 1) / kGran * m.ksteps; }
unsigned place_blocks(const MatPlace &m) { return (unsigned)((place_warps(m) + 7) / 8); }

// Source of the group's dense matrices: device memory, or loaded matrices decoded one at a time into a buffer.
struct Source {
    const uint16_t *dense[2];
    const uw_matrix *const *mats[2];
    uint16_t *buf;
    uw_status get(int expert, int up, int64_t N, int64_t K, uw_stream st, const uint16_t **out) const
    {
        if (dense[up]) {
            *out = dense[up] + (uint64_t)expert * (uint64_t)N * (uint64_t)K;
            return UW_OK;
        }
        *out = buf;
        return uw_decode(mats[up][expert], buf, st);
    }
};

uw_status make_group(const Source &src, int experts, bool gated, int64_t N, int64_t K, uw_stream stream, uw_group **out)
{
    cudaStream_t st = (cudaStream_t)stream;
    uw_group *g = new (std::nothrow) uw_group();
    if (!g) return fail(UW_ERR_NO_MEMORY, "uw_group_create: host allocation");
    GroupView &v = g->v;
    const int mats = gated ? 2 : 1;
    v.N = N;
    v.K = K;
    v.experts = experts;
    v.gated = gated;
    v.granules = (int)((N + kGran - 1) / kGran * mats);
    v.tiles = (v.granules + 7) / 8;
    v.ksteps = (int)(K / kStepW);
    const uint64_t n_steps = (uint64_t)experts * (uint64_t)v.tiles * (uint64_t)v.ksteps;
    const uint64_t o_base = n_steps * kStepBytes, o_hist = o_base + (uint64_t)experts * 8 + 256;
    const uint64_t o_total = (o_hist + 2048 + 255) / 256 * 256, o_status = o_total + 256, bytes = o_status + 256;
    cudaGetDevice(&g->device);
    uw_status s = UW_OK;
    auto check = [&](cudaError_t e, const char *what) {
        if (e != cudaSuccess && s == UW_OK)
            s = e == cudaErrorMemoryAllocation ? fail(UW_ERR_NO_MEMORY, "uw_group_create: %s: %s", what, cudaGetErrorString(e))
                                               : cuda_fail(e, what);
        return s == UW_OK;
    };
    auto done = [&](uw_status code) {
        if (code != UW_OK) {
            cudaStreamSynchronize(st);
            uw_group_free(g);
        }
        return code;
    };
    if (!check(device_alloc(&g->dev, bytes), "memory of the steps")) return done(s);
    uint8_t *d = (uint8_t *)g->dev;
    unsigned long long *hist = (unsigned long long *)(d + o_hist), *total = (unsigned long long *)(d + o_total);
    v.steps = d;
    v.base = (const uint32_t *)(d + o_base);
    v.status = (int *)(d + o_status);
    // padding granules keep zeros
    if (!check(cudaMemsetAsync(d, 0, bytes, st), "memset")) return done(s);
    for (int e = 0; e < experts; e++)
        for (int u = 0; u < mats; u++) {
            MatPlace m = place_of(g, e, u);
            if ((s = src.get(e, u, N, K, stream, &m.w)) != UW_OK) return done(s);
            if (!check(cudaMemsetAsync(hist, 0, 2048, st), "memset")) return done(s);
            const uint64_t n8 = (uint64_t)N * (uint64_t)K / 8;
            histogram_kernel<<<(unsigned)std::min<uint64_t>((n8 + 255) / 256, 8ull * num_sms()), 256, 0, st>>>(m.w, n8, hist);
            base_kernel<<<1, 256, 0, st>>>(hist, m.base);
            mask_kernel<<<place_blocks(m), 256, 0, st>>>(m, place_warps(m));
            if (!check(cudaGetLastError(), "uw_group_create: launch")) return done(s);
        }
    scan_kernel<<<1, 1024, 0, st>>>(d, (int64_t)n_steps, total);
    unsigned long long n_verb = 0;
    if (!check(cudaGetLastError(), "uw_group_create: launch") ||
        !check(cudaMemcpyAsync(&n_verb, total, 8, cudaMemcpyDeviceToHost, st), "uw_group_create: count") ||
        !check(cudaStreamSynchronize(st), "uw_group_create: synchronize"))
        return done(s);
    if (n_verb >= (1ull << 32)) return done(fail(UW_ERR_SHAPE, "uw_group_create: %llu verbatim runs", n_verb));
    g->n_verb = n_verb;
    if (!check(device_alloc(&g->verb, n_verb * 64 + 256), "memory of the verbatim runs")) return done(s);
    v.verb = (const uint8_t *)g->verb;
    g->bytes = bytes + n_verb * 64 + 256;
    for (int e = 0; e < experts; e++)
        for (int u = 0; u < mats; u++) {
            MatPlace m = place_of(g, e, u);
            if ((s = src.get(e, u, N, K, stream, &m.w)) != UW_OK) return done(s);
            pack_kernel<<<place_blocks(m), 256, 0, st>>>(m, place_warps(m));
            if (!check(cudaGetLastError(), "uw_group_create: launch")) return done(s);
        }
    if (!check(cudaStreamSynchronize(st), "uw_group_create: synchronize")) return done(s);
    *out = g;
    return UW_OK;
}

uw_status check_shape(int experts, int64_t N, int64_t K)
{
    if (experts < 1 || experts > kMaxExperts)
        return fail(UW_ERR_INVALID_ARG, "uw_group_create: %d experts (1..%d)", experts, kMaxExperts);
    const int64_t most = ((int64_t)1 << 31) - 256;
    if (N < 1 || K < 1 || K % kStepW || N > most || K > most)
        return fail(UW_ERR_SHAPE, "uw_group_create: N=%lld K=%lld (K a multiple of 64)", (long long)N, (long long)K);
    // a matrix is walked by one launch of a warp per granule and step
    if ((N + kGran - 1) / kGran * (K / kStepW) > ((int64_t)1 << 33))
        return fail(UW_ERR_SHAPE, "uw_group_create: N=%lld K=%lld is too large", (long long)N, (long long)K);
    return UW_OK;
}

}  // namespace

extern "C" uw_status uw_group_create_dense(const uint16_t *w, const uint16_t *w_up, int experts, int64_t N, int64_t K,
                                           uw_stream stream, uw_group **out)
{
    clear_error();
    if (!out) return fail(UW_ERR_INVALID_ARG, "uw_group_create: out is NULL");
    *out = nullptr;
    uw_status s = check_shape(experts, N, K);
    if (s != UW_OK) return s;
    if (!w || !aligned16(w) || !aligned16(w_up)) return fail(UW_ERR_INVALID_ARG, "uw_group_create: weights NULL or not 16-byte aligned");
    Source src{{w, w_up}, {nullptr, nullptr}, nullptr};
    return make_group(src, experts, w_up != nullptr, N, K, stream, out);
}

extern "C" uw_status uw_group_create(const uw_matrix *const *w, const uw_matrix *const *w_up, int experts, uw_stream stream,
                                     uw_group **out)
{
    clear_error();
    if (!out) return fail(UW_ERR_INVALID_ARG, "uw_group_create: out is NULL");
    *out = nullptr;
    if (!w || experts < 1 || experts > kMaxExperts)
        return fail(UW_ERR_INVALID_ARG, "uw_group_create: %s", w ? "experts outside 1..1024" : "NULL matrices");
    int device = 0;
    cudaGetDevice(&device);
    for (int u = 0; u < (w_up ? 2 : 1); u++)
        for (int e = 0; e < experts; e++) {
            const uw_matrix *m = (u ? w_up : w)[e];
            if (!m) return fail(UW_ERR_INVALID_ARG, "uw_group_create: matrix %d is NULL", e);
            if (m->device != device) return fail(UW_ERR_INVALID_ARG, "uw_group_create: matrix %d is on device %d, not %d", e, m->device, device);
            if (!w[0] || m->h.N != w[0]->h.N || m->h.K != w[0]->h.K)
                return fail(UW_ERR_SHAPE, "uw_group_create: matrix %d is [%lld, %lld]", e, (long long)m->h.N, (long long)m->h.K);
        }
    const int64_t N = w[0]->h.N, K = w[0]->h.K;
    uw_status s = check_shape(experts, N, K);
    if (s != UW_OK) return s;
    uint16_t *buf = nullptr;
    const cudaError_t e = device_alloc(&buf, (uint64_t)N * (uint64_t)K * 2);
    if (e != cudaSuccess) return fail(UW_ERR_NO_MEMORY, "uw_group_create: decode buffer: %s", cudaGetErrorString(e));
    Source src{{nullptr, nullptr}, {w, w_up}, buf};
    s = make_group(src, experts, w_up != nullptr, N, K, stream, out);
    // a corrupt stream is latched in its matrix
    for (int u = 0; u < (w_up ? 2 : 1) && s == UW_OK; u++)
        for (int i = 0; i < experts && s == UW_OK; i++) s = uw_check((u ? w_up : w)[i], stream);
    if (s != UW_OK && *out) {
        uw_group_free(*out);
        *out = nullptr;
    }
    cudaFree(buf);
    return s;
}

extern "C" void uw_group_free(uw_group *g)
{
    if (!g) return;
    cudaFree(g->verb);
    cudaFree(g->dev);
    delete g;
}

extern "C" uw_status uw_group_get_info(const uw_group *g, uw_group_info *out)
{
    clear_error();
    if (!g || !out) return fail(UW_ERR_INVALID_ARG, "uw_group_get_info: NULL argument");
    memset(out, 0, sizeof *out);
    out->N = g->v.N;
    out->K = g->v.K;
    out->experts = g->v.experts;
    out->gated = g->v.gated;
    out->n_verbatim = g->n_verb;
    out->device_bytes = g->bytes;
    return UW_OK;
}

extern "C" uw_status uw_group_decode(const uw_group *g, int expert, int up, uint16_t *w_dev, uw_stream stream)
{
    clear_error();
    if (!g || !w_dev || !aligned16(w_dev)) return fail(UW_ERR_INVALID_ARG, "uw_group_decode: NULL argument or output not 16-byte aligned");
    if (expert < 0 || expert >= g->v.experts) return fail(UW_ERR_INVALID_ARG, "uw_group_decode: expert %d of %d", expert, g->v.experts);
    if (up && !g->v.gated) return fail(UW_ERR_UNSUPPORTED, "uw_group_decode: the group has no up matrices");
    const uw_status s = check_device(g, "uw_group_decode");
    if (s != UW_OK) return s;
    const MatPlace m = place_of(g, expert, up ? 1 : 0);
    unpack_kernel<<<place_blocks(m), 256, 0, (cudaStream_t)stream>>>(m, w_dev, place_warps(m));
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? UW_OK : cuda_fail(e, "uw_group_decode: launch");
}

extern "C" uw_status uw_group_check(const uw_group *g, uw_stream stream)
{
    clear_error();
    if (!g) return fail(UW_ERR_INVALID_ARG, "uw_group_check: NULL group");
    cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
    if (e != cudaSuccess) return cuda_fail(e, "uw_group_check: synchronize");
    int s = 0;
    if ((e = cudaMemcpy(&s, g->v.status, sizeof s, cudaMemcpyDeviceToHost)) != cudaSuccess) return cuda_fail(e, "uw_group_check: status read");
    if (s) {
        if ((e = cudaMemset(g->v.status, 0, sizeof s)) != cudaSuccess) return cuda_fail(e, "uw_group_check: status clear");
        return fail(UW_ERR_TIMEOUT, "a bounded device wait expired");
    }
    return UW_OK;
}

extern "C" uw_status uw_group_matmul(const uw_group *g, const uint16_t *x, int64_t x_rows, int64_t ldx, const int32_t *row_src,
                                     const int32_t *offsets, int64_t rows, void *y, int64_t ldy, uw_out_dtype od,
                                     uw_stream stream)
{
    clear_error();
    if (!g) return fail(UW_ERR_INVALID_ARG, "uw_group_matmul: NULL group");
    const int64_t most = ((int64_t)1 << 31) - 1024;
    if (ldx == 0) ldx = g->v.K;
    if (ldy == 0) ldy = g->v.N;
    if (rows < 0 || x_rows < 0 || rows > most || x_rows > most || ldx < g->v.K || ldx % 8 || ldy < g->v.N)
        return fail(UW_ERR_SHAPE, "uw_group_matmul: rows=%lld x_rows=%lld ldx=%lld ldy=%lld (N=%lld K=%lld)", (long long)rows,
                    (long long)x_rows, (long long)ldx, (long long)ldy, (long long)g->v.N, (long long)g->v.K);
    if (od != UW_OUT_F32 && od != UW_OUT_BF16) return fail(UW_ERR_INVALID_ARG, "uw_group_matmul: bad output dtype");
    if (rows == 0) return UW_OK;
    if (!offsets || !y || !aligned16(y) || (x_rows && !x) || !aligned16(x))
        return fail(UW_ERR_INVALID_ARG, "uw_group_matmul: NULL argument, or x or y not 16-byte aligned");
    if (((uintptr_t)offsets | (uintptr_t)row_src) & 3)
        return fail(UW_ERR_INVALID_ARG, "uw_group_matmul: offsets or row_src not 4-byte aligned");
    const uw_status s = check_device(g, "uw_group_matmul");
    if (s != UW_OK) return s;
    GroupCall c{};
    c.v = g->v;
    c.x = x;
    c.x_rows = x_rows;
    c.ldx = ldx;
    c.row_src = row_src;
    c.offsets = offsets;
    c.rows = rows;
    c.y = y;
    c.ldy = ldy;
    c.out_bf16 = od == UW_OUT_BF16;
    // Few rows an expert on average take the matrix-vector kernel, which reads the weights of an expert again for every eight of
    // its rows, else tcgen05: up to two rows for a bf16 output, and four for an fp32 one, whose segments cost tcgen05 more.
    // Matrix-vector against tcgen05 in us (tokens' own choices, weights from memory):
    //   rows each                             2              3              4              6
    //   64 of [2048, 1408]         bf16   49.6   51.4    57.2   52.8    63.0   58.1    74.8   58.6
    //                              fp32   49.7   55.2    57.1   56.5    63.2   62.5    74.5   63.0
    //   64 gated of [1408, 2048]   bf16   86.9   88.1    94.9   97.2   105.3   98.3   127.7   98.4
    //                              fp32   87.2   94.4    94.7  103.9   105.5  105.1   127.9  105.0
    //   8 gated of [14336, 4096]   bf16  234.3  231.3   208.3  212.5   234.6  231.5   262.0  212.6
    //                              fp32  245.8  247.5   217.9  227.5   246.3  247.6   274.7  227.8
    //   8 of [4096, 14336]         bf16  128.8  136.1   135.7  137.4   136.0  137.1   141.9  137.2
    //                              fp32  130.4  145.9   137.7  146.0   138.4  146.0   144.0  146.2
    const bool tc = rows > (c.out_bf16 ? 2 : 4) * (int64_t)g->v.experts && group_tc_supported(c);
    const cudaError_t e = (cudaError_t)(tc ? launch_group_tc(c, stream) : launch_group_gemv(c, stream));
    return e == cudaSuccess ? UW_OK : cuda_fail(e, "uw_group_matmul: launch");
}
