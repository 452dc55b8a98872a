// k_kv.cu - a cache of keys and values in pages: its handle, the frequencies of the rotation, and the append of new tokens
// with the rotation of their queries and keys on the way (sm_103a).
//
// A token's row is cut into items of 16 elements of one head: two chunks of eight (16 bytes of bf16) that are turned
// against each other - i and i + dim / 2 of the halves' layout - or that lie side by side.  A thread asks for its items'
// elements first; meanwhile the CTA's first warp finds the token's sequence among `starts` (32 at a time: two steps
// for 1024 sequences) and its slot, and the first dim / 2 threads turn the position into cos and sin for all heads.
// The angle is position * freq in turns: in 64 bits the product is exact to 1e-10 of a turn at position 2^20, its fraction goes
// into sincospi in fp32, so a far position costs no accuracy (the product in fp32 is off by 0.06 radians there).
// 4096 tokens of 32 query and 8 key heads of 128, bf16, take 20.4 us as ordinary calls (4.9 TB/s) and 17.0 in a captured chain on the same
// tensors, a part of which stays in L2 (20.1 there with the angles in their order in shared memory, where lanes of neighbouring items met in
// the same banks).  Memory does not bound it: a CTA's threads wait at the barrier for the look-ups and for 64 angles in 64 bits, which this
// GPU computes slowly (ncu: barrier first among the stalls, DRAM at 35 %).  253 tokens of 64 and 8 heads take 6.0 us in a chain, one token 2.6,
// the launch and three loads that depend on each other.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "kv.cuh"
#include "launch.cuh"
#include "uw_internal.h"

using namespace uw;

namespace {

struct AppendArgs {
    KvBatch b;
    uw_kv_desc c;
    const void *q, *k, *v;
    int64_t ldq, ldk, ldv, ldq_out;
    const int32_t *positions;
    uint16_t *q_out;
    const double *freq;
    float scale;
    int rot, interleaved;       // elements of a head that are turned (0: none)
    int q_heads, heads;         // heads: all of q, k and v
};

// 16 elements as loaded: two chunks of eight
template <bool F32>
struct Item {
    uint4 a[F32 ? 4 : 2];
};

template <bool F32>
__device__ __forceinline__ void load_chunk(const void *p, int64_t at, uint4 *a)
{
    const uint4 *q = (const uint4 *)((const uint8_t *)p + at * (F32 ? 4 : 2));
    a[0] = q[0];
    if constexpr (F32) a[1] = q[1];
}

template <bool F32>
__device__ __forceinline__ void unpack_chunk(const uint4 *a, float (&f)[8])
{
    const uint32_t w[4] = {a[0].x, a[0].y, a[0].z, a[0].w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if constexpr (F32) {
            f[i] = __uint_as_float(w[i]);
        } else {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    if constexpr (F32) {
        f[4] = __uint_as_float(a[1].x);
        f[5] = __uint_as_float(a[1].y);
        f[6] = __uint_as_float(a[1].z);
        f[7] = __uint_as_float(a[1].w);
    }
}

__device__ __forceinline__ uint4 pack_chunk(const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *(const uint32_t *)&v;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The sequence of row t, by a whole warp: the last s with starts[s] <= t (that one has the row, if any has).  -1: none.
__device__ __forceinline__ int seq_of_row(const KvBatch &b, int t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, n = b.sequences + 1;  // the last index in [lo, lo + n) with starts <= t
    while (n > 1) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const bool le = lane * step < n && min(max(b.starts[at], 0), b.rows) <= t;
        const unsigned m = __ballot_sync(0xFFFFFFFFu, le);
        if (!(m & 1u)) return -1;
        const int last = 31 - __clz(m);
        lo += last * step;
        n = min(step, n - last * step);
    }
    return lo < b.sequences ? lo : -1;
}

template <bool F32, int ITEMS>
__global__ void __launch_bounds__(128) append_kernel(const AppendArgs a)
{
    __shared__ float2 turn[64];     // pair 8 m + e at 8 e + m: lanes with neighbouring items read neighbouring places
    __shared__ int64_t slot_at;     // element of the slot in k and v; -1: the token is not stored
    __shared__ int live;
    const int t = blockIdx.x, D = a.c.head_dim, per = D / 16;
    const int lane = threadIdx.x & 31;
    pdl_trigger();
    pdl_wait();
    // the items' chunks c0, c1 of head h: of q, then k, then v
    const int items = a.heads * per;
    const int first = (blockIdx.y * ITEMS) * 128 + threadIdx.x;
    Item<F32> it[ITEMS];
    const int kh = a.c.kv_heads;
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
        const int i = first + 128 * j;
        if (i >= items) break;
        const int h = i / per, m = i - h * per;
        const bool is_v = h >= a.q_heads + kh;
        const bool halves = m < a.rot / 16 && !a.interleaved && !is_v;
        const int c0 = halves ? 8 * m : 16 * m, c1 = halves ? c0 + a.rot / 2 : c0 + 8;
        const void *p = h < a.q_heads ? a.q : is_v ? a.v : a.k;
        const int64_t row = h < a.q_heads ? t * a.ldq + h * (int64_t)D
                                          : is_v ? t * a.ldv + (h - a.q_heads - kh) * (int64_t)D : t * a.ldk + (h - a.q_heads) * (int64_t)D;
        load_chunk<F32>(p, row + c0, it[j].a);
        load_chunk<F32>(p, row + c1, it[j].a + (F32 ? 2 : 1));
    }
    // every warp that needs the position finds it; the first stores the slot
    const int pairs = a.rot / 2;
    if ((int)threadIdx.x < max(32, (pairs + 31) / 32 * 32)) {
        double f = 0.0;
        if ((int)threadIdx.x < pairs) f = a.freq[threadIdx.x];
        const int s = seq_of_row(a.b, t);
        int pos = 0;
        bool mine = false;
        if (s >= 0) {
            const KvSeq q = kv_seq(a.b, s);
            mine = t >= q.first && t < q.first + q.n;
            pos = q.len - q.n + (t - q.first);
        }
        if (threadIdx.x < 32) {
            int64_t at = -1;
            if (lane == 0 && mine && pos >= 0 && pos < a.b.capacity) {
                const int pi = pos / a.c.page_size;
                const int64_t page = a.b.pages[(int64_t)s * a.b.ld_pages + pi];
                if (page >= 0 && page < a.c.pages) at = page * a.c.page_stride + (int64_t)(pos - pi * a.c.page_size) * a.c.slot_stride;
            }
            if (lane == 0) {
                slot_at = at;
                live = mine;
            }
        }
        if ((int)threadIdx.x < pairs) {
            if (a.positions) pos = a.positions[t];
            double x = (double)pos * (f * 0.15915494309189533577);  // turns
            x -= rint(x);
            float sn, cs;
            sincospif((float)(2.0 * x), &sn, &cs);
            turn[8 * (threadIdx.x & 7) + (threadIdx.x >> 3)] = make_float2(cs * a.scale, sn * a.scale);
        }
    }
    __syncthreads();
    if (!live) return;
    const int64_t at = slot_at;
#pragma unroll
    for (int j = 0; j < ITEMS; j++) {
        const int i = first + 128 * j;
        if (i >= items) break;
        const int h = i / per, m = i - h * per;
        const bool is_v = h >= a.q_heads + kh, turned = m < a.rot / 16 && !is_v;
        const bool halves = turned && !a.interleaved;
        const int c0 = halves ? 8 * m : 16 * m, c1 = halves ? c0 + a.rot / 2 : c0 + 8;
        float x[8], y[8];
        unpack_chunk<F32>(it[j].a, x);
        unpack_chunk<F32>(it[j].a + (F32 ? 2 : 1), y);
        if (halves) {
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float2 w = turn[8 * e + m];
                const float u = x[e] * w.x - y[e] * w.y, v = x[e] * w.y + y[e] * w.x;
                x[e] = u;
                y[e] = v;
            }
        } else if (turned) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 w = turn[4 * e + m], z = turn[32 + 4 * e + m];
                const float u = x[e] * w.x - x[e + 1] * w.y, v = x[e] * w.y + x[e + 1] * w.x;
                x[e] = u;
                x[e + 1] = v;
                const float p = y[e] * z.x - y[e + 1] * z.y, q = y[e] * z.y + y[e + 1] * z.x;
                y[e] = p;
                y[e + 1] = q;
            }
        }
        uint16_t *o;
        if (h < a.q_heads) {
            o = a.q_out + (t * a.ldq_out + h * (int64_t)D);
        } else {
            if (at < 0) continue;
            o = (is_v ? a.c.v : a.c.k) + at + (h - a.q_heads - (is_v ? kh : 0)) * a.c.head_stride;
        }
        *(uint4 *)(o + c0) = pack_chunk(x);
        *(uint4 *)(o + c1) = pack_chunk(y);
    }
}

bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

bool map_of(CUtensorMap *m, const uw_kv_desc &d, uint16_t *base, int box)
{
    auto fn = (PFN_cuTensorMapEncodeTiled_v12000)tensor_map_encoder();
    if (!fn) return false;
    const cuuint64_t dims[4] = {(cuuint64_t)d.head_dim, (cuuint64_t)d.page_size, (cuuint64_t)d.kv_heads, (cuuint64_t)d.pages};
    const cuuint64_t strides[3] = {(cuuint64_t)d.slot_stride * 2, (cuuint64_t)d.head_stride * 2, (cuuint64_t)d.page_stride * 2};
    const cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1}, estr[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int power_in(int n, int most)
{
    int p = 8;
    while (2 * p <= most && n % (2 * p) == 0) p *= 2;
    return p;
}

}  // namespace

namespace uw {

uw_status check_kv_device(const uw_kv_cache *c, const char *who)
{
    int device = 0;
    const cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return fail(UW_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
    return device == c->device ? UW_OK : fail(UW_ERR_INVALID_ARG, "%s: the cache is on device %d, the current one is %d", who, c->device, device);
}

uw_status check_kv_batch(const uw_kv_cache *c, const uw_kv_batch *b, int64_t rows, KvBatch *out, const char *who)
{
    if (!b || !b->starts || !b->lengths || !b->pages) return fail(UW_ERR_INVALID_ARG, "%s: NULL batch", who);
    if (!aligned(b->starts, 4) || !aligned(b->lengths, 4) || !aligned(b->pages, 4)) return fail(UW_ERR_INVALID_ARG, "%s: the batch is not 4-byte aligned", who);
    if (rows < 0 || rows > ((int64_t)1 << 31) - 1024) return fail(UW_ERR_SHAPE, "%s: rows=%lld", who, (long long)rows);
    if (b->sequences < 1 || b->sequences > 65536) return fail(UW_ERR_SHAPE, "%s: %d sequences outside 1..65536", who, b->sequences);
    const int64_t ld = b->ld_pages ? b->ld_pages : b->max_pages;
    if (b->max_pages < 1 || b->max_pages > ((int64_t)1 << 30) / c->d.page_size || (b->sequences > 1 && (ld < b->max_pages || ld > ((int64_t)1 << 40))))
        return fail(UW_ERR_SHAPE, "%s: max_pages=%lld ld_pages=%lld", who, (long long)b->max_pages, (long long)b->ld_pages);
    out->starts = b->starts;
    out->lengths = b->lengths;
    out->pages = b->pages;
    out->ld_pages = ld;
    out->sequences = b->sequences;
    out->rows = (int32_t)rows;
    out->capacity = (int32_t)(b->max_pages * c->d.page_size);
    return UW_OK;
}

}  // namespace uw

extern "C" uw_status uw_rotary_frequencies(int dim, double base, uw_rotary_scaling scaling, double factor, double low, double high,
                                           int64_t original, double *freq, float *scale)
{
    clear_error();
    if (!freq) return fail(UW_ERR_INVALID_ARG, "uw_rotary_frequencies: NULL output");
    if (dim < 16 || dim > 128 || dim % 16) return fail(UW_ERR_SHAPE, "uw_rotary_frequencies: dim %d", dim);
    if (!std::isfinite(base) || base <= 1.0) return fail(UW_ERR_INVALID_ARG, "uw_rotary_frequencies: base %g", base);
    if (scaling < UW_ROTARY_PLAIN || scaling > UW_ROTARY_RAMP) return fail(UW_ERR_INVALID_ARG, "uw_rotary_frequencies: scaling %d", (int)scaling);
    if (scaling != UW_ROTARY_PLAIN && (!std::isfinite(factor) || factor < 1.0)) return fail(UW_ERR_INVALID_ARG, "uw_rotary_frequencies: factor %g", factor);
    const bool ends = scaling == UW_ROTARY_BANDS || scaling == UW_ROTARY_RAMP;
    if (ends && (!std::isfinite(low) || !std::isfinite(high) || low < 0 || high <= low || (scaling == UW_ROTARY_RAMP && low <= 0) || original < 1))
        return fail(UW_ERR_INVALID_ARG, "uw_rotary_frequencies: low %g high %g original %lld", low, high, (long long)original);
    const double tau = 6.283185307179586476925;
    if (scaling == UW_ROTARY_STRETCHED) base *= std::pow(factor, dim / (dim - 2.0));
    double lo = 0, hi = 0;
    if (scaling == UW_ROTARY_RAMP) {  // the indices that make `high` and `low` turns over the original length
        const auto at = [&](double turns) { return dim * std::log((double)original / (turns * tau)) / (2 * std::log(base)); };
        lo = std::max(std::floor(at(high)), 0.0);
        hi = std::min(std::ceil(at(low)), dim - 1.0);
    }
    for (int i = 0; i < dim / 2; i++) {
        const double f = std::pow(base, -2.0 * i / dim);
        double keep = 1.0;
        if (scaling == UW_ROTARY_LINEAR) keep = 0.0;
        if (scaling == UW_ROTARY_BANDS) keep = std::min(std::max(((double)original * f / tau - low) / (high - low), 0.0), 1.0);
        if (scaling == UW_ROTARY_RAMP) keep = 1.0 - std::min(std::max((i - lo) / std::max(hi - lo, 0.001), 0.0), 1.0);
        freq[i] = scaling == UW_ROTARY_PLAIN || scaling == UW_ROTARY_STRETCHED ? f : keep * f + (1.0 - keep) * f / factor;
    }
    if (scale) *scale = scaling == UW_ROTARY_RAMP && factor > 1.0 ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    return UW_OK;
}

extern "C" uw_status uw_kv_create(const uw_kv_desc *desc, uw_kv_cache **out)
{
    clear_error();
    if (!desc || !out) return fail(UW_ERR_INVALID_ARG, "uw_kv_create: NULL argument");
    *out = nullptr;
    uw_kv_desc d = *desc;
    if (!d.k || !d.v || !aligned(d.k, 16) || !aligned(d.v, 16)) return fail(UW_ERR_INVALID_ARG, "uw_kv_create: k or v NULL or not 16-byte aligned");
    if (d.head_dim != 64 && d.head_dim != 128) return fail(UW_ERR_UNSUPPORTED, "uw_kv_create: head_dim %d (64 and 128 are supported)", d.head_dim);
    if (d.pages < 1 || d.pages > ((int64_t)1 << 31) - 1 || d.page_size < 8 || d.page_size > 65536 || d.page_size % 8 || d.kv_heads < 1 || d.kv_heads > 1024)
        return fail(UW_ERR_SHAPE, "uw_kv_create: pages=%lld page_size=%d kv_heads=%d", (long long)d.pages, d.page_size, d.kv_heads);
    if (d.kv_heads == 1) d.head_stride = d.head_dim;
    if (d.pages == 1) d.page_stride = d.head_dim;
    for (int64_t s : {d.page_stride, d.slot_stride, d.head_stride})
        if (s < d.head_dim || s % 8 || s >= ((int64_t)1 << 39))
            return fail(UW_ERR_INVALID_ARG, "uw_kv_create: strides %lld %lld %lld", (long long)d.page_stride, (long long)d.slot_stride, (long long)d.head_stride);
    uw_kv_cache *c = new (std::nothrow) uw_kv_cache;
    if (!c) return fail(UW_ERR_NO_MEMORY, "uw_kv_create: out of memory");
    memset((void *)c, 0, sizeof *c);
    c->d = d;
    c->box16 = power_in(d.page_size, 16);
    c->box128 = power_in(d.page_size, 128);
    uw_status s = UW_OK;
    cudaError_t e = cudaGetDevice(&c->device);
    if (e != cudaSuccess) s = fail(UW_ERR_CUDA, "uw_kv_create: %s", cudaGetErrorString(e));
    else if ((e = cudaMalloc(&c->status, 2 * sizeof(int))) != cudaSuccess) {
        cudaGetLastError();
        c->status = nullptr;
        s = fail(UW_ERR_NO_MEMORY, "uw_kv_create: %s", cudaGetErrorString(e));
    } else if ((e = cudaMemset(c->status, 0, 2 * sizeof(int))) != cudaSuccess || (e = cudaStreamSynchronize(0)) != cudaSuccess)
        s = fail(UW_ERR_CUDA, "uw_kv_create: %s", cudaGetErrorString(e));
    else if (!map_of(&c->k16, d, d.k, c->box16) || !map_of(&c->v16, d, d.v, c->box16) || !map_of(&c->k128, d, d.k, c->box128) ||
             !map_of(&c->v128, d, d.v, c->box128))
        s = fail(UW_ERR_UNSUPPORTED, "uw_kv_create: the driver describes no such copies");
    if (s != UW_OK) {
        if (c->status) cudaFree(c->status);
        delete c;
        return s;
    }
    *out = c;
    return UW_OK;
}

extern "C" void uw_kv_free(uw_kv_cache *c)
{
    if (!c) return;
    cudaFree(c->status);
    delete c;
}

extern "C" uw_status uw_kv_check(const uw_kv_cache *c, uw_stream stream)
{
    clear_error();
    if (!c) return fail(UW_ERR_INVALID_ARG, "uw_kv_check: NULL cache");
    cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
    if (e != cudaSuccess) return fail(UW_ERR_CUDA, "uw_kv_check: %s", cudaGetErrorString(e));
    int s = 0;
    if ((e = cudaMemcpy(&s, c->status, sizeof s, cudaMemcpyDeviceToHost)) != cudaSuccess) return fail(UW_ERR_CUDA, "uw_kv_check: %s", cudaGetErrorString(e));
    if (s) {
        if ((e = cudaMemset(c->status, 0, sizeof s)) != cudaSuccess) return fail(UW_ERR_CUDA, "uw_kv_check: %s", cudaGetErrorString(e));
        return fail(UW_ERR_TIMEOUT, "a bounded device wait expired");
    }
    return UW_OK;
}

extern "C" uw_status uw_kv_append(const uw_kv_cache *c, const uw_kv_batch *b, const uw_rotary *r, int64_t rows, uw_out_dtype dtype,
                                  const void *q, int64_t ldq, int q_heads, const void *k, int64_t ldk, const void *v, int64_t ldv,
                                  const int32_t *positions, uint16_t *q_out, int64_t ldq_out, uw_stream stream)
{
    clear_error();
    if (!c) return fail(UW_ERR_INVALID_ARG, "uw_kv_append: NULL cache");
    AppendArgs a{};
    uw_status s = check_kv_batch(c, b, rows, &a.b, "uw_kv_append");
    if (s != UW_OK) return s;
    if (dtype != UW_OUT_F32 && dtype != UW_OUT_BF16) return fail(UW_ERR_INVALID_ARG, "uw_kv_append: bad dtype");
    if (!q != !q_out || !k != !v) return fail(UW_ERR_INVALID_ARG, "uw_kv_append: q and q_out, k and v go together");
    if (!q && !k) return fail(UW_ERR_INVALID_ARG, "uw_kv_append: nothing to do");
    const int D = c->d.head_dim;
    if (q && (q_heads < 1 || q_heads > 65536)) return fail(UW_ERR_SHAPE, "uw_kv_append: %d query heads", q_heads);
    const int64_t dense_q = (int64_t)q_heads * D, dense_k = (int64_t)c->d.kv_heads * D, most = (int64_t)1 << 39;
    a.ldq = ldq ? ldq : dense_q;
    a.ldq_out = ldq_out ? ldq_out : dense_q;
    a.ldk = ldk ? ldk : dense_k;
    a.ldv = ldv ? ldv : dense_k;
    if ((q && rows > 1 && (a.ldq < dense_q || a.ldq_out < dense_q || a.ldq >= most || a.ldq_out >= most)) ||
        (k && rows > 1 && (a.ldk < dense_k || a.ldv < dense_k || a.ldk >= most || a.ldv >= most)) ||
        (q && (a.ldq % 8 || a.ldq_out % 8)) || (k && (a.ldk % 8 || a.ldv % 8)))
        return fail(UW_ERR_SHAPE, "uw_kv_append: ldq=%lld ldk=%lld ldv=%lld ldq_out=%lld", (long long)ldq, (long long)ldk, (long long)ldv, (long long)ldq_out);
    if (r) {
        if (r->dim < 16 || r->dim > D || r->dim % 16) return fail(UW_ERR_SHAPE, "uw_kv_append: rotary dim %d of %d", r->dim, D);
        if (r->layout != UW_ROTARY_HALF && r->layout != UW_ROTARY_INTERLEAVED) return fail(UW_ERR_INVALID_ARG, "uw_kv_append: layout %d", r->layout);
        if (!r->freq || !aligned(r->freq, 8)) return fail(UW_ERR_INVALID_ARG, "uw_kv_append: freq NULL or not 8-byte aligned");
        a.rot = r->dim;
        a.interleaved = r->layout == UW_ROTARY_INTERLEAVED;
        a.freq = r->freq;
        a.scale = r->scale;
    }
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(positions, 4))
        return fail(UW_ERR_INVALID_ARG, "uw_kv_append: a pointer is not aligned");
    if (rows == 0) return UW_OK;
    if (q) {
        // a CTA's queries are another's keys and values, or another part of the same row: only its own may be written over
        const int es = dtype == UW_OUT_F32 ? 4 : 2;
        const bool place = q == q_out && dtype == UW_OUT_BF16 && (rows == 1 || a.ldq == a.ldq_out);
        const RowBytes o{q_out, a.ldq_out * 2, dense_q * 2};
        if ((!place && rows_overlap({q, a.ldq * es, dense_q * es}, o, rows)) ||
            (k && (rows_overlap({k, a.ldk * es, dense_k * es}, o, rows) || rows_overlap({v, a.ldv * es, dense_k * es}, o, rows))))
            return fail(UW_ERR_INVALID_ARG, "uw_kv_append: q_out overlaps q, k or v (it may be q itself, of bf16 and with its stride)");
    }
    if ((s = check_kv_device(c, "uw_kv_append")) != UW_OK) return s;
    a.c = c->d;
    a.q = q;
    a.k = k;
    a.v = v;
    a.positions = positions;
    a.q_out = q_out;
    a.q_heads = q ? q_heads : 0;
    if (!k) a.c.kv_heads = 0;
    a.heads = a.q_heads + 2 * a.c.kv_heads;
    const int64_t items = (int64_t)a.heads * (D / 16);
    // Few tokens: an item a thread, so that many CTAs share a token.  Many: several, for one lookup and one set of angles.
    const bool f32 = dtype == UW_OUT_F32, few = rows * ((items + 127) / 128) <= 8 * (int64_t)num_sms();
    const int per = few ? 1 : f32 ? 2 : 4;
    const dim3 grid((unsigned)rows, (unsigned)((items + 128 * per - 1) / (128 * per)));
    const cudaError_t e = f32 ? launch_dependent(few ? append_kernel<true, 1> : append_kernel<true, 2>, grid, 128, 0, 0, (cudaStream_t)stream, a)
                              : launch_dependent(few ? append_kernel<false, 1> : append_kernel<false, 4>, grid, 128, 0, 0, (cudaStream_t)stream, a);
    return e == cudaSuccess ? UW_OK : fail(UW_ERR_CUDA, "uw_kv_append: launch: %s", cudaGetErrorString(e));
}
