// k_norm.cu - the norms before and after a block with its gate and residual, one pass (sm_103a).
//
// Per row: o = block output (a row, or the weighted sum of a token's expert rows); optionally o <- post o / rms(o);
// optionally o <- gate o; h' = a h + s o; optionally u = pre h' / rms(h').  Two sums of squares depend on each other
// (the second needs the first), so a row is held on chip between them and each input is read once.
//
// One CTA per row, several rows on an SM.  A row's inputs are asked for at once, two chunks of eight elements a thread,
// before the first of its two sums of squares; the weights, which all rows share, come when they are needed.  A join of a
// sum takes one barrier, in a fixed order.  Rows of a multiple of 8 elements are read in 16-byte pieces, others in pairs or
// single elements with neighbouring threads side by side.
// Bound by memory: 4096 rows of 4096 bf16 with residual and pre-norm take 22.0 us (6.1 TB/s), with post-norm and gate too
// 26.8 (27.5 without instructions on pairs); 8192 rows of 8192 fp32 137 us (6.9 TB/s); 4096 rows of 2048 joined from 8 expert rows each 37.1 us (5.9 TB/s).
// Rows of odd lengths, read by single elements, are bound by the loads in flight: 2258 rows of 4173 joined from 8 bf16 expert
// rows take 140 us against 34 for their bytes, 4171 of 4098 in pairs 93 against 56.  They take 64 registers a thread and
// fewer expert rows at once (128 registers and four: 280 and 176 us).
// One chunk a thread took 31.3 us in the second case, four 30.5; a persistent CTA that keeps the weights and asks for its
// next row ahead 54, as its registers leave too few rows on an SM to hide the joins.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "f32x2.cuh"
#include "launch.cuh"
#include "uw_internal.h"

using namespace uw;
using namespace uw::dev;

namespace {

struct NormArgs {
    uw_norm n;
    int64_t rows, y_rows;
    const void *h, *y;
    void *h_out;
    const int32_t *pos;
    const float *weights;
    int topk;
    uint16_t *u;
    uint32_t gate_every;  // as in n, at most 2^31 (rows are fewer): a 64-bit division cost 1 us of 28
};

// eight elements as loaded: bf16 in a, fp32 in a and b
template <bool F32>
struct Raw {
    uint4 a;
};
template <>
struct Raw<true> {
    uint4 a, b;
};

// A thread's chunk c of a row of D elements is 8 / W pieces of W elements, blockDim pieces apart.
template <int W>
__device__ __forceinline__ int piece_at(int c, int j)
{
    return ((c * (8 / W) + j) * (int)blockDim.x + (int)threadIdx.x) * W;
}

// zeros past the row's end, or where !in
template <int W, bool F32>
__device__ __forceinline__ Raw<F32> load8(const void *p, int64_t row, int D, int c, bool in = true)
{
    Raw<F32> r;
    const uint8_t *base = (const uint8_t *)p + row * D * (F32 ? 4 : 2);
    if constexpr (W == 8) {
        const uint4 zero = make_uint4(0, 0, 0, 0);
        const int i = piece_at<W>(c, 0);
        const uint4 *q = (const uint4 *)(base + (int64_t)i * (F32 ? 4 : 2));
        in = in && i < D;
        r.a = in ? q[0] : zero;
        if constexpr (F32) r.b = in ? q[1] : zero;
    } else {
        uint32_t w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        uint32_t piece[8 / W], high[8 / W];  // every load before the first use
#pragma unroll
        for (int j = 0; j < 8 / W; j++) {
            const int i = piece_at<W>(c, j);
            const bool here = in && i < D;
            const uint8_t *q = base + (int64_t)i * (F32 ? 4 : 2);
            if constexpr (F32 && W == 2) {
                const uint2 v = here ? *(const uint2 *)q : make_uint2(0, 0);
                piece[j] = v.x;
                high[j] = v.y;
            } else if constexpr (F32 || W == 2) {
                piece[j] = here ? *(const uint32_t *)q : 0u;
            } else {
                piece[j] = here ? *(const uint16_t *)q : 0u;
            }
        }
#pragma unroll
        for (int j = 0; j < 8 / W; j++) {
            if constexpr (F32 && W == 2) {
                w[2 * j] = piece[j];
                w[2 * j + 1] = high[j];
            } else if constexpr (F32 || W == 2) {
                w[j] = piece[j];
            } else if (j % 2 == 0) {
                w[j / 2] = piece[j] | piece[j + 1] << 16;
            }
        }
        r.a = make_uint4(w[0], w[1], w[2], w[3]);
        if constexpr (F32) r.b = make_uint4(w[4], w[5], w[6], w[7]);
    }
    return r;
}

template <bool F32>
__device__ __forceinline__ void unpack8(const Raw<F32> &r, float (&f)[8])
{
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int q = 0; q < 4; q++) {
        if constexpr (F32) {
            f[q] = __uint_as_float(w[q]);
        } else {
            f[2 * q] = __uint_as_float(w[q] << 16);
            f[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
        }
    }
    if constexpr (F32) {
        f[4] = __uint_as_float(r.b.x);
        f[5] = __uint_as_float(r.b.y);
        f[6] = __uint_as_float(r.b.z);
        f[7] = __uint_as_float(r.b.w);
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *(const uint32_t *)&v;
}

template <int W, bool F32>
__device__ __forceinline__ void store8(void *p, int64_t row, int D, int c, const float (&f)[8])
{
    uint8_t *base = (uint8_t *)p + row * D * (F32 ? 4 : 2);
#pragma unroll
    for (int j = 0; j < 8 / W; j++) {
        const int i = piece_at<W>(c, j);
        if (i >= D) continue;
        if constexpr (F32) {
            float *q = (float *)(base + (int64_t)i * 4);
            if constexpr (W == 8) {
                *(float4 *)q = make_float4(f[0], f[1], f[2], f[3]);
                *(float4 *)(q + 4) = make_float4(f[4], f[5], f[6], f[7]);
            } else if constexpr (W == 2) {
                *(float2 *)q = make_float2(f[2 * j], f[2 * j + 1]);
            } else {
                *q = f[j];
            }
        } else {
            uint8_t *q = base + (int64_t)i * 2;
            if constexpr (W == 8) *(uint4 *)q = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
            else if constexpr (W == 2) *(uint32_t *)q = pack2(f[2 * j], f[2 * j + 1]);
            else *(__nv_bfloat16 *)q = __float2bfloat16_rn(f[j]);
        }
    }
}

// a chunk's eight elements two at a time
__device__ __forceinline__ void mul8(float (&o)[8], const float (&f)[8])
{
#pragma unroll
    for (int q = 0; q < 8; q += 2) unpair(mul2(pair(o[q], o[q + 1]), pair(f[q], f[q + 1])), o[q], o[q + 1]);
}
__device__ __forceinline__ void scale8(float (&o)[8], float s)
{
#pragma unroll
    for (int q = 0; q < 8; q += 2) unpair(mul2(pair(o[q], o[q + 1]), pair(s, s)), o[q], o[q + 1]);
}
// o += s f
__device__ __forceinline__ void add8(float (&o)[8], float s, const float (&f)[8])
{
#pragma unroll
    for (int q = 0; q < 8; q += 2) unpair(fma2(pair(s, s), pair(f[q], f[q + 1]), pair(o[q], o[q + 1])), o[q], o[q + 1]);
}
__device__ __forceinline__ Pair squares8(const float (&o)[8], Pair ss)
{
#pragma unroll
    for (int q = 0; q < 8; q += 2) ss = fma2(pair(o[q], o[q + 1]), pair(o[q], o[q + 1]), ss);
    return ss;
}
__device__ __forceinline__ float both(Pair p)
{
    float a, b;
    unpair(p, a, b);
    return a + b;
}

// the sum over the CTA, in a fixed order, to every thread; red: a buffer of this call's own
__device__ __forceinline__ float block_sum(float v, float *red)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if (warps == 1) return v;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    float s = lane < warps ? red[lane] : 0.f;
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    return s;
}

// Five CTAs of 256 threads an SM hide more of the joins, at 48 registers; rows of y in fp32 or joined need more (4096 rows of
// 4096 with post-norm and gate took 28.8 us with five, 30.9 with three; all in fp32 42.3 and 41.4).
// CH: chunks of 8 elements a thread holds (dim <= 8 CH blockDim); TOPK: y holds expert rows; W: elements of an access;
// RF, BF: h and h_out, y in fp32
template <int CH, int MAXT, bool TOPK, int W, bool RF, bool BF>
__global__ void __launch_bounds__(MAXT, W < 8 ? 1024 / MAXT : MAXT == 256 ? (TOPK || BF ? 3 : 5) : 1) norm_kernel(const NormArgs a)
{
    __shared__ float red[2][32];
    const int D = (int)a.n.dim;
    const int64_t row = blockIdx.x;
    pdl_trigger();
    const uint32_t gate_row = a.n.gate ? blockIdx.x / a.gate_every : 0u;
    pdl_wait();
    float o[CH][8];
    Raw<RF> h[CH];
    if constexpr (TOPK) {
        // lane j: place and weight of the row's j-th expert row
        const int lane = threadIdx.x & 31;
        int pos = -1;
        float weight = 0.f;
        if (lane < a.topk) {
            pos = a.pos[row * a.topk + lane];
            weight = a.weights[row * a.topk + lane];
        }
#pragma unroll
        for (int c = 0; c < CH; c++) {
            if (a.h) h[c] = load8<W, RF>(a.h, row, D, c);
#pragma unroll
            for (int q = 0; q < 8; q++) o[c][q] = 0.f;
        }
        constexpr int kB = CH > 2 ? 1 : W == 8 ? 4 : W;  // expert rows on their way, as registers allow
        for (int j0 = 0; j0 < a.topk; j0 += kB) {
            Raw<BF> e[kB][CH];
            float w[kB];
#pragma unroll
            for (int j = 0; j < kB; j++) {
                const int p = __shfl_sync(0xFFFFFFFFu, pos, (j0 + j) & 31);
                const bool in = j0 + j < a.topk && p >= 0 && p < a.y_rows;
                w[j] = __shfl_sync(0xFFFFFFFFu, weight, (j0 + j) & 31);
                if (!in) w[j] = 0.f;
#pragma unroll
                for (int c = 0; c < CH; c++) e[j][c] = load8<W, BF>(a.y, in ? p : 0, D, c, in);
            }
#pragma unroll
            for (int j = 0; j < kB; j++)
#pragma unroll
                for (int c = 0; c < CH; c++) {
                    float f[8];
                    unpack8(e[j][c], f);
                    add8(o[c], w[j], f);
                }
        }
    } else {
        Raw<BF> y[CH];
#pragma unroll
        for (int c = 0; c < CH; c++) {
            if (a.y) y[c] = load8<W, BF>(a.y, row, D, c);
            if (a.h) h[c] = load8<W, RF>(a.h, row, D, c);
        }
#pragma unroll
        for (int c = 0; c < CH; c++) {
            if (a.y) unpack8(y[c], o[c]);
            else
#pragma unroll
                for (int q = 0; q < 8; q++) o[c][q] = 0.f;
        }
    }
    float scale = a.n.out_scale;
    Pair ss = pair(0.f, 0.f);
    if (a.n.post_weight) {
#pragma unroll
        for (int c = 0; c < CH; c++) ss = squares8(o[c], ss);  // zeros past the row's end
        scale *= rsqrtf(block_sum(both(ss), red[0]) / (float)D + a.n.eps);
        ss = pair(0.f, 0.f);
    }
#pragma unroll
    for (int c = 0; c < CH; c++) {
        float f[8];
        if (a.y && a.n.post_weight) {
            unpack8(load8<W, false>(a.n.post_weight, 0, D, c), f);
            mul8(o[c], f);
        }
        if (a.y && a.n.gate) {
            unpack8(load8<W, false>(a.n.gate, gate_row, D, c), f);
            mul8(o[c], f);
        }
        scale8(o[c], a.y ? scale : 0.f);
        if (a.h) {
            unpack8(h[c], f);
            add8(o[c], a.n.res_scale, f);
        }
        if (a.h_out) store8<W, RF>(a.h_out, row, D, c, o[c]);
    }
    if (!a.u) return;
    // zeros past the row's end, unless a scale is not finite
#pragma unroll
    for (int c = 0; c < CH; c++) {
        bool whole = true;
#pragma unroll
        for (int j = 0; j < 8 / W; j++) whole = whole && piece_at<W>(c, j) < D;
        if (whole) ss = squares8(o[c], ss);
        else if constexpr (W < 8) {
#pragma unroll
            for (int q = 0; q < 8; q++)
                if (piece_at<W>(c, q / W) < D) ss = fma2(pair(o[c][q], 0.f), pair(o[c][q], 0.f), ss);
        }
    }
    const float inv = rsqrtf(block_sum(both(ss), red[1]) / (float)D + a.n.eps);
#pragma unroll
    for (int c = 0; c < CH; c++) {
        float f[8];
        unpack8(load8<W, false>(a.n.pre_weight, 0, D, c), f);
        scale8(o[c], inv);
        mul8(f, o[c]);
        store8<W, false>(a.u, row, D, c, f);
    }
}

template <int CH, int MAXT, bool TOPK, int W>
cudaError_t launch_width(const NormArgs &a, int threads, cudaStream_t st)
{
    const bool rf = a.n.res_dtype == UW_OUT_F32, bf = a.n.block_dtype == UW_OUT_F32;
    auto kernel = rf ? (bf ? norm_kernel<CH, MAXT, TOPK, W, true, true> : norm_kernel<CH, MAXT, TOPK, W, true, false>)
                     : (bf ? norm_kernel<CH, MAXT, TOPK, W, false, true> : norm_kernel<CH, MAXT, TOPK, W, false, false>);
    return launch_dependent(kernel, dim3((unsigned)a.rows), (unsigned)threads, 0, 0, st, a);
}

template <int CH, int MAXT>
cudaError_t launch_chunks(const NormArgs &a, int threads, cudaStream_t st)
{
    const int w = a.n.dim % 8 == 0 ? 8 : a.n.dim % 2 == 0 ? 2 : 1;
    if (a.topk)
        return w == 8 ? launch_width<CH, MAXT, true, 8>(a, threads, st)
               : w == 2 ? launch_width<CH, MAXT, true, 2>(a, threads, st) : launch_width<CH, MAXT, true, 1>(a, threads, st);
    return w == 8 ? launch_width<CH, MAXT, false, 8>(a, threads, st)
           : w == 2 ? launch_width<CH, MAXT, false, 2>(a, threads, st) : launch_width<CH, MAXT, false, 1>(a, threads, st);
}

// two chunks a thread up to 1024 threads, then eight
cudaError_t launch_norm(const NormArgs &a, cudaStream_t st)
{
    const int64_t chunks = (a.n.dim + 7) / 8;
    const int ch = chunks <= 2048 ? 2 : 8;
    const int threads = (int)(((chunks + ch - 1) / ch + 31) / 32 * 32);
    if (ch == 2 && threads <= 256) return launch_chunks<2, 256>(a, threads, st);
    if (ch == 2) return threads <= 512 ? launch_chunks<2, 512>(a, threads, st) : launch_chunks<2, 1024>(a, threads, st);
    return launch_chunks<8, 1024>(a, threads, st);
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

extern "C" uw_status uw_block_norm(const uw_norm *n, int64_t rows, const void *h, void *h_out, const void *y, int64_t y_rows,
                                   const int32_t *pos, const float *weights, int topk, uint16_t *u, uw_stream stream)
{
    clear_error();
    if (!n) return fail(UW_ERR_INVALID_ARG, "uw_block_norm: NULL description");
    if (n->dim < 1 || n->dim > 65536 || rows < 0 || rows > ((int64_t)1 << 31) - 1024 || y_rows < 0)
        return fail(UW_ERR_SHAPE, "uw_block_norm: rows=%lld dim=%lld y_rows=%lld", (long long)rows, (long long)n->dim, (long long)y_rows);
    if ((n->res_dtype != UW_OUT_F32 && n->res_dtype != UW_OUT_BF16) || (n->block_dtype != UW_OUT_F32 && n->block_dtype != UW_OUT_BF16))
        return fail(UW_ERR_INVALID_ARG, "uw_block_norm: bad dtype");
    if (topk < 0 || topk > 16) return fail(UW_ERR_INVALID_ARG, "uw_block_norm: topk %d outside 0..16", topk);
    if (topk && (!pos || !weights || !y || (((uintptr_t)pos | (uintptr_t)weights) & 3)))
        return fail(UW_ERR_INVALID_ARG, "uw_block_norm: topk needs y, pos and weights (4-byte aligned)");
    if (n->gate && n->gate_every < 1) return fail(UW_ERR_INVALID_ARG, "uw_block_norm: gate_every %lld", (long long)n->gate_every);
    if (!u != !n->pre_weight) return fail(UW_ERR_INVALID_ARG, "uw_block_norm: u and pre_weight go together");
    if (!u && !h_out) return fail(UW_ERR_INVALID_ARG, "uw_block_norm: nothing to write");
    if (!h && !y) return fail(UW_ERR_INVALID_ARG, "uw_block_norm: nothing to read");
    if (!aligned16(h) || !aligned16(h_out) || !aligned16(y) || !aligned16(u) || !aligned16(n->post_weight) || !aligned16(n->gate) ||
        !aligned16(n->pre_weight))
        return fail(UW_ERR_INVALID_ARG, "uw_block_norm: a pointer is not 16-byte aligned");
    if (rows == 0) return UW_OK;
    const NormArgs a{*n, rows, y_rows, h, y, h_out, pos, weights, topk, u, (uint32_t)std::min<int64_t>(n->gate_every, (int64_t)1 << 31)};
    const cudaError_t e = launch_norm(a, (cudaStream_t)stream);
    return e == cudaSuccess ? UW_OK : fail(UW_ERR_CUDA, "uw_block_norm: launch: %s", cudaGetErrorString(e));
}
