// k_norm.cu - the norms before and after a block with its gate and residual, one pass (sm_103a).
//
// Per row: o = block output (a row, or the weighted sum of a token's expert rows); optionally o <- post o / rms(o);
// optionally o <- gate o; h' = a h + s o; optionally u = pre h' / rms(h').  Two sums of squares depend on each other
// (the second needs the first), so a row is held on chip between them and each input is read once.
//
// One CTA per row.  Each thread holds kVec * chunks elements of o in registers; a row's sum of squares is joined
// through shared memory in a fixed order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.cuh"
#include "uw_internal.h"

using namespace uw;

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
};

__device__ __forceinline__ float bf(uint32_t bits) { return __uint_as_float(bits << 16); }

// eight elements at i of an fp32 or bf16 array, the first cnt of them (VEC: all, 16-byte aligned)
template <bool VEC>
__device__ __forceinline__ void load8(const void *p, int dtype, int64_t i, int cnt, float (&f)[8])
{
    if (VEC) {
        if (dtype == UW_OUT_BF16) {
            const uint4 v = *(const uint4 *)((const uint16_t *)p + i);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int q = 0; q < 4; q++) {
                f[2 * q] = __uint_as_float(w[q] << 16);
                f[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
            }
        } else {
            const float4 a = *(const float4 *)((const float *)p + i), b = *(const float4 *)((const float *)p + i + 4);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        }
        return;
    }
#pragma unroll
    for (int q = 0; q < 8; q++)
        f[q] = q < cnt ? (dtype == UW_OUT_BF16 ? bf(((const uint16_t *)p)[i + q]) : ((const float *)p)[i + q]) : 0.f;
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *(const uint32_t *)&v;
}

template <bool VEC>
__device__ __forceinline__ void store8(void *p, int dtype, int64_t i, int cnt, const float (&f)[8])
{
    if (VEC) {
        if (dtype == UW_OUT_BF16) {
            *(uint4 *)((uint16_t *)p + i) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
        } else {
            *(float4 *)((float *)p + i) = make_float4(f[0], f[1], f[2], f[3]);
            *(float4 *)((float *)p + i + 4) = make_float4(f[4], f[5], f[6], f[7]);
        }
        return;
    }
#pragma unroll
    for (int q = 0; q < 8; q++)
        if (q < cnt) {
            if (dtype == UW_OUT_BF16) ((__nv_bfloat16 *)p)[i + q] = __float2bfloat16_rn(f[q]);
            else ((float *)p)[i + q] = f[q];
        }
}

// the sum over the CTA, in a fixed order, to every thread
__device__ __forceinline__ float block_sum(float v, float *red)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if (warps == 1) return v;
    __syncthreads();
    if (lane == 0) red[warp] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < warps; w++) s += red[w];
    return s;
}

// CH: chunks of 8 elements a thread holds (dim <= 8 CH blockDim)
template <int CH, bool VEC>
__global__ void __launch_bounds__(1024) norm_kernel(const NormArgs a)
{
    __shared__ float red[32];
    const int64_t D = a.n.dim;
    const int64_t row = blockIdx.x;
    pdl_trigger();
    pdl_wait();
    float o[CH][8];
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < CH; c++) {
        const int64_t i = 8 * ((int64_t)c * blockDim.x + threadIdx.x);
        const int cnt = (int)max((int64_t)0, min((int64_t)8, D - i));
#pragma unroll
        for (int q = 0; q < 8; q++) o[c][q] = 0.f;
        if (cnt <= 0 || !a.y) continue;
        if (a.topk) {
            for (int j = 0; j < a.topk; j++) {
                const int64_t p = __ldg(a.pos + row * a.topk + j);
                if (p < 0 || p >= a.y_rows) continue;
                const float w = __ldg(a.weights + row * a.topk + j);
                float f[8];
                load8<VEC>(a.y, a.n.block_dtype, p * D + i, cnt, f);
#pragma unroll
                for (int q = 0; q < 8; q++) o[c][q] = fmaf(w, f[q], o[c][q]);
            }
        } else {
            load8<VEC>(a.y, a.n.block_dtype, row * D + i, cnt, o[c]);
        }
#pragma unroll
        for (int q = 0; q < 8; q++)
            if (q < cnt) ss = fmaf(o[c][q], o[c][q], ss);
    }
    float scale = a.n.out_scale;
    if (a.n.post_weight) scale *= rsqrtf(block_sum(ss, red) / (float)D + a.n.eps);
    ss = 0.f;
#pragma unroll
    for (int c = 0; c < CH; c++) {
        const int64_t i = 8 * ((int64_t)c * blockDim.x + threadIdx.x);
        const int cnt = (int)max((int64_t)0, min((int64_t)8, D - i));
        if (cnt <= 0) continue;
        float f[8];
        if (a.n.post_weight) {
            load8<VEC>(a.n.post_weight, UW_OUT_BF16, i, cnt, f);
#pragma unroll
            for (int q = 0; q < 8; q++) o[c][q] *= f[q];
        }
        if (a.n.gate) {
            load8<VEC>(a.n.gate, UW_OUT_BF16, row / a.n.gate_every * D + i, cnt, f);
#pragma unroll
            for (int q = 0; q < 8; q++) o[c][q] *= f[q];
        }
        if (a.h) load8<VEC>(a.h, a.n.res_dtype, row * D + i, cnt, f);
#pragma unroll
        for (int q = 0; q < 8; q++) {
            float r = a.y ? scale * o[c][q] : 0.f;
            if (a.h) r = fmaf(a.n.res_scale, f[q], r);
            o[c][q] = r;
            if (q < cnt) ss = fmaf(r, r, ss);
        }
        if (a.h_out) store8<VEC>(a.h_out, a.n.res_dtype, row * D + i, cnt, o[c]);
    }
    if (!a.u) return;
    const float inv = rsqrtf(block_sum(ss, red) / (float)D + a.n.eps);
#pragma unroll
    for (int c = 0; c < CH; c++) {
        const int64_t i = 8 * ((int64_t)c * blockDim.x + threadIdx.x);
        const int cnt = (int)max((int64_t)0, min((int64_t)8, D - i));
        if (cnt <= 0) continue;
        float f[8];
        load8<VEC>(a.n.pre_weight, UW_OUT_BF16, i, cnt, f);
#pragma unroll
        for (int q = 0; q < 8; q++) f[q] *= o[c][q] * inv;
        store8<VEC>(a.u, UW_OUT_BF16, row * D + i, cnt, f);
    }
}

template <int CH>
cudaError_t launch_ch(const NormArgs &a, int threads, bool vec, cudaStream_t st)
{
    return launch_dependent(vec ? norm_kernel<CH, true> : norm_kernel<CH, false>, dim3((unsigned)a.rows), (unsigned)threads, 0, 0, st, a);
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
    const NormArgs a{*n, rows, y_rows, h, y, h_out, pos, weights, topk, u};
    const int64_t chunks = (n->dim + 7) / 8;
    const bool vec = n->dim % 8 == 0;
    cudaStream_t st = (cudaStream_t)stream;
    // up to 512 threads of one chunk each, then more chunks a thread, then more threads
    const int ch = chunks <= 512 ? 1 : chunks <= 1024 ? 2 : chunks <= 4096 ? 4 : 8;
    const int threads = (int)(((chunks + ch - 1) / ch + 31) / 32 * 32);
    cudaError_t e;
    switch (ch) {
    case 1: e = launch_ch<1>(a, threads, vec, st); break;
    case 2: e = launch_ch<2>(a, threads, vec, st); break;
    case 4: e = launch_ch<4>(a, threads, vec, st); break;
    default: e = launch_ch<8>(a, threads, vec, st); break;
    }
    return e == cudaSuccess ? UW_OK : fail(UW_ERR_CUDA, "uw_block_norm: launch: %s", cudaGetErrorString(e));
}
