// k_group_gemv.cu - the grouped product for experts with a few rows each (sm_103a): every expert that has rows
// streams its compressed weights once and multiplies them on the tensor pipe (mma.sync m16n8k16, fp32 accumulate).
//
// A CTA owns one granule of 16 outputs (gated: of both matrices) of one expert over all of K; its warps take the
// 64-weight steps in turn.  A lane loads its part of a granule with three 16-byte loads straight into the registers
// of the A operand (the group's form is laid out for that), so the weights pass through no shared memory; one
// shared-memory sum joins the warps, in a fixed order.  The logical k of the instruction is permuted so that a lane's
// pairs are its 16 consecutive weights; X is read in the same order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "group.cuh"
#include "uw_internal.h"

namespace uw {

namespace {

using namespace dev;

constexpr int kWarps = 8;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// weights are read once: no place in L1
__device__ __forceinline__ uint4 ld_stream(const void *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// a lane's part of one granule of a step
struct Part {
    uint4 s0, s1, c;  // sign+mantissa of rows g and g + 8, distances of both
    uint32_t mask;    // verbatim bits of the granule's 16 rows
};

__device__ __forceinline__ Part load_part(const GroupView &v, int64_t step, int gi, int at)
{
    const uint8_t *st = v.steps + step * kStepBytes;
    Part p;
    p.s0 = ld_stream(st + gi * 1024 + at);
    p.s1 = ld_stream(st + gi * 1024 + 512 + at);
    p.c = ld_stream(st + kStepSm + gi * 512 + at);
    p.mask = __ldg((const uint16_t *)(st + kStepRec) + gi);
    return p;
}

// rows g and g + 8 of a granule's step as bf16 pairs
__device__ __forceinline__ void rebuild_part(const GroupView &v, const Part &p, int64_t step, int gi, int g, int t, uint32_t B,
                                             uint32_t (&a)[8], uint32_t (&b)[8])
{
    rebuild_chunk(p.s0, make_uint2(p.c.x, p.c.y), B, a);
    rebuild_chunk(p.s1, make_uint2(p.c.z, p.c.w), B, b);
    if (p.mask) {
        const StepRec &r = *step_rec(v.steps, step);
        uint32_t m[4];
#pragma unroll
        for (int i = 0; i < 4; i++) m[i] = __ldg(&r.mask[i]);
        const uint8_t *vb = v.verb + (uint64_t)__ldg(&r.first) * 64 + 16 * t;
        const int row = 16 * gi + g;
        if ((p.mask >> g) & 1u) rebuild_chunk_verbatim(p.s0, __ldg((const uint4 *)(vb + (uint64_t)verbatim_rank(m, row) * 64)), a);
        if ((p.mask >> (g + 8)) & 1u)
            rebuild_chunk_verbatim(p.s1, __ldg((const uint4 *)(vb + (uint64_t)verbatim_rank(m, row + 8) * 64)), b);
        __syncwarp();  // the products need the warp together again
    }
}

template <bool GATED>
__global__ void __launch_bounds__(32 * kWarps) group_gemv_kernel(const GroupCall c, int all_experts)
{
    constexpr int NG = GATED ? 2 : 1;
    __shared__ float part[kWarps][NG][16][8];
    const GroupView &v = c.v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

    // the expert: blockIdx.y itself, or (fewer rows than experts) the blockIdx.y-th that has rows
    int e = blockIdx.y, lo = 0, hi = 0;
    const int R = (int)c.rows;
    auto off = [&](int i) { return min(max(__ldg(c.offsets + i), 0), R); };
    if (all_experts) {
        lo = off(e);
        hi = off(e + 1);
    } else {
        int left = e;
        e = -1;
        for (int e0 = 0; e0 < v.experts && e < 0; e0 += 32) {
            int l = 0, h = 0;
            if (e0 + lane < v.experts) {
                l = off(e0 + lane);
                h = off(e0 + lane + 1);
            }
            const uint32_t has = __ballot_sync(0xFFFFFFFFu, h > l);
            if (left < __popc(has)) {
                const int i = __fns(has, 0, left + 1);
                e = e0 + i;
                lo = __shfl_sync(0xFFFFFFFFu, l, i);
                hi = __shfl_sync(0xFFFFFFFFu, h, i);
            } else {
                left -= __popc(has);
            }
        }
        if (e < 0) return;
    }
    if (hi <= lo) return;

    const int64_t vg = (int64_t)blockIdx.x * NG;
    const int gi = (int)(vg & 7);
    const int64_t s0 = ((int64_t)e * v.tiles + (vg >> 3)) * v.ksteps;
    const int at = 128 * t + 16 * g;
    uint32_t B[NG];
#pragma unroll
    for (int n = 0; n < NG; n++) B[n] = __ldg(v.base + e * NG + n);

    for (int r0 = lo; r0 < hi; r0 += 8) {
        // this lane's row of X (row g of the eight)
        const int r = r0 + g;
        const uint16_t *xr = nullptr;
        if (r < hi) {
            const int64_t src = c.row_src ? __ldg(c.row_src + r) : r;
            if (src >= 0 && src < c.x_rows) xr = c.x + src * c.ldx + 16 * t;
        }
        float acc[NG][4];
#pragma unroll
        for (int n = 0; n < NG; n++)
#pragma unroll
            for (int i = 0; i < 4; i++) acc[n][i] = 0.f;
        for (int ks = warp; ks < v.ksteps; ks += kWarps) {
            Part p[NG];
#pragma unroll
            for (int n = 0; n < NG; n++) p[n] = load_part(v, s0 + ks, gi + n, at);
            uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
            if (xr) {
                x0 = __ldg((const uint4 *)(xr + (int64_t)ks * kStepW));
                x1 = __ldg((const uint4 *)(xr + (int64_t)ks * kStepW) + 1);
            }
#pragma unroll
            for (int n = 0; n < NG; n++) {
                uint32_t a[8], b[8];
                rebuild_part(v, p[n], s0 + ks, gi + n, g, t, B[n], a, b);
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    const uint4 &x = q < 2 ? x0 : x1;
                    mma16816(acc[n], a[2 * q], b[2 * q], a[2 * q + 1], b[2 * q + 1], word_of(x, 2 * (q & 1)), word_of(x, 2 * (q & 1) + 1));
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NG; n++)
#pragma unroll
            for (int i = 0; i < 4; i++) part[warp][n][g + 8 * (i >> 1)][2 * t + (i & 1)] = acc[n][i];
        __syncthreads();
        if (threadIdx.x < 128) {
            const int o = threadIdx.x & 15, j = threadIdx.x >> 4;
            float s[NG];
#pragma unroll
            for (int n = 0; n < NG; n++) {
                s[n] = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; w++) s[n] += part[w][n][o][j];
            }
            float f = s[0];
            if (GATED) f = gated(s[0], s[NG - 1]);
            const int64_t col = (int64_t)blockIdx.x * kGran + o;
            if (r0 + j < hi && col < v.N) {
                const int64_t i = (int64_t)(r0 + j) * c.ldy + col;
                if (c.out_bf16) ((__nv_bfloat16 *)c.y)[i] = __float2bfloat16_rn(f);
                else ((float *)c.y)[i] = f;
            }
        }
        __syncthreads();
    }
}

}  // namespace

int launch_group_gemv(const GroupCall &c, void *stream)
{
    const int64_t grans = (c.v.N + kGran - 1) / kGran;
    const int all = c.rows >= c.v.experts;
    const dim3 grid((unsigned)grans, (unsigned)(all ? c.v.experts : (int)c.rows));
    if (c.v.gated) group_gemv_kernel<true><<<grid, 32 * kWarps, 0, (cudaStream_t)stream>>>(c, all);
    else group_gemv_kernel<false><<<grid, 32 * kWarps, 0, (cudaStream_t)stream>>>(c, all);
    return cudaGetLastError();
}

}  // namespace uw
