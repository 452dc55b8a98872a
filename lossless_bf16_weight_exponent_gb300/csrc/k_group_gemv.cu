// k_group_gemv.cu - the grouped product for experts with a few rows each (sm_103a): every expert that has rows
// streams its compressed weights once and multiplies them on the tensor pipe (mma.sync m16n8k16, fp32 accumulate).
//
// A CTA owns two granules, 32 outputs (gated: 16 of both matrices), of one expert over all of K; its warps take the
// 64-weight steps in turn.  A lane loads its part of a granule with three 16-byte loads straight into the registers
// of the A operand (the group's form is laid out for that), so the weights pass through no shared memory; one
// shared-memory sum joins the warps, in a fixed order.  The logical k of the instruction is permuted so that a lane's
// pairs are its 16 consecutive weights; X is read in the same order.
//
// Bound by memory, then by the latency of its loads: 1 token top 8 of 64 gated experts of [1408, 2048] takes 20.7 us (69 MB: 10.3
// at the copy rate; 704 CTAs, two an SM, are 2.3 waves with a cold start each), 8 tokens 61 us with 61 % of the DRAM rate, 42 % of
// the integer rate (the rebuild) and 4.6 of a warp's 8 waiting cycles for memory; 16 tokens top 8 of 64 of [2048, 1408] 49.6 us.
// Eight warps a CTA rather than four where the grid is small; registers held to 96 or 80 for a third CTA an SM spilled and
// lost.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "group.cuh"
#include "launch.cuh"
#include "uw_internal.h"

namespace uw {

namespace {

using namespace dev;

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

// step: the step's bytes; at: this lane's place in a granule
__device__ __forceinline__ Part load_part(const uint8_t *step, int gi, int at)
{
    Part p;
    p.s0 = ld_stream(step + gi * 1024 + at);
    p.s1 = ld_stream(step + gi * 1024 + 512 + at);
    p.c = ld_stream(step + kStepSm + gi * 512 + at);
    p.mask = __ldg((const uint16_t *)(step + kStepRec) + gi);
    return p;
}

// rows g and g + 8 of a granule's step as bf16 pairs
__device__ __forceinline__ void rebuild_part(const uint8_t *verb, const Part &p, const uint8_t *step, int gi, int g, int t, uint32_t B,
                                             uint32_t (&a)[8], uint32_t (&b)[8])
{
    rebuild_chunk(p.s0, make_uint2(p.c.x, p.c.y), B, a);
    rebuild_chunk(p.s1, make_uint2(p.c.z, p.c.w), B, b);
    if (p.mask) {
        const StepRec &r = *(const StepRec *)(step + kStepRec);
        uint32_t m[4];
#pragma unroll
        for (int i = 0; i < 4; i++) m[i] = __ldg(&r.mask[i]);
        const uint8_t *vb = verb + (uint64_t)__ldg(&r.first) * 64 + 16 * t;
        const int row = 16 * gi + g;
        if ((p.mask >> g) & 1u) rebuild_chunk_verbatim(p.s0, __ldg((const uint4 *)(vb + (uint64_t)verbatim_rank(m, row) * 64)), a);
        if ((p.mask >> (g + 8)) & 1u)
            rebuild_chunk_verbatim(p.s1, __ldg((const uint4 *)(vb + (uint64_t)verbatim_rank(m, row + 8) * 64)), b);
        __syncwarp();  // the products need the warp together again
    }
}

// The output: bf16; fp32; or fp32 with more than a segment of steps for a warp, whose sums are taken in segments as by tcgen05
// (the tensor pipe cuts low bits off a running sum at every product).  One instance for both types took 21.0 us for 1 token
// where the bf16 one takes 20.7: the fp32 gate's code is in the way.
enum Output { BF16, F32, F32_SEGMENTS };

template <bool GATED, int WARPS, Output OUT>
__global__ void __launch_bounds__(32 * WARPS, 16 / WARPS) group_gemv_kernel(const GroupCall c, int all_experts)
{
    constexpr int NG = 2;  // granules of a CTA: gate and up, or 32 outputs
    constexpr bool SUMS = OUT == F32_SEGMENTS;
    __shared__ float part[WARPS][NG][16][8];
    const GroupView &v = c.v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    pdl_trigger();
    pdl_wait();

    // the expert: blockIdx.y itself, or (fewer rows than experts) the blockIdx.y-th that has rows
    int e = blockIdx.y, lo = 0, hi = 0;
    const int R = (int)c.rows;
    auto off = [&](int i) { return min(max(c.offsets[i], 0), R); };
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
    const uint8_t *steps = v.steps + (((int64_t)e * v.tiles + (vg >> 3)) * v.ksteps + warp) * kStepBytes;
    const int at = chunk_at(g, t);
    const int mine = (v.ksteps - warp + WARPS - 1) / WARPS;  // this warp's steps: warp, warp + WARPS, ...
    uint32_t B[NG];
#pragma unroll
    for (int n = 0; n < NG; n++) B[n] = __ldg(v.base + (GATED ? 2 * e + n : e));

    for (int r0 = lo; r0 < hi; r0 += 8) {
        const uint8_t *sp = steps;
        Part p[NG], pn[NG];
        if (mine > 0)
#pragma unroll
            for (int n = 0; n < NG; n++) pn[n] = load_part(sp, gi + n, at);
        // this lane's row of X (row g of the eight)
        const int r = r0 + g;
        const uint4 *xp = nullptr;
        if (r < hi) {
            const int64_t src = c.row_src ? c.row_src[r] : r;
            if (src >= 0 && src < c.x_rows) xp = (const uint4 *)(c.x + src * c.ldx + 16 * t + warp * kStepW);
        }
        uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0, xn0 = x0, xn1 = x0;
        if (xp && mine > 0) {
            xn0 = xp[0];
            xn1 = xp[1];
        }
        float acc[NG][4], sum[NG][4];
#pragma unroll
        for (int n = 0; n < NG; n++)
#pragma unroll
            for (int i = 0; i < 4; i++) acc[n][i] = sum[n][i] = 0.f;
        for (int i = 0; i < mine; i++) {
            if (SUMS && i % kSegSteps == 0)
#pragma unroll
                for (int n = 0; n < NG; n++)
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        sum[n][j] += acc[n][j];
                        acc[n][j] = 0.f;
                    }
            // the next step's loads leave before this step's products
            const uint8_t *cur = sp;
            sp += (size_t)WARPS * kStepBytes;
#pragma unroll
            for (int n = 0; n < NG; n++) p[n] = pn[n];
            x0 = xn0;
            x1 = xn1;
            if (i + 1 < mine) {
#pragma unroll
                for (int n = 0; n < NG; n++) pn[n] = load_part(sp, gi + n, at);
                if (xp) {
                    xp += WARPS * kStepW / 8;
                    xn0 = xp[0];
                    xn1 = xp[1];
                }
            }
#pragma unroll
            for (int n = 0; n < NG; n++) {
                uint32_t a[8], b[8];
                rebuild_part(v.verb, p[n], cur, gi + n, g, t, B[n], a, b);
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
            for (int i = 0; i < 4; i++) part[warp][n][g + 8 * (i >> 1)][2 * t + (i & 1)] = SUMS ? sum[n][i] + acc[n][i] : acc[n][i];
        __syncthreads();
        for (int at128 = threadIdx.x; at128 < 128; at128 += 32 * WARPS) {
            const int o = at128 & 15, j = at128 >> 4;
            float s[NG];
#pragma unroll
            for (int n = 0; n < NG; n++) {
                s[n] = 0.f;
#pragma unroll
                for (int w = 0; w < WARPS; w++) s[n] += part[w][n][o][j];
            }
            if (r0 + j >= hi) continue;
            if (GATED) s[0] = gated<OUT != BF16>(s[0], s[1]);
#pragma unroll
            for (int n = 0; n < (GATED ? 1 : NG); n++) {
                const int64_t col = ((int64_t)blockIdx.x * (GATED ? 1 : NG) + n) * kGran + o;
                if (col >= v.N) continue;
                const int64_t i = (int64_t)(r0 + j) * c.ldy + col;
                if (OUT == BF16) ((__nv_bfloat16 *)c.y)[i] = __float2bfloat16_rn(s[n]);
                else ((float *)c.y)[i] = s[n];
            }
        }
        __syncthreads();
    }
}

template <int WARPS, Output OUT>
cudaError_t launch_output(const GroupCall &c, dim3 grid, int all, cudaStream_t st)
{
    return c.v.gated ? launch_dependent(group_gemv_kernel<true, WARPS, OUT>, grid, 32 * WARPS, 0, 0, st, c, all)
                     : launch_dependent(group_gemv_kernel<false, WARPS, OUT>, grid, 32 * WARPS, 0, 0, st, c, all);
}

template <int WARPS>
cudaError_t launch_warps(const GroupCall &c, dim3 grid, int all, cudaStream_t st)
{
    if (c.out_bf16) return launch_output<WARPS, BF16>(c, grid, all, st);
    return c.v.ksteps > WARPS * kSegSteps ? launch_output<WARPS, F32_SEGMENTS>(c, grid, all, st) : launch_output<WARPS, F32>(c, grid, all, st);
}

}  // namespace

int launch_group_gemv(const GroupCall &c, void *stream)
{
    // a CTA's two virtual granules: gate and up of 16 outputs, or 32 outputs
    const int64_t pairs = (c.v.granules + 1) / 2;
    const int all = c.rows >= c.v.experts;
    const dim3 grid((unsigned)pairs, (unsigned)(all ? c.v.experts : (int)c.rows));
    // Four CTAs of four warps fit on an SM; with fewer CTAs than that in all, twice the warps over K keep as many bytes on
    // the way (2 experts of [4096, 14336]: 33 us against 55; where CTAs abound, the longer runs of four warps win: 8 tokens,
    // 64 experts of [2048, 1408]: 35 us against 41).
    if ((int64_t)grid.x * grid.y <= 5 * (int64_t)num_sms()) return launch_warps<8>(c, grid, all, (cudaStream_t)stream);
    return launch_warps<4>(c, grid, all, (cudaStream_t)stream);
}

}  // namespace uw
