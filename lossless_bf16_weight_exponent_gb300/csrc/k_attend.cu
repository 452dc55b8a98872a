// k_attend.cu - attention of few new tokens over a cache of keys and values in pages, and the joining of what was cut
// (sm_103a).
//
// An item is 16 query rows - the tokens' query heads that share a key head - against one key head of a sequence.  Eight
// warps of a CTA take 16 keys each of a unit's 128, with maxima, sums and outputs of their own, so nothing is exchanged until
// the item ends; then they are joined in shared memory in three rounds.  A warp brings its own keys and values: tensor
// copies of a page's slots of one head into a ring of three stages of its own (8 KB of a head of 128 each, 192 KB an SM), so that
// two are on their way while it works on the third.
// Products are mma.sync m16n8k16 of bf16: with 16 rows a step is bound by the copies, and the legacy instruction leaves the
// scores in the registers in which the second product wants its operand.
//   scores = q k^T: q in registers for the whole item, k by ldmatrix; p = 2^(scale2 s - m); out += p v, v by ldmatrix.trans
// Probabilities are rounded to bf16 as the operand of the second product (by 2^-8 of each at most; their sum is taken before).
// Slots that no row of the item sees (behind the sequence's length, in front of a window) may hold anything: their scores are
// replaced, their values set to zero in shared memory.
//
// Bound by memory: 64 sequences of up to 8191 tokens (8 key heads of 128, 1.15 GB) take 194 us, 5.9 TB/s (197 as ordinary calls), all of 8191
// tokens 348 (6.2 TB/s), one of 131000 93 us.  One token over 8190 takes 15.1 us in a captured chain, 16.6 as ordinary calls, of which the first
// kernel and the hand-over are 5, looking up pages and queries 2, the copies 3 and the joins (of warps, of CTAs, by the last CTA) 4.  Items of 32 rows, two tiles of 16 in
// a CTA with their queries in shared memory, took 305 us for 64 sequences of 24 rows, where tcgen05 takes 266.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "attend.cuh"
#include "dev_async.cuh"
#include "launch.cuh"
#include "uw_internal.h"

namespace uw {

namespace {

using namespace dev;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kRows = 16, kStep = 16;
constexpr int kItem16 = 2;        // what an item costs beside its tiles of keys: the warps' sums joined, its queries (0 to 6 measured: 1 token
                                  // over 8190 takes 14.7, 17.5, 15.1, 15.2, 14.5 us by 0 to 4, 64 sequences 219, 197, 194, 196, 202)
static_assert(kStep * kWarps == kKeys, "a tile is a step of every warp");
constexpr int kStages = 3;
constexpr float kNegInf = -INFINITY;

template <int D>
struct Layout {
    static constexpr uint32_t half = kStep * 128;               // a copy's 64 elements of each key
    static constexpr uint32_t mat = half * (D / 64), stage = 2 * mat;
    static constexpr uint32_t ring = kWarps * kStages * stage;
    static constexpr uint32_t merge = 4 * (D / 16) * 32 * 16;   // half of four warps' outputs
    static constexpr size_t smem = 1024 + ring + merge + 4 * 32 * 16 + kWarps * kStages * 8;
};

struct Args {
    CUtensorMap km, vm;
    AttendCall c;
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void tma4d(uint32_t dst, const CUtensorMap *map, int x, int slot, int head, int page, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(slot), "r"(head), "r"(page), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *(const uint32_t *)&v;
}

using Cur = Cursor<kRows, kItem16>;

__device__ __forceinline__ int key0_of(const Cur &c, int j, int warp) { return (c.k.t0 + c.off + j) * kKeys + warp * kStep; }
// some row of the item sees one of the warp's 16 keys
__device__ __forceinline__ bool active(const Cur &c, int key0) { return key0 < c.k.hi && key0 + kStep > c.k.lo; }

// Joins the parts of an item of xn rows that was cut: those of ranges r0 .. r0 + parts - 1, by the whole CTA.  Four columns of
// a row a thread, and where threads are left, a lot of the parts each; eight parts on their way at a time.
template <int D>
__device__ __forceinline__ void join16(const AttendCall &a, const Cur &c, int r0, int parts, int xn, float4 *buf, float2 *red)
{
    constexpr size_t kSlot = slot_floats<kRows, D>();
    constexpr int kAt = 8;
    const int tid = threadIdx.x, E = xn * (D / 4), lots = max(1, kThreads / E);
    const float *base = a.part + 2 * (size_t)r0 * kSlot;
    for (int e0 = 0; e0 < E; e0 += kThreads) {
        const int e = lots > 1 ? tid % E : e0 + tid, lot = lots > 1 ? tid / E : 0, r = e / (D / 4);
        const bool in = e < E && lot < lots;
        float m = kNegInf, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = lot; in && i0 < parts; i0 += kAt * lots) {
            float pm[kAt], pl[kAt];
            float4 v[kAt];
#pragma unroll
            for (int k = 0; k < kAt; k++) {
                const int i = i0 + k * lots;
                const float *p = base + (2 * (size_t)i + (i == 0)) * kSlot;
                pm[k] = kNegInf;
                pl[k] = 0.f;
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i < parts) {
                    v[k] = __ldcg((const float4 *)p + e);
                    pm[k] = __ldcg(p + kRows * D + r);
                    pl[k] = __ldcg(p + kRows * D + kRows + r);
                }
            }
            float mm = m;
#pragma unroll
            for (int k = 0; k < kAt; k++) mm = fmaxf(mm, pm[k]);
            const float b = mm == kNegInf ? 0.f : mm, f0 = exp2_fast(m - b);
            m = mm;
            l *= f0;
            o.x *= f0;
            o.y *= f0;
            o.z *= f0;
            o.w *= f0;
#pragma unroll
            for (int k = 0; k < kAt; k++) {
                const float f = exp2_fast(pm[k] - b);
                l += pl[k] * f;
                o.x += v[k].x * f;
                o.y += v[k].y * f;
                o.z += v[k].z * f;
                o.w += v[k].w * f;
            }
        }
        if (lots > 1) {
            buf[tid] = o;
            red[tid] = make_float2(m, l);
            __syncthreads();
            if (in && lot == 0) {
                float mm = m;
                for (int i = 1; i < lots; i++) mm = fmaxf(mm, red[i * E + e].x);
                const float b = mm == kNegInf ? 0.f : mm, f0 = exp2_fast(m - b);
                m = mm;
                l *= f0;
                o.x *= f0;
                o.y *= f0;
                o.z *= f0;
                o.w *= f0;
                for (int i = 1; i < lots; i++) {
                    const float2 t = red[i * E + e];
                    const float4 v = buf[i * E + e];
                    const float f = exp2_fast(t.x - b);
                    l += t.y * f;
                    o.x += v.x * f;
                    o.y += v.y * f;
                    o.z += v.z * f;
                    o.w += v.w * f;
                }
            }
        }
        if (in && lot == 0) {
            const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
            const int x = c.rt * kRows + r, tok = x / a.group, h = c.head * a.group + x - tok * a.group, col = 4 * (e % (D / 4));
            const int64_t row = c.w.q.first + tok;
            *(uint2 *)(a.out + row * a.ldo + (int64_t)h * D + col) = make_uint2(pack2(o.x * inv, o.y * inv), pack2(o.z * inv, o.w * inv));
            if (a.lse && col == 0) a.lse[row * a.q_heads + h] = l == 0.f ? kNegInf : (m + log2f(l)) * 0.69314718f;
        }
    }
    __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attend16_kernel(const __grid_constant__ Args g)
{
    using L = Layout<D>;
    constexpr int KS = D / 16;        // steps of the first product, and pairs of column tiles of the second
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ float2 red[kThreads];
    __shared__ int last;
    const AttendCall &a = g.c;
    uint8_t *ring = smem_raw + ((1024u - (saddr(smem_raw) & 1023u)) & 1023u);
    float4 *merge = (float4 *)(ring + L::ring);
    float4 *stats = (float4 *)((uint8_t *)merge + L::merge);   // [4][32]: maxima and sums of two rows
    uint64_t *full = (uint64_t *)(stats + 4 * 32);
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (lane == 0) {
        for (int i = 0; i < kStages; i++) mbar_init(&full[warp * kStages + i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_trigger();
    pdl_wait();
    const int range = blockIdx.x;
    if (range >= a.plan->ranges) return;
    const int64_t C = a.plan->per, U = a.plan->units;
    __syncthreads();

    // ---------------------------------------------------------------------------------- cursors
    Cur use, ld;                     // of the step at work, of the copies
    use.set(a, a.begin[range], range * C, min((range + 1) * C, U));
    ld = use;
    int ld_j = 0;
    uint32_t asked = 0, used = 0;    // steps copied, steps consumed
    bool ok = true;
    const uint32_t my_ring = saddr(ring) + warp * kStages * L::stage;
    uint64_t *bars = full + warp * kStages;

    // asks for the warp's next step, if there is one
    auto ask = [&]() -> bool {
        if (!ok) return false;
        for (;; ld.next(a), ld_j = 0) {
            if (!ld.more()) return false;
            while (ld_j < ld.cnt && !active(ld, key0_of(ld, ld_j, warp))) ld_j++;
            if (ld_j < ld.cnt) break;
        }
        const uint32_t st = asked % kStages;
        if (lane == 0) mbar_expect_tx(&bars[st], L::stage);
        __syncwarp();
        const int boxes = kStep / a.box;
        if (lane < 2 * (D / 64) * boxes) {
            const int is_v = lane & 1, half = (lane >> 1) % (D / 64), bx = lane / (2 * (D / 64));
            const int key = key0_of(ld, ld_j, warp) + bx * a.box;
            const int pi = key / a.page_size;
            const int page = key < ld.w.keys ? a.b.pages[(int64_t)ld.s * a.b.ld_pages + pi] : -1;
            tma4d(my_ring + st * L::stage + is_v * L::mat + half * L::half + bx * a.box * 128, is_v ? &g.vm : &g.km, half * 64, key - pi * a.page_size, ld.head,
                  page, saddr(&bars[st]));
        }
        __syncwarp();
        asked++;
        ld_j++;
        return true;
    };
    while (asked < kStages && ask()) {}

    // ---------------------------------------------------------------------------------- items
    const int gq = lane >> 2, tq = lane & 3;
    for (; use.more(); use.next(a)) {
        const int seg = use.cnt;
        const bool begins = use.begins(), ends = use.ends();
        // the two rows of this thread: their queries, and the keys [from, upto) that they see
        uint32_t aq[KS][4];
        int from[2], upto[2];
        const int x0 = use.rt * kRows, xn = use.rows(a);
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int r = gq + 8 * j;
            const bool in = r < xn;
            const int i = in ? (x0 + r) / a.group : 0;
            const int64_t pos = (int64_t)use.w.q.len - use.w.q.n + i;
            upto[j] = !in ? 0 : a.causal ? (int)min(max(pos + 1, (int64_t)0), (int64_t)use.w.keys) : use.w.keys;
            from[j] = a.window ? (int)max(pos - a.window + 1, (int64_t)0) : 0;
            const uint16_t *p = a.q + (use.w.q.first + i) * a.ldq + (int64_t)(use.head * a.group + (in ? x0 + r - i * a.group : 0)) * D;
#pragma unroll
            for (int k = 0; k < KS; k++) {
                aq[k][j] = in ? *(const uint32_t *)(p + 16 * k + 2 * tq) : 0u;
                aq[k][2 + j] = in ? *(const uint32_t *)(p + 16 * k + 8 + 2 * tq) : 0u;
            }
        }
        float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};
        float o[2 * KS][4];
#pragma unroll
        for (int n = 0; n < 2 * KS; n++) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;

        for (int k = 0; k < seg; k++) {
            const int key0 = key0_of(use, k, warp);
            if (active(use, key0)) {
                while (asked < used + kStages && ask()) {}
                const uint32_t st = used % kStages;
                if (ok && !mbar_wait_short(&bars[st], (used / kStages) & 1)) ok = false;
                ok = __all_sync(0xFFFFFFFFu, ok);
                used++;
                const uint32_t ks = my_ring + st * L::stage, vs = ks + L::mat;
                if (key0 < use.k.lo || key0 + kStep > use.k.hi) {
                    // values that no row of the item sees: behind the sequence, or in pages that a window has left
                    const int r0 = max(use.k.lo - key0, 0), r1 = min(use.k.hi - key0, kStep);
                    for (int i = lane; i < kStep * (D / 8); i += 32) {
                        const int row = i / (D / 8), c = i % (D / 8);
                        if (row >= r0 && row < r1) continue;
                        *(uint4 *)(ring + (vs - saddr(ring)) + (c >> 3) * L::half + row * 128 + ((c & 7) ^ (row & 7)) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                }
                float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                const int mi = lane >> 3, mr = lane & 7;
#pragma unroll
                for (int q = 0; q < KS; q++) {
                    const int row = (mi >> 1) * 8 + mr, c = 2 * q + (mi & 1);
                    uint32_t b[4];
                    ldsm4(b, ks + (c >> 3) * L::half + row * 128 + ((c & 7) ^ mr) * 16);
                    mma16816(s[0], aq[q], b[0], b[1]);
                    mma16816(s[1], aq[q], b[2], b[3]);
                }
                float mx[2] = {kNegInf, kNegInf};
#pragma unroll
                for (int n = 0; n < 2; n++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int key = key0 + 8 * n + 2 * tq + (e & 1), j = e >> 1;
                        s[n][e] = key >= from[j] && key < upto[j] ? s[n][e] * a.scale2 : kNegInf;
                        mx[j] = fmaxf(mx[j], s[n][e]);
                    }
                float base[2], keep[2];
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xFFFFFFFFu, mx[j], 1));
                    mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xFFFFFFFFu, mx[j], 2));
                    mx[j] = fmaxf(mx[j], m[j]);
                    base[j] = mx[j] == kNegInf ? 0.f : mx[j];
                    keep[j] = exp2_fast(m[j] - base[j]);
                }
                if (__any_sync(0xFFFFFFFFu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
                    for (int n = 0; n < 2 * KS; n++) {
                        o[n][0] *= keep[0];
                        o[n][1] *= keep[0];
                        o[n][2] *= keep[1];
                        o[n][3] *= keep[1];
                    }
                    l[0] *= keep[0];
                    l[1] *= keep[1];
                    m[0] = mx[0];
                    m[1] = mx[1];
                }
#pragma unroll
                for (int n = 0; n < 2; n++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        s[n][e] = exp2_fast(s[n][e] - base[e >> 1]);
                        l[e >> 1] += s[n][e];
                    }
                const uint32_t p[4] = {pack2(s[0][0], s[0][1]), pack2(s[0][2], s[0][3]), pack2(s[1][0], s[1][1]), pack2(s[1][2], s[1][3])};
#pragma unroll
                for (int q = 0; q < KS; q++) {
                    const int row = (mi & 1) * 8 + mr, c = 2 * q + (mi >> 1);
                    uint32_t b[4];
                    ldsm4t(b, vs + (c >> 3) * L::half + row * 128 + ((c & 7) ^ mr) * 16);
                    mma16816(o[2 * q], p, b[0], b[1]);
                    mma16816(o[2 * q + 1], p, b[2], b[3]);
                }
                // the stage's reads are done before the next copy into it (the async proxy) is asked for
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            }
        }

        // ------------------------------------------------------------------------------ the warps' sums
        float f_other[2];
#pragma unroll
        for (int h = 4; h; h >>= 1) {
            // warps h .. 2h - 1 join warps 0 .. h - 1; half of the columns at a time where all do not fit
            constexpr int kParts = 2;
            float keep[2] = {1.f, 1.f};
#pragma unroll
            for (int part = 0; part < kParts; part++) {
                __syncthreads();
                if (warp >= h && warp < 2 * h) {
                    if (part == 0) stats[(warp - h) * 32 + lane] = make_float4(m[0], m[1], l[0], l[1]);
#pragma unroll
                    for (int n = 0; n < KS; n++) {
                        const float *x = o[part * KS + n];
                        merge[((warp - h) * KS + n) * 32 + lane] = make_float4(x[0], x[1], x[2], x[3]);
                    }
                }
                __syncthreads();
                if (warp < h) {
                    if (part == 0) {
                        const float4 t = stats[warp * 32 + lane];
                        const float mo[2] = {t.x, t.y}, lo[2] = {t.z, t.w};
#pragma unroll
                        for (int j = 0; j < 2; j++) {
                            const float mm = fmaxf(m[j], mo[j]), b = mm == kNegInf ? 0.f : mm;
                            keep[j] = exp2_fast(m[j] - b);
                            f_other[j] = exp2_fast(mo[j] - b);
                            l[j] = l[j] * keep[j] + lo[j] * f_other[j];
                            m[j] = mm;
                        }
                    }
#pragma unroll
                    for (int n = 0; n < KS; n++) {
                        float *x = o[part * KS + n];
                        const float4 t = merge[(warp * KS + n) * 32 + lane];
                        x[0] = x[0] * keep[0] + t.x * f_other[0];
                        x[1] = x[1] * keep[0] + t.y * f_other[0];
                        x[2] = x[2] * keep[1] + t.z * f_other[1];
                        x[3] = x[3] * keep[1] + t.w * f_other[1];
                    }
                }
            }
        }
        if (warp == 0) {
#pragma unroll
            for (int j = 0; j < 2; j++) {
                l[j] += __shfl_xor_sync(0xFFFFFFFFu, l[j], 1);
                l[j] += __shfl_xor_sync(0xFFFFFFFFu, l[j], 2);
            }
            if (begins && ends) {
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const int r = gq + 8 * j;
                    if (r >= xn) continue;
                    const int i = (x0 + r) / a.group, h = use.head * a.group + (x0 + r - i * a.group);
                    const int64_t row = use.w.q.first + i;
                    const float inv = l[j] > 0.f ? 1.f / l[j] : l[j] == 0.f ? 0.f : l[j];
                    uint16_t *p = a.out + row * a.ldo + (int64_t)h * D;
#pragma unroll
                    for (int n = 0; n < 2 * KS; n++) *(uint32_t *)(p + 8 * n + 2 * tq) = pack2(o[n][2 * j] * inv, o[n][2 * j + 1] * inv);
                    if (a.lse && tq == 0) a.lse[row * a.q_heads + h] = l[j] == 0.f ? kNegInf : (m[j] + log2f(l[j])) * 0.69314718f;
                }
            } else {
                float *p = a.part + (2 * (size_t)range + (begins ? 1 : 0)) * slot_floats<kRows, D>();
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const int r = gq + 8 * j;
                    if (r >= xn) continue;
#pragma unroll
                    for (int n = 0; n < 2 * KS; n++) *(float2 *)(p + r * D + 8 * n + 2 * tq) = make_float2(o[n][2 * j], o[n][2 * j + 1]);
                    if (tq == 0) {
                        p[kRows * D + r] = m[j];
                        p[kRows * D + kRows + r] = l[j];
                    }
                }
            }
        }
        if (!begins || !ends) {
            // the part that comes last joins them all
            const int r0 = use.first_range(C), parts = use.last_range(C) - r0 + 1;
            if (warp == 0) {
                __threadfence();
                __syncwarp();
                if (lane == 0) last = atomicAdd(&a.arrived[2 * r0], 1) == parts - 1;
            }
            __syncthreads();
            if (last) {
                __threadfence();
                join16<D>(a, use, r0, parts, xn, merge, red);
            }
        }
    }
    if (!ok) {
        // what was asked for lands before the block ends
        if (lane == 0) atomicExch(a.status, (int)DEV_TIMEOUT);
        for (uint32_t i = asked > kStages ? asked - kStages : 0; i < asked; i++) mbar_wait_short(&bars[i % kStages], (i / kStages) & 1);
    }
}

// ------------------------------------------------------------------------------------------------ the first kernel
constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr int kLineShared = 2048;      // sequences whose places in the line fit in shared memory

// Sums over the threads in front of this one; all: over all threads.  sums: [kPlanWarps], free for the next call after a barrier.
template <typename T>
__device__ __forceinline__ T scan_before(T v, T *sums, T &all)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    T x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T o = __shfl_up_sync(0xFFFFFFFFu, x, d);
        if (lane >= d) x += o;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    T y = sums[lane];                  // every warp adds them up
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T o = __shfl_up_sync(0xFFFFFFFFu, y, d);
        if (lane >= d) y += o;
    }
    const T front = __shfl_sync(0xFFFFFFFFu, y, warp ? warp - 1 : 0);
    all = __shfl_sync(0xFFFFFFFFu, y, 31);
    return (warp ? front : (T)0) + x - v;
}

// the last i in [lo, hi) for which at(i) <= x; at(lo) <= x
template <typename F, typename T>
__device__ __forceinline__ int last_at(int lo, int hi, T x, F at)
{
    int n = hi - lo;
    while (n > 1) {
        const int h = n >> 1;
        if (at(lo + h) <= x) {
            lo += h;
            n -= h;
        } else {
            n = h;
        }
    }
    return lo;
}

// The line's length, the ranges - one for each of the next kernel's CTAs - and where they begin; one CTA.  This form holds every
// tile of rows in shared memory, up to kSmallSeqs sequences and kSmallTiles tiles: a tile or a few a thread, a sum over the
// threads, two searches for each range (3 us where the form below takes 12, for the 128 tiles of 8191 tokens).
// Ranges taken in turn by CTAs that are done, up to six for each, were no faster: 64 sequences of up to 8191 tokens took 213 us
// against 200, one token over 131000 122 against 95, as each range ends with sums to be joined.
constexpr int kSmallSeqs = 512, kSmallTiles = 4096;

template <int R, int kItem>
__global__ void __launch_bounds__(kPlanThreads) plan_small_kernel(const AttendCall a, int ctas)
{
    __shared__ int64_t pre[kSmallTiles + 1];       // of a key head's line, in front of each tile of rows
    __shared__ int n_s[kSmallSeqs], len_s[kSmallSeqs], first_s[kSmallSeqs], tile0[kSmallSeqs + 1];
    __shared__ int64_t sums[kPlanWarps];
    __shared__ int isums[kPlanWarps];
    const int tid = threadIdx.x, S = a.b.sequences;
    pdl_trigger();
    pdl_wait();
    Seq w{};
    if (tid < S) {
        w = seq_at<R>(a, tid);
        n_s[tid] = w.q.n;
        len_s[tid] = w.q.len;
        first_s[tid] = w.q.first;
    }
    int T;
    const int mine = scan_before(w.row_tiles, isums, T);
    T = min(T, kSmallTiles);           // as the host has counted them, unless `starts` is not ascending
    if (tid < S) tile0[tid] = min(mine, T);
    if (tid == 0) {
        tile0[S] = T;
        pre[0] = 0;
    }
    __syncthreads();
    const int per = (T + kPlanThreads - 1) / kPlanThreads, f0 = tid * per, f1 = min(f0 + per, T);
    int64_t cost = 0;
    if (f0 < f1) {
        int s = last_at(0, S, f0, [&](int i) { return tile0[i]; });
        for (int f = f0; f < f1; f++) {
            while (f >= tile0[s + 1]) s++;
            const int tiles = tile0[s + 1] - tile0[s];
            cost += span_of<R>(a, n_s[s], len_s[s], min(len_s[s], a.b.capacity), tile_of(f - tile0[s], tiles)).nt + kItem;
            pre[f + 1] = cost;
        }
    }
    int64_t P;
    const int64_t front = scan_before(cost, sums, P);
    for (int f = f0; f < f1; f++) pre[f + 1] += front;
    __syncthreads();
    const int64_t U = P * a.kv_heads, C = max((U + ctas - 1) / ctas, (int64_t)1);
    const int N = (int)((U + C - 1) / C);
    if (tid == 0) *a.plan = PlanHead{U, C, N};
    for (int i = tid; i < 2 * N; i += kPlanThreads) a.arrived[i] = 0;
    for (int r = tid; r < N; r += kPlanThreads) {
        const int64_t ua = r * C;
        const int s = last_at(0, S, ua, [&](int i) { return pre[tile0[i]] * a.kv_heads; });
        const int64_t p0 = pre[tile0[s]], w1 = pre[tile0[s + 1]] - p0, in = ua - p0 * a.kv_heads;
        const int head = (int)(in / w1);
        const int64_t at = in - head * w1;
        const int f = last_at(tile0[s], tile0[s + 1], at, [&](int i) { return pre[i] - p0; });
        a.begin[r] = Start{ua - (at - (pre[f] - p0)), s, head, f - tile0[s], KvSeq{first_s[s], n_s[s], len_s[s]}};
    }
}

// units of sequence s for one key head, by the whole warp, a sequence a lane (s past the end: none)
template <int R, int kItem>
__device__ __forceinline__ int64_t units_of(const AttendCall &a, int s)
{
    const int lane = threadIdx.x & 31;
    Seq w{};
    if (s < a.b.sequences) w = seq_at<R>(a, s);
    int64_t u = 0;
    const bool many = w.row_tiles > 2;
    if (!many)
        for (int rt = 0; rt < w.row_tiles; rt++) u += span_of<R>(a, w.q.n, w.q.len, w.keys, rt).nt + kItem;
    unsigned left = __ballot_sync(0xFFFFFFFFu, many);
    while (left) {
        const int src = __ffs(left) - 1;
        left &= left - 1;
        const int n = __shfl_sync(0xFFFFFFFFu, w.q.n, src), len = __shfl_sync(0xFFFFFFFFu, w.q.len, src);
        const int keys = __shfl_sync(0xFFFFFFFFu, w.keys, src), tiles = __shfl_sync(0xFFFFFFFFu, w.row_tiles, src);
        int64_t x = 0;
        for (int rt = lane; rt < tiles; rt += 32) x += span_of<R>(a, n, len, keys, rt).nt + kItem;
#pragma unroll
        for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
        if (lane == src) u = x;
    }
    return u;
}

// The same for any number of sequences and tiles, which are measured a warp at a time and again for each range.
template <int R, int kItem>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const AttendCall a, int ctas)
{
    __shared__ int64_t line_s[kLineShared + 1];
    __shared__ int64_t sums[kPlanWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, S = a.b.sequences;
    int64_t *line = S <= kLineShared ? line_s : a.line;   // before each sequence
    pdl_trigger();
    pdl_wait();
    int64_t before = 0;
    for (int s0 = 0; s0 < S; s0 += kPlanThreads) {
        const int s = s0 + threadIdx.x;
        const int64_t n = units_of<R, kItem>(a, s) * a.kv_heads;
        __syncthreads();
        int64_t all;
        const int64_t front = scan_before(n, sums, all);
        if (s < S) line[s + 1] = before + front + n;
        before += all;
    }
    if (threadIdx.x == 0) line[0] = 0;
    __syncthreads();
    const int64_t U = before, C = max((U + ctas - 1) / ctas, (int64_t)1);
    const int N = (int)((U + C - 1) / C);
    if (threadIdx.x == 0) *a.plan = PlanHead{U, C, N};
    for (int i = threadIdx.x; i < 2 * N; i += kPlanThreads) a.arrived[i] = 0;
    for (int r0 = 0; r0 < N; r0 += kPlanThreads) {
        const int r = r0 + lane * kPlanWarps + warp;   // neighbours on different warps, which work through theirs one by one
        // the sequence: the last whose place is at or before the range's
        const int64_t ua = r * C;
        const int lo = last_at(0, r < N ? S : 1, ua, [&](int i) { return line[i]; });
        Seq w{};
        Start f{};
        f.s = lo;
        int64_t at = 0;                // of the range in the head's part of the line
        if (r < N) {
            w = seq_at<R>(a, lo);
            f.q = w.q;
            const int64_t per = (line[lo + 1] - line[lo]) / a.kv_heads, in = ua - line[lo];
            f.head = (int)(in / per);
            at = in - f.head * per;
            f.at = ua - at;
        }
        const bool many = w.row_tiles > 1;
        unsigned left = __ballot_sync(0xFFFFFFFFu, many);
        while (left) {
            const int src = __ffs(left) - 1;
            left &= left - 1;
            const int qn = __shfl_sync(0xFFFFFFFFu, w.q.n, src), len = __shfl_sync(0xFFFFFFFFu, w.q.len, src);
            const int keys = __shfl_sync(0xFFFFFFFFu, w.keys, src), tiles = __shfl_sync(0xFFFFFFFFu, w.row_tiles, src);
            int64_t rest = __shfl_sync(0xFFFFFFFFu, at, src);
            for (int i0 = 0; i0 < tiles; i0 += 32) {
                const int nt = i0 + lane < tiles ? span_of<R>(a, qn, len, keys, tile_of(i0 + lane, tiles)).nt + kItem : 0;
                int64_t x = nt;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int64_t o = __shfl_up_sync(0xFFFFFFFFu, x, d);
                    if (lane >= d) x += o;
                }
                const int64_t all = __shfl_sync(0xFFFFFFFFu, x, 31);
                if (rest < all) {
                    const unsigned hit = __ballot_sync(0xFFFFFFFFu, rest < x);   // the first of them has it
                    const int l = __ffs(hit) - 1;
                    const int64_t in_item = rest - (__shfl_sync(0xFFFFFFFFu, x, l) - __shfl_sync(0xFFFFFFFFu, nt, l));
                    if (lane == src) {
                        f.i = i0 + l;
                        f.at = ua - in_item;
                    }
                    break;
                }
                rest -= all;
            }
        }
        if (r < N) a.begin[r] = f;
    }
}

template <int R, int kItem>
cudaError_t launch_plan(const AttendCall &a, int ctas, cudaStream_t st)
{
    const bool small = a.b.sequences <= kSmallSeqs && (int64_t)a.b.rows * a.group / R + a.b.sequences <= kSmallTiles;
    return launch_dependent(small ? plan_small_kernel<R, kItem> : plan_kernel<R, kItem>, dim3(1), kPlanThreads, 0, 0, st, a, ctas);
}

template <int D>
cudaError_t launch16(const uw_kv_cache *c, const AttendCall &call, int ctas, cudaStream_t st)
{
    static OncePerDevice once;
    cudaError_t e = allow_shared(once, attend16_kernel<D>, Layout<D>::smem);
    if (e != cudaSuccess) return e;
    Args g;
    g.km = c->k16;
    g.vm = c->v16;
    g.c = call;
    g.c.box = c->box16;
    if ((e = launch_plan<kRows, kItem16>(call, ctas, st)) != cudaSuccess) return e;
    return launch_dependent(attend16_kernel<D>, dim3((unsigned)ctas), kThreads, Layout<D>::smem, 0, st, g);
}

// How a call's workspace is laid out, and which kernel it takes.
struct Plan {
    int rows;                    // of an item: 16, or 128 or 256 on tcgen05
    int ctas;
    size_t begin, arrived, line, part, bytes;
};

Plan plan_of(const uw_kv_cache *c, int sequences, int64_t rows, int q_heads)
{
    Plan p;
    const int64_t each = rows * (q_heads / c->d.kv_heads);
    // Rows of a sequence on average; in us, for 64 sequences of up to 8191 tokens before the new ones, key heads of 4 query heads, by
    // items of 16, of 128 and of 256 rows:
    //   new tokens       2     4     5     8    32    48     one sequence of 8190 + 8   509 x 8 rows over 7171   2047 x 4 rows
    //   16             201   206   398   414  1579  2346                        23.2                      838             322
    //   128            262   263   264   253   256   494                        33.6                      140            62.4
    //   256            270   270   271   259   259   311                        34.1                      115            55.8
    // One kernel for a whole call, by its average; sequences that bring nothing count too.  The table is of batches of equal sequences; what the
    // rule makes of mixed ones, key heads of 4 query heads, in us in a captured chain: 256 single tokens over up to 8191 and a chunk of 512 take
    // 703 (items of 16 rows; alone 658 and, over 4000, 52), 100 of them and a chunk of 300 344 (alone 308 and 43); but a step of 256 places of which
    // one brings 512 tokens and the others nothing takes 51 where those 512 alone, by items of 256, take 25; and 46 single tokens beside two chunks of
    // 755 go by items of 256 rows, 8 of which hold queries.
    p.rows = each <= 16 * (int64_t)sequences ? 16 : each <= 128 * (int64_t)sequences ? 128 : 256;
    p.ctas = std::max(1, device_sms());
    const size_t ranges = (size_t)p.ctas;
    const auto up = [](size_t n) { return (n + 255) / 256 * 256; };
    p.begin = up(sizeof(PlanHead));
    p.arrived = p.begin + up(ranges * sizeof(Start));
    p.line = p.arrived + up(2 * ranges * sizeof(int));
    p.part = p.line + (sequences > kLineShared ? up(((size_t)sequences + 1) * sizeof(int64_t)) : 0);
    const size_t slot = (size_t)p.rows * (c->d.head_dim + 2);   // slot_floats
    p.bytes = p.part + 2 * ranges * slot * sizeof(float);
    return p;
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

uw_status check_heads(const uw_kv_cache *c, int sequences, int64_t rows, int q_heads, const char *who)
{
    if (rows < 0 || rows > ((int64_t)1 << 31) - 1024 || sequences < 1 || sequences > 65536 || q_heads < 1 || q_heads % c->d.kv_heads ||
        q_heads / c->d.kv_heads > 64 || rows * (q_heads / c->d.kv_heads) > ((int64_t)1 << 31) - 65536)
        return fail(UW_ERR_SHAPE, "%s: %d sequences, rows=%lld, %d query heads over %d", who, sequences, (long long)rows, q_heads, c->d.kv_heads);
    return UW_OK;
}

}  // namespace

int launch_attend_plan(const AttendCall &a, int rows, int ctas, void *stream)
{
    return rows == 128 ? launch_plan<128, kItemTc>(a, ctas, (cudaStream_t)stream) : launch_plan<256, kItemTc>(a, ctas, (cudaStream_t)stream);
}

}  // namespace uw

using namespace uw;

extern "C" uw_status uw_kv_attend_workspace_size(const uw_kv_cache *c, int sequences, int64_t rows, int q_heads, size_t *bytes)
{
    clear_error();
    if (!c || !bytes) return fail(UW_ERR_INVALID_ARG, "uw_kv_attend_workspace_size: NULL argument");
    const uw_status s = check_heads(c, sequences, rows, q_heads, "uw_kv_attend_workspace_size");
    if (s != UW_OK) return s;
    *bytes = plan_of(c, sequences, rows, q_heads).bytes;
    return UW_OK;
}

extern "C" uw_status uw_kv_attend(const uw_kv_cache *c, const uw_kv_batch *b, int64_t rows, const uint16_t *q, int64_t ldq, int q_heads, float scale,
                                  int causal, int64_t window, uint16_t *out, int64_t ldo, float *lse, void *workspace, size_t ws_bytes,
                                  uw_stream stream)
{
    clear_error();
    if (!c) return fail(UW_ERR_INVALID_ARG, "uw_kv_attend: NULL cache");
    AttendCall a{};
    uw_status s = check_kv_batch(c, b, rows, &a.b, "uw_kv_attend");
    if (s != UW_OK) return s;
    if ((s = check_heads(c, b->sequences, rows, q_heads, "uw_kv_attend")) != UW_OK) return s;
    if (!std::isfinite(scale) || !std::isfinite(scale * 1.4426950408889634f)) return fail(UW_ERR_INVALID_ARG, "uw_kv_attend: scale %g", (double)scale);
    if (window < 0 || (window && !causal)) return fail(UW_ERR_INVALID_ARG, "uw_kv_attend: window %lld", (long long)window);
    const int64_t dense = (int64_t)q_heads * c->d.head_dim, most = (int64_t)1 << 39;
    a.ldq = ldq ? ldq : dense;
    a.ldo = ldo ? ldo : dense;
    if (a.ldq % 8 || a.ldo % 8 || (rows > 1 && (a.ldq < dense || a.ldo < dense || a.ldq >= most || a.ldo >= most)))
        return fail(UW_ERR_SHAPE, "uw_kv_attend: ldq=%lld ldo=%lld", (long long)ldq, (long long)ldo);
    if (rows == 0) return UW_OK;
    if (!q || !out || !aligned16(q) || !aligned16(out) || ((uintptr_t)lse & 3)) return fail(UW_ERR_INVALID_ARG, "uw_kv_attend: q or out NULL, or a pointer not aligned");
    // a row's queries are read by every CTA that has a part of its keys, at its own time
    if (rows_overlap({q, a.ldq * 2, dense * 2}, {out, a.ldo * 2, dense * 2}, rows)) return fail(UW_ERR_INVALID_ARG, "uw_kv_attend: out overlaps q");
    if ((s = check_kv_device(c, "uw_kv_attend")) != UW_OK) return s;
    const Plan p = plan_of(c, b->sequences, rows, q_heads);
    if (ws_bytes < p.bytes || !workspace) return fail(UW_ERR_WORKSPACE, "uw_kv_attend: workspace of %zu bytes, %zu needed", ws_bytes, p.bytes);
    if (!aligned16(workspace)) return fail(UW_ERR_INVALID_ARG, "uw_kv_attend: workspace not 16-byte aligned");
    a.q = q;
    a.out = out;
    a.lse = lse;
    a.q_heads = q_heads;
    a.kv_heads = c->d.kv_heads;
    a.group = q_heads / a.kv_heads;
    a.page_size = c->d.page_size;
    a.causal = causal != 0;
    a.window = (int)std::min<int64_t>(window, ((int64_t)1 << 31) - 1);
    a.scale2 = scale * 1.4426950408889634f;
    uint8_t *ws = (uint8_t *)workspace;
    a.plan = (PlanHead *)ws;
    a.begin = (Start *)(ws + p.begin);
    a.arrived = (int *)(ws + p.arrived);
    a.line = (int64_t *)(ws + p.line);
    a.part = (float *)(ws + p.part);
    a.status = c->status;
    const int ctas = std::min(p.ctas, num_sms());
    const cudaError_t e = p.rows > kRows ? (cudaError_t)launch_attend_tc(c, a, p.rows, ctas, stream)
                        : c->d.head_dim == 128 ? launch16<128>(c, a, ctas, (cudaStream_t)stream) : launch16<64>(c, a, ctas, (cudaStream_t)stream);
    return e == cudaSuccess ? UW_OK : fail(UW_ERR_CUDA, "uw_kv_attend: launch: %s", cudaGetErrorString(e));
}
