// k_attend.cu - attention of few new tokens over a cache of keys and values in pages, and the joining of what was cut
// (sm_103a).
//
// An item is 16 query rows - the tokens' query heads that share a key head - against one key head of a sequence.  Eight
// warps of a CTA take 16 keys each of a unit's 128, with maxima, sums and outputs of their own, so nothing is exchanged until
// the item ends; then they are joined in shared memory in three rounds.  A warp brings its own keys and values: tensor
// copies of a page's slots of one head into a ring of three stages (6 KB each way of a head of 128), asked for two steps ahead.
// Products are mma.sync m16n8k16 of bf16: with 16 rows a step is bound by the copies, and the legacy instruction leaves the
// scores in the registers in which the second product wants its operand.
//   scores = q k^T: q in registers for the whole item, k by ldmatrix; p = 2^(scale2 s - m); out += p v, v by ldmatrix.trans
// Probabilities are rounded to bf16 as the operand of the second product (2^-9 of each; their sum is taken before the rounding).
// Slots that no row of the item sees (behind the sequence's length, in front of a window) may hold anything: their scores are
// replaced, their values set to zero in shared memory.
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
constexpr int kRows = 16, kStep = 16, kTile = kStep * kWarps;
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

// a place in the line of units: sequence, item (key head x row tiles + row tile), tile of keys
struct Cursor {
    SeqWork<kRows, kTile> w;
    int s, item, off;          // off: tiles of the item before this one
    int head, rt;              // of the item
    int lo, hi;                // keys that a row of the item may see: [lo, hi)
    __device__ __forceinline__ void enter_item(const AttendCall &a)
    {
        head = item / w.row_tiles;
        rt = item - head * w.row_tiles;
        const int i0 = rt * kRows / a.group, i1 = (int)(min((int64_t)w.q.n * a.group, (int64_t)(rt + 1) * kRows) - 1) / a.group;
        const int64_t p0 = (int64_t)w.q.len - w.q.n;
        hi = a.causal ? (int)min(max(p0 + i1 + 1, (int64_t)0), (int64_t)w.keys) : w.keys;
        lo = a.window ? (int)min(max(p0 + i0 - a.window + 1, (int64_t)0), (int64_t)w.keys) : 0;
    }
    __device__ __forceinline__ void enter_seq(const AttendCall &a)
    {
        for (;; s++) {
            w = seq_work<kRows, kTile>(a, s);
            if (w.row_tiles) break;
        }
        item = 0;
        enter_item(a);
    }
    // the next unit; only called while one is left
    __device__ __forceinline__ void next(const AttendCall &a)
    {
        if (++off < w.tiles) return;
        off = 0;
        if (++item < w.row_tiles * a.kv_heads) enter_item(a);
        else {
            s++;
            enter_seq(a);
        }
    }
    __device__ __forceinline__ int key0(int warp) const { return (w.tile0 + off) * kTile + warp * kStep; }
    __device__ __forceinline__ bool active(int warp) const { return key0(warp) < hi && key0(warp) + kStep > lo; }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attend16_kernel(const __grid_constant__ Args g)
{
    using L = Layout<D>;
    constexpr int KS = D / 16;        // steps of the first product, and pairs of column tiles of the second
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ int64_t sums[kWarps];
    __shared__ int64_t found_at;
    __shared__ int found_s;
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

    // ---------------------------------------------------------------------------------- this CTA's units
    int64_t mine = 0, one = 0;
    for (int s = threadIdx.x; s < a.b.sequences; s += kThreads) {
        one = seq_work<kRows, kTile>(a, s).units(a);
        mine += one;
    }
    int64_t v = mine;
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if (lane == 0) sums[warp] = v;
    __syncthreads();
    int64_t U = 0;
    for (int i = 0; i < kWarps; i++) U += sums[i];
    const int64_t G = gridDim.x;
    const int64_t ua = U * blockIdx.x / G, ub = U * (blockIdx.x + 1) / G;
    Cut cut{0, U, 0, 0, 0, 0};
    if (ua >= ub) {
        if (threadIdx.x == 0) a.cuts[blockIdx.x] = cut;
        return;
    }
    // the sequence with unit ua: 256 at a time in order
    int64_t before = 0;
    for (int s0 = 0; s0 < a.b.sequences; s0 += kThreads) {
        const int s = s0 + threadIdx.x;
        int64_t n = 0;
        if (s < a.b.sequences) n = a.b.sequences <= kThreads ? one : seq_work<kRows, kTile>(a, s).units(a);
        int64_t incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= d) incl += o;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        int64_t excl = before + incl - n;
        for (int i = 0; i < kWarps; i++) {
            if (i < warp) excl += sums[i];
            before += sums[i];
        }
        if (n && excl <= ua && ua < excl + n) {
            found_s = s;
            found_at = excl;
        }
        if (before > ua) break;
    }
    __syncthreads();

    // ---------------------------------------------------------------------------------- cursors
    Cursor use;
    use.s = found_s;
    use.enter_seq(a);
    {
        const int64_t in = ua - found_at;
        use.item = (int)(in / use.w.tiles);
        use.off = (int)(in - (int64_t)use.item * use.w.tiles);
        use.enter_item(a);
    }
    Cursor ld = use;
    int64_t ul = ua;                 // unit of ld
    uint32_t asked = 0, used = 0;    // steps copied, steps consumed
    bool ok = true;
    const uint32_t my_ring = saddr(ring) + warp * kStages * L::stage;
    uint64_t *bars = full + warp * kStages;

    // asks for the warp's next step, if there is one
    auto ask = [&] {
        while (ul < ub && !ld.active(warp)) {
            if (++ul < ub) ld.next(a);
        }
        if (ul >= ub || !ok) return;
        const uint32_t st = asked % kStages;
        if (lane == 0) mbar_expect_tx(&bars[st], L::stage);
        __syncwarp();
        const int boxes = kStep / a.box;
        if (lane < 2 * (D / 64) * boxes) {
            const int is_v = lane & 1, half = (lane >> 1) % (D / 64), bx = lane / (2 * (D / 64));
            const int key = ld.key0(warp) + bx * a.box;
            const int pi = key / a.page_size;
            const int page = key < ld.w.keys ? a.b.pages[(int64_t)ld.s * a.b.ld_pages + pi] : -1;
            tma4d(my_ring + st * L::stage + is_v * L::mat + half * L::half + bx * a.box * 128, is_v ? &g.vm : &g.km, half * 64, key - pi * a.page_size, ld.head,
                  page, saddr(&bars[st]));
        }
        __syncwarp();
        asked++;
        if (++ul < ub) ld.next(a);
    };
    for (int i = 0; i < kStages - 1; i++) ask();

    // ---------------------------------------------------------------------------------- items
    const int gq = lane >> 2, tq = lane & 3;
    int64_t u = ua;
    while (u < ub) {
        const int seg = (int)min((int64_t)use.w.tiles - use.off, ub - u);
        const bool begins = use.off == 0, ends = use.off + seg == use.w.tiles;
        // the two rows of this thread: their queries, and the keys [from, upto) that they see
        uint32_t aq[KS][4];
        int from[2], upto[2];
        const int x0 = use.rt * kRows, xn = (int)min((int64_t)use.w.q.n * a.group - x0, (int64_t)kRows);
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
            if (use.active(warp)) {
                ask();
                const uint32_t st = used % kStages;
                if (ok && !mbar_wait_short(&bars[st], (used / kStages) & 1)) ok = false;
                ok = __all_sync(0xFFFFFFFFu, ok);
                used++;
                const uint32_t ks = my_ring + st * L::stage, vs = ks + L::mat;
                const int key0 = use.key0(warp);
                if (key0 < use.lo || key0 + kStep > use.hi) {
                    // values that no row of the item sees: behind the sequence, or in pages that a window has left
                    const int r0 = max(use.lo - key0, 0), r1 = min(use.hi - key0, kStep);
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
                __syncwarp();
            }
            u++;
            if (k + 1 < seg) use.off++;
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
                float *p = a.part + (2 * (size_t)blockIdx.x + (begins ? 1 : 0)) * slot_floats<kRows, D>();
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const int r = gq + 8 * j;
#pragma unroll
                    for (int n = 0; n < 2 * KS; n++) *(float2 *)(p + r * D + 8 * n + 2 * tq) = make_float2(o[n][2 * j], o[n][2 * j + 1]);
                    if (tq == 0) {
                        p[kRows * D + r] = m[j];
                        p[kRows * D + kRows + r] = l[j];
                    }
                }
                if (begins) {
                    cut.valid = 1;
                    cut.seq = use.s;
                    cut.item = use.item;
                    cut.end = u + (use.w.tiles - seg);
                }
            }
        }
        if (u < ub) use.next(a);
    }
    if (threadIdx.x == 0) a.cuts[blockIdx.x] = cut;
    if (!ok) {
        // what was asked for lands before the block ends
        if (lane == 0) atomicExch(a.status, (int)DEV_TIMEOUT);
        for (uint32_t i = asked > kStages ? asked - kStages : 0; i < asked; i++) mbar_wait_short(&bars[i % kStages], (i / kStages) & 1);
    }
}

// joins the sums of items that were cut: block c those of the item that begins in CTA c's range
template <int R, int D, int K>
__global__ void __launch_bounds__(256) join_kernel(const AttendCall a)
{
    pdl_trigger();
    pdl_wait();
    const Cut cut = a.cuts[blockIdx.x];
    if (!cut.valid) return;
    const int64_t G = gridDim.x;
    const SeqWork<R, K> w = seq_work<R, K>(a, cut.seq);
    const int head = cut.item / w.row_tiles, rt = cut.item - head * w.row_tiles;
    constexpr int kCols = D / 16;        // of a thread
    constexpr size_t kSlot = slot_floats<R, D>();
    const int col = (threadIdx.x % 16) * kCols;
    for (int r = threadIdx.x / 16; r < R; r += 16) {
        const int64_t x = (int64_t)rt * R + r;
        if (x >= (int64_t)w.q.n * a.group) break;
        // slot 1 of this CTA, then slot 0 of those behind it that have units of the item
        auto each = [&](auto f) {
            f(a.part + (2 * (size_t)blockIdx.x + 1) * kSlot);
            for (int64_t c = blockIdx.x + 1; c < G; c++) {
                const int64_t ua = cut.units * c / G, ub = cut.units * (c + 1) / G;
                if (ua >= cut.end) break;
                if (ua < ub) f(a.part + 2 * (size_t)c * kSlot);
            }
        };
        float m = kNegInf, l = 0.f, o[kCols];
#pragma unroll
        for (int i = 0; i < kCols; i++) o[i] = 0.f;
        each([&](const float *p) { m = fmaxf(m, p[R * D + r]); });
        const float b = m == kNegInf ? 0.f : m;
        each([&](const float *p) {
            const float f = exp2_fast(p[R * D + r] - b);
            l += p[R * D + R + r] * f;
#pragma unroll
            for (int i = 0; i < kCols; i += 4) {
                const float4 t = *(const float4 *)(p + (size_t)r * D + col + i);
                o[i] += t.x * f;
                o[i + 1] += t.y * f;
                o[i + 2] += t.z * f;
                o[i + 3] += t.w * f;
            }
        });
        const int i = (int)(x / a.group), h = head * a.group + (int)(x - (int64_t)i * a.group);
        const int64_t row = w.q.first + i;
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
        uint16_t *p = a.out + row * a.ldo + (int64_t)h * D + col;
#pragma unroll
        for (int c = 0; c < kCols; c += 2) *(uint32_t *)(p + c) = pack2(o[c] * inv, o[c + 1] * inv);
        if (a.lse && col == 0) a.lse[row * a.q_heads + h] = l == 0.f ? kNegInf : (m + log2f(l)) * 0.69314718f;
    }
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
    if ((e = launch_dependent(attend16_kernel<D>, dim3((unsigned)ctas), kThreads, Layout<D>::smem, 0, st, g)) != cudaSuccess) return e;
    return launch_dependent(join_kernel<kRows, D, kTile>, dim3((unsigned)ctas), 256, 0, 0, st, g.c);
}

struct Plan {
    bool tc;                     // items of 256 rows on tcgen05, else of 16
    int ctas;
    size_t cuts, bytes;          // bytes of the cuts, of all
};

Plan plan_of(const uw_kv_cache *c, int sequences, int64_t rows, int q_heads)
{
    Plan p;
    p.tc = rows * (q_heads / c->d.kv_heads) > 64 * (int64_t)sequences;
    p.ctas = std::max(1, device_sms());
    p.cuts = (p.ctas * sizeof(Cut) + 255) / 256 * 256;
    const size_t slot = p.tc ? attend_tc_slot_floats(c->d.head_dim) : c->d.head_dim == 128 ? slot_floats<kRows, 128>() : slot_floats<kRows, 64>();
    p.bytes = p.cuts + 2 * (size_t)p.ctas * slot * sizeof(float);
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
    if (q == out) return fail(UW_ERR_INVALID_ARG, "uw_kv_attend: out is q");
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
    a.cuts = (Cut *)workspace;
    a.part = (float *)((uint8_t *)workspace + p.cuts);
    a.status = c->status;
    const int ctas = std::min(p.ctas, num_sms());
    const cudaError_t e = p.tc ? (cudaError_t)launch_attend_tc(c, a, ctas, stream)
                        : c->d.head_dim == 128 ? launch16<128>(c, a, ctas, (cudaStream_t)stream) : launch16<64>(c, a, ctas, (cudaStream_t)stream);
    return e == cudaSuccess ? UW_OK : fail(UW_ERR_CUDA, "uw_kv_attend: launch: %s", cudaGetErrorString(e));
}
