// k_group_tc.cu - the grouped product for experts with many rows (sm_103a): weights rebuilt into tensor memory, tcgen05.
//
// Many rows run on pairs of CTAs (cta_group::2).  A unit is two weight tiles (2 x 128 virtual rows of an expert's matrices,
// one for each CTA) times up to 192 of the expert's rows of X, over all of K; each CTA rebuilds its own tile, holds half of
// the X tile and the accumulator of its 128 rows.  On a single CTA every SM took in 36.9 KB a step and the copies from L2
// bounded it at 59 bytes a cycle; a pair takes 24.6.  Few rows run on single CTAs, up to 64 rows of X a unit, with a weight
// ring of twelve stages: their weights' bytes in flight bound them.  Persistent CTAs take every gridDim-th unit of the list
// (expert, row tile of X, weight tile), the weight tile innermost so that CTAs that run together share their rows of X.
// The list follows from the offsets, which each CTA reads on the device.
//
// Roles of the 28 warps:
//   - 0-15, four groups of four: group i % 4 rebuilds step i (128 rows x 64 weights).  Thread = row: four 16-byte and
//     four 8-byte reads of shared memory without bank conflicts, 32 bf16 pairs, one tcgen05.st of 32 columns.  The
//     A operand never passes through shared memory, which the X tiles need.
//   - 16, 23: bulk copies of the steps (12 KB and the record, one run of memory) and their verbatim runs, alternate
//     steps each;
//   - 17: four tcgen05.mma a step (M = 128, or 256 on a pair; N = rows of X up to a multiple of 16, or 32; K = 16), A from
//     tensor memory.  On a pair the first CTA issues, and its barriers count what both CTAs bring;
//   - 18-22: X tiles [rows x 64] bf16 in the 128-byte swizzle, a warp for each stage of the ring.  Rows in order come in
//     tensor copies of 32 rows, rows with sources in tensor copies that gather four (a source outside X reads zeros);
//   - 24-27: the epilogue of a finished unit, a warp per lane quarter of tensor memory.  In a gated tile lanes 0-15 of a
//     warp hold gate rows and lanes 16-31 the up rows that belong to them: eight exchanges between the halves per 16
//     columns give each lane both factors of eight outputs.
// Tensor memory: two accumulators of 192 columns, so that a unit's epilogue runs under the next unit's products, and four
// slots of 32 columns for A (64 and eight in the shape for few rows).  A sum of segments takes 128 columns beside two
// accumulators of 128.
//
// Measured on weights of which 1.1 % of the runs are verbatim (4096 tokens top 8 of 64 gated experts of [1408, 2048]): 355 us,
// 1.07 PFLOP/s, and 341 on weights without such runs, which a warp with one among its 32 rows rebuilds twice.  Of a form that
// took 325 there, the rebuild left out took 278, the epilogue left out 301, both 261.  4096 tokens of [2048, 1408]: 167 us.
// 333 tokens top 2 of 8 gated experts of [14336, 4096]: 246 to 257 us, 5.6 to 5.8 TB/s of compressed weights.  128 tokens top 8
// of 64 experts of [2048, 1408]: 57 us, 4.9 TB/s.  fp32 from segments: 494 us for the first, 240 for the second; on weights without
// verbatim runs 477 and 224.
// Every wait is bounded; when one runs out the kernel latches DEV_TIMEOUT, waits for its copies and products in flight,
// frees its tensor memory and ends.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "group.cuh"
#include "launch.cuh"
#include "uw_internal.h"

namespace uw {

namespace {

using namespace dev;

constexpr int kWarps = 28, kThreads = 32 * kWarps;
constexpr int kXWarps = 5;
constexpr int kVCs = 8;                       // verbatim runs of a step staged with it (beyond: global loads)
constexpr uint32_t kVOff = kStepRec + 128;    // a stage: the step with its record, then its verbatim runs
constexpr uint32_t kWStage = kVOff + kVCs * 64;

// The shapes: 192 rows of X per unit at most on a pair of CTAs, each with half of the X tile; 64 on one, where the weights
// have most of shared memory: their bytes in flight bound a product of few rows; 128 on a pair for an fp32 output of several
// segments, whose sums take a third region of tensor memory.
template <int BN_, bool PAIR_, bool SUMS_>
struct Shape {
    static constexpr int BN = BN_;
    static constexpr bool PAIR = PAIR_, SUMS = SUMS_;  // SUMS: the segments of an fp32 output are summed in tensor memory
    // roles: rebuild groups of four warps, a copying warp, the issuing warp, the X warps, another copying warp, the
    // epilogue's warps (the first a multiple of four: warp % 4 is the lane quarter of tensor memory)
    static constexpr int Groups = 4, EpiWarps = 4;
    static constexpr int ProdWarp = 4 * Groups, MmaWarp = ProdWarp + 1, XWarp0 = ProdWarp + 2, ProdWarp2 = XWarp0 + kXWarps;
    static constexpr int EpiWarp0 = ProdWarp2 + 1;
    static_assert(EpiWarp0 % 4 == 0 && EpiWarp0 + EpiWarps == kWarps, "roles");
    static constexpr int SX = kXWarps, SW = 12, SA = BN == 64 ? 8 : 4;   // stages of X, of the weights; A slots
    static constexpr int XRows = PAIR ? BN / 2 : BN;                      // rows of the X tile in a CTA
    static constexpr uint32_t XStage = XRows * 128;
    static constexpr int RunCol = 2 * BN;     // tensor memory: two accumulators, the sums of segments, the A slots of 32 columns
    static constexpr int ACol = (SUMS ? 3 : 2) * BN;
    static constexpr size_t smem = 1024 + (size_t)SX * XStage + (size_t)SW * kWStage + 512 + 2 * 4 * (kMaxExperts + 4) + 4 * SX * XRows;
    static_assert(smem <= 227 * 1024, "shared memory");
    // A stage of the weight ring belongs to one rebuild group and one copying warp for good.  Copies land out of order,
    // so a group that waited for a stage last read by another group could be a whole turn ahead of a copy that has not
    // landed, where the barrier's parity is the same as of the turn it waits for.  (The A slots need no such rule: products
    // complete in order, and a group that is at step q has seen step q - Groups - SA done.)
    static_assert(SW % Groups == 0 && SW % 2 == 0 && SA >= Groups, "rings");
    static_assert(ACol + 32 * SA <= 512 && XRows % 32 == 0, "layout");
    static_assert((2 * (SW + SX + SA) + 5) * 8 + 8 <= 512, "barriers");
};
static_assert(kWStage % 128 == 0, "layout");

struct TcArgs {
    CUtensorMap tm_x;  // X [x_rows, K] bf16, box {64, 32} or (sources) {64, 1}, 128-byte swizzle
    GroupCall c;
};

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// true in one thread of the (whole) warp
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// the address, for both CTAs of a pair, of what lies at this address in the first one's shared memory
__device__ __forceinline__ uint32_t in_first(uint32_t addr)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(addr));
    return a;
}

// Tensor copies into this CTA's shared memory; on a pair the barrier is either CTA's.
// four rows of a map whose box is one row high (a row past the end reads zeros)
template <bool PAIR>
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, int x, const int4 &y, uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, "
            "%4, %5, %6}], [%7];" ::"r"(dst),
            "l"(map), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
            "%5, %6}], [%7];" ::"r"(dst),
            "l"(map), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w), "r"(bar)
            : "memory");
}

// a box of rows
template <bool PAIR>
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(
                dst),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem descriptor].  On a pair of CTAs (cta_group::2) D has 256 rows, each CTA's tensor memory holds
// its 128 of A and D, each CTA's shared memory half of the rows of B; one thread of the first CTA issues.
template <bool PAIR>
__device__ __forceinline__ void mma_of(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc)
{
    if constexpr (PAIR)
        asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
                         d_tmem),
                     "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
                     : "memory");
    else
        mma_ts(d_tmem, a_tmem, b, idesc, acc);
}

// arrive on this barrier (of a pair: in both CTAs) once every product issued so far by this thread has completed
template <bool PAIR>
__device__ __forceinline__ void commit_to(uint64_t *bar)
{
    if constexpr (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(saddr(bar)),
                     "h"((uint16_t)3)
                     : "memory");
    else
        mma_commit(bar);
}

// Arrive on the first CTA's barrier at the same place.  What it tells of is tensor memory alone, written or read by this CTA
// and waited for, which the fences around the arrival and the wait order; no shared or global memory is handed over, so
// the arrival is a relaxed one.
__device__ __forceinline__ void arrive_first(uint64_t *bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(in_first(saddr(bar))) : "memory");
}

// True when the phase is complete.  On a pair both CTAs' copies, or both CTAs' warps, arrive on the barrier: copies hand over
// shared memory, so the wait for them acquires at cluster scope, warps tensor memory alone (RELAXED).
template <bool PAIR, bool RELAXED>
__device__ __forceinline__ bool test_of(uint64_t *b, uint32_t parity)
{
    if constexpr (!PAIR) return mbar_test(b, parity);
    uint32_t ok;
    if constexpr (RELAXED)
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(saddr(b)), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(ok)
            : "r"(saddr(b)), "r"(parity)
            : "memory");
    return ok != 0;
}

// until test() holds; false after kWaitLimitNs
template <typename T>
__device__ __forceinline__ bool wait_until(T test)
{
    if (test()) return true;
    const uint64_t t0 = gtime();
    for (;;) {
        for (int i = 0; i < 64; i++)
            if (test()) return true;
        if (gtime() - t0 > kWaitLimitNs) return false;
    }
}

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\n barrier.cluster.wait.acquire;" ::: "memory");
}

struct Unit {
    int e, r0, n, tile;  // expert, first row, rows (1..BN), weight tile
    bool real;           // false: the second CTA of a pair has no tile of its own and stores nothing
};

// this CTA's (a pair's) units in order; off: clamped offsets, tcum: row tiles of X before each expert (shared memory)
template <typename Sh>
struct Units {
    const int *off, *tcum;
    int64_t u, total;
    int e, tiles, per;  // per: units for each row tile of X
    __device__ __forceinline__ Units(const int *off_, const int *tcum_, const GroupView &v)
        : off(off_), tcum(tcum_), u(Sh::PAIR ? blockIdx.x >> 1 : blockIdx.x), e(0), tiles(v.tiles), per(Sh::PAIR ? (v.tiles + 1) / 2 : v.tiles)
    {
        total = (int64_t)__reduce_max_sync(0xFFFFFFFFu, tcum[v.experts]) * per;  // a uniform register
    }
    __device__ __forceinline__ bool next(Unit &w)
    {
        if (u >= total) return false;
        const int tt = (int)(u / per), t = (int)(u - (int64_t)tt * per);
        const int tile = Sh::PAIR ? 2 * t + (int)(blockIdx.x & 1) : t;
        w.real = tile < tiles;
        w.tile = min(tile, tiles - 1);
        while (tt >= tcum[e + 1]) e++;
        w.e = e;
        w.r0 = off[e] + (tt - tcum[e]) * Sh::BN;
        w.n = min(Sh::BN, off[e + 1] - w.r0);
        u += Sh::PAIR ? gridDim.x >> 1 : gridDim.x;
        return true;
    }
};

template <bool GATED, bool GATHER, typename Sh>
__global__ void __launch_bounds__(kThreads, 1) group_tc_kernel(const __grid_constant__ TcArgs a)
{
    constexpr int BN = Sh::BN, kBN = BN, kSX = Sh::SX, kSW = Sh::SW, kSA = Sh::SA, kACol = Sh::ACol;
    constexpr uint32_t kXStage = Sh::XStage;
    constexpr bool PAIR = Sh::PAIR, SUMS = Sh::SUMS;
    constexpr int kGroups = Sh::Groups, kRebuildWarps = 4 * kGroups, kProdWarp = Sh::ProdWarp, kMmaWarp = Sh::MmaWarp, kXWarp0 = Sh::XWarp0;
    constexpr int kProdWarp2 = Sh::ProdWarp2, kEpiWarp0 = Sh::EpiWarp0, kEpiWarps = Sh::EpiWarps;
    constexpr int kXRows = Sh::XRows, kNStep = PAIR ? 32 : 16;  // N is a multiple of kNStep
    const int rank = PAIR ? (int)(blockIdx.x & 1) : 0;            // in the pair
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t pad = (1024u - (saddr(smem_raw) & 1023u)) & 1023u;
    uint8_t *xring = smem_raw + pad;                  // [kSX][kXStage], 1024-aligned
    uint8_t *wring = xring + kSX * kXStage;           // [kSW][kWStage]: step, record, verbatim runs
    uint64_t *wfull = (uint64_t *)(wring + kSW * kWStage);
    uint64_t *wempty = wfull + kSW;
    uint64_t *xfull = wempty + kSW;
    uint64_t *xempty = xfull + kSX;
    uint64_t *afull = xempty + kSX;
    uint64_t *aempty = afull + kSA;
    uint64_t *accfull = aempty + kSA, *accempty = accfull + 2, *done = accempty + 2;
    uint32_t *tmem_slot = (uint32_t *)(done + 1);
    int *off = (int *)((uint8_t *)wfull + 512);       // [experts + 1]
    int *tcum = off + kMaxExperts + 4;                // [experts + 1]
    int *xrows = tcum + kMaxExperts + 4;              // [kSX][kXRows] (sources) a warp's unit's rows of X (past the end: zeros)

    const GroupView &v = a.c.v;
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp: a uniform value
    const int ksteps = v.ksteps;

    if (threadIdx.x == 32 * kProdWarp) {
        for (int s = 0; s < kSW; s++) {
            mbar_init(&wfull[s], 1);
            mbar_init(&wempty[s], 4);
        }
        for (int s = 0; s < kSX; s++) {
            mbar_init(&xfull[s], 1);
            mbar_init(&xempty[s], 1);
        }
        for (int s = 0; s < kSA; s++) {
            mbar_init(&afull[s], PAIR && rank == 0 ? 8 : 4);  // a rebuild group's warps, in the first CTA those of both
            mbar_init(&aempty[s], 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(&accfull[b], 1);
            mbar_init(&accempty[b], PAIR && rank == 0 ? 2 * kEpiWarps : kEpiWarps);
        }
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        if constexpr (PAIR) {
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)), "r"(512)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        } else {
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)), "r"(512)
                         : "memory");
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        }
    }
    pdl_trigger();
    pdl_wait();
    if (warp == 0) {
        // the experts' row tiles: a running sum, 32 experts at a time
        const int R = (int)a.c.rows;
        int carry = 0;
        for (int e0 = 0; e0 < v.experts; e0 += 32) {
            const int e = e0 + lane;
            int l = 0, h = 0;
            if (e < v.experts) {
                l = min(max(a.c.offsets[e], 0), R);
                h = min(max(a.c.offsets[e + 1], 0), R);
            }
            const int t = h > l ? (h - l + kBN - 1) / kBN : 0;
            int s = t;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xFFFFFFFFu, s, d);
                if (lane >= d) s += o;
            }
            if (e < v.experts) {
                off[e] = l;
                tcum[e] = carry + s - t;
                if (e == v.experts - 1) {
                    off[e + 1] = h;
                    tcum[e + 1] = carry + s;
                }
            }
            carry += __shfl_sync(0xFFFFFFFFu, s, 31);
        }
    }
    tc_fence_before();
    if constexpr (PAIR) cluster_barrier();  // the barriers of both CTAs are set up
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Units<Sh> units(off, tcum, v);
    Unit w;
    const bool any = units.u < units.total;
    // A unit's sums are taken in segments of K, the two accumulators in turn: the tensor core cuts low bits off a running
    // sum at every product, an error that grows with the sum's length (2e-6 of a result at K = 4096).  For a bf16 output
    // that is far below the rounding, and a segment is all of K; an fp32 output gets segments of 512, added in fp32.
    const int seg_steps = SUMS ? kSegSteps : ksteps;

    if (warp == kProdWarp || warp == kProdWarp2) {
        // ---------------------------------------------------------------------------------------- weight copies
        // Two warps take alternate steps: one alone, with a wait, a copy or two and their addresses, took 820 cycles a
        // step, twice what the products of a step take.
        const int p = warp == kProdWarp ? 0 : 1;
        bool ok = true;
        const bool leader = elect_one();
        int i = 0, last = -1;  // steps before this unit; the last step asked for
        // lane l: {first, count} of the verbatim runs of step l of the 32 at hand; the next 32 in flight
        auto recs_at = [&](const Unit &q, int ks) {
            const int64_t st = ((int64_t)q.e * v.tiles + q.tile) * ksteps + ks + lane;
            return ks + lane < ksteps ? __ldg((const uint2 *)&step_rec(v.steps, st)->first) : make_uint2(0, 0);
        };
        Unit nx;
        bool have = units.next(w), have_nx = false;
        uint2 cur = make_uint2(0, 0), nxt = cur;
        if (have) nxt = recs_at(w, 0);
        while (have && ok) {
            have_nx = units.next(nx);
            const uint8_t *src = v.steps + ((int64_t)w.e * v.tiles + w.tile) * ksteps * kStepBytes;
            for (int k0 = 0; k0 < ksteps && ok; k0 += 32) {
                cur = nxt;
                if (k0 + 32 < ksteps) nxt = recs_at(w, k0 + 32);
                else if (have_nx) nxt = recs_at(nx, 0);
                const int ke = min(ksteps, k0 + 32);
                for (int ks = k0 + ((i + k0 + p) & 1); ks < ke; ks += 2) {
                    const int q = i + ks, s = q % kSW;
                    const uint32_t first = __shfl_sync(0xFFFFFFFFu, cur.x, ks - k0);
                    const uint32_t nv = min(__shfl_sync(0xFFFFFFFFu, cur.y, ks - k0), (uint32_t)kVCs);
                    if (q >= kSW && !__all_sync(0xFFFFFFFFu, mbar_wait(&wempty[s], ((q / kSW) & 1) ^ 1))) { ok = false; break; }
                    if (leader) {
                        const uint32_t d = saddr(wring) + s * kWStage, fb = saddr(&wfull[s]);
                        mbar_expect_tx(&wfull[s], kStepBytes + 64u * nv);
                        bulk_copy(d, src + (int64_t)ks * kStepBytes, kStepBytes, fb);
                        if (nv) bulk_copy(d + kVOff, v.verb + (uint64_t)first * 64, nv * 64u, fb);
                    }
                    __syncwarp();
                    last = q;
                }
            }
            if (!ok) break;
            i += ksteps;
            w = nx;
            have = have_nx;
        }
        if (!ok && leader) {
            // the copies in flight land before the block ends
            atomicExch(v.status, (int)DEV_TIMEOUT);
            for (int n = 0; n < kSW / 2 && last >= 0; n++, last -= 2) mbar_wait(&wfull[last % kSW], (last / kSW) & 1);
        }
    } else if (warp >= kXWarp0 && warp < kXWarp0 + kXWarps) {
        // ---------------------------------------------------------------------------------------- X copies
        // Warp x brings steps x, x + kSX, ... into stage x: a step's copies take one warp longer than its products.
        const int x = warp - kXWarp0;
        const uint32_t xs = saddr(xring + x * kXStage);
        // On a pair both CTAs' copies complete on the first one's barrier, which expects the bytes of both: the product that the
        // first CTA issues reads both halves of the tile.  The second is never a turn ahead of that barrier: its stage is free
        // once the products on the turn before, and so that turn's phase, are complete.
        const uint32_t fb = PAIR ? in_first(saddr(&xfull[x])) : saddr(&xfull[x]);
        const uint32_t both = PAIR ? 2 : 1;
        bool ok = true;
        int i = 0, turn = 0;  // steps before this unit, this stage's turns
        // this CTA's rows of a unit's X tile: how many, and the first (of a pair's, each half)
        auto x_rows = [&](const Unit &q) { return ((q.n + kNStep - 1) / kNStep * kNStep) / (PAIR ? 2 : 1); };
        auto x_first = [&](const Unit &q) { return PAIR ? rank * x_rows(q) : 0; };
        auto stage_free = [&] { return turn == 0 || __all_sync(0xFFFFFFFFu, mbar_wait(&xempty[x], (turn - 1) & 1)); };
        if constexpr (GATHER) {
            int *rows = xrows + x * kXRows;
            constexpr int kL = kXRows / 32;
            const bool leader = elect_one();
            const int none = (int)a.c.x_rows;  // past the end
            int r[kL];  // the next unit's rows, on their way before it begins
            auto fetch = [&](const Unit &q) {
#pragma unroll
                for (int j = 0; j < kL; j++) {
                    const int row = x_first(q) + 32 * j + lane;
                    r[j] = 32 * j + lane < x_rows(q) && row < q.n ? a.c.row_src[q.r0 + row] : -1;
                }
            };
            Unit nx;
            bool have = units.next(w);
            if (have) fetch(w);
            while (ok && have) {
                __syncwarp();
#pragma unroll
                for (int j = 0; j < kL; j++) rows[32 * j + lane] = r[j] >= 0 && r[j] < none ? r[j] : none;
                __syncwarp();
                const bool more = units.next(nx);
                if (more) fetch(nx);
                const int bn = x_rows(w);
                for (int ks = (kSX - i % kSX + x) % kSX; ks < ksteps; ks += kSX, turn++) {
                    if (!stage_free()) { ok = false; break; }
                    if (leader) {
                        if (rank == 0) mbar_expect_tx(&xfull[x], both * (uint32_t)bn * 128u);
                        for (int q = 0; q < bn; q += 16) {
                            int4 y[4];
#pragma unroll
                            for (int j = 0; j < 4; j++) y[j] = *(const int4 *)(rows + q + 4 * j);
#pragma unroll
                            for (int j = 0; j < 4; j++) tma_gather4<PAIR>(xs + 128 * q + 512 * j, &a.tm_x, ks * kStepW, y[j], fb);
                        }
                    }
                    __syncwarp();
                }
                i += ksteps;
                w = nx;
                have = more;
            }
        } else {
            while (ok && units.next(w)) {
                const int boxes = (x_rows(w) + 31) / 32, first = w.r0 + x_first(w);
                for (int ks = (kSX - i % kSX + x) % kSX; ks < ksteps; ks += kSX, turn++) {
                    if (!stage_free()) { ok = false; break; }
                    if (rank == 0 && lane == 0) mbar_expect_tx(&xfull[x], both * (uint32_t)boxes * 4096u);
                    __syncwarp();
                    if (lane < boxes) tma_box<PAIR>(xs + 4096u * lane, &a.tm_x, ks * kStepW, first + 32 * lane, fb);
                    __syncwarp();
                }
                i += ksteps;
            }
        }
        // The copies in flight land before the block ends.  (The second CTA of a pair has no barrier of its own for them; the
        // wait that ran out began after its last one was asked for.)
        if (!ok && lane == 0 && turn > 0 && rank == 0) mbar_wait(&xfull[x], (turn - 1) & 1);
        if (!ok && lane == 0) atomicExch(v.status, (int)DEV_TIMEOUT);
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------------------------------------- MMA issue
        // The whole warp walks the steps, so that the addresses and descriptors are uniform values, and elects the issuing
        // thread for each step, so that the compiler sees that one thread issues.  (A loop inside `if (lane == 0)` took 870
        // cycles a step at any N, one whose thread is elected once 600.)
        bool ok = true;
        int sx = 0, sa = 0, ns = 0;  // ns: segments begun
        uint32_t phx = 0, pha = 0;
        const uint64_t desc0 = smem_desc_sw128(saddr(xring));
        while (rank == 0 && ok && units.next(w)) {
            // reductions give uniform registers
            const int wn = __reduce_max_sync(0xFFFFFFFFu, w.n);
            const uint32_t id = idesc_bf16(PAIR ? 2 * kTileRows : kTileRows, (wn + kNStep - 1) / kNStep * kNStep);
            for (int k0 = 0; k0 < ksteps && ok; k0 += seg_steps, ns++) {
                const int buf = ns & 1, n = min(seg_steps, ksteps - k0);
                if (ns >= 2 && !__all_sync(0xFFFFFFFFu, wait_until([&] { return test_of<PAIR, true>(&accempty[buf], ((ns >> 1) - 1) & 1); }))) { ok = false; break; }
                tc_fence_after();
                const uint32_t d = buf * kBN;  // all of tensor memory is this block's: it begins at 0
                for (int j = 0; j < n; j++) {
                    auto operands = [&] {
                        const bool p = test_of<PAIR, true>(&afull[sa], pha), q = test_of<PAIR, false>(&xfull[sx], phx);
                        return p && q;
                    };
                    if (!__all_sync(0xFFFFFFFFu, wait_until(operands))) { ok = false; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t at = kACol + 32 * sa;
                        const uint64_t xd = desc0 + (uint64_t)(sx * (int)(kXStage >> 4));
#pragma unroll
                        for (int kk = 0; kk < 4; kk++) mma_of<PAIR>(d, at + 8 * kk, xd + 2 * kk, id, (j | kk) ? 1u : 0u);
                        commit_to<PAIR>(&aempty[sa]);
                        commit_to<PAIR>(&xempty[sx]);
                        if (j == n - 1) commit_to<PAIR>(&accfull[buf]);
                    }
                    __syncwarp();
                    if (++sa == kSA) { sa = 0; pha ^= 1u; }
                    if (++sx == kSX) { sx = 0; phx ^= 1u; }
                }
            }
        }
        if (!ok && lane == 0) atomicExch(v.status, (int)DEV_TIMEOUT);
        if (ns > 0) {
            // every product issued has completed before the tensor memory is freed
            if (elect_one()) commit_to<PAIR>(done);
            __syncwarp();
            if (!mbar_wait(done, 0) && lane == 0) atomicExch(v.status, (int)DEV_TIMEOUT);
        }
    } else if (warp < kRebuildWarps) {
        // ---------------------------------------------------------------------------------------- rebuild
        const int grp = warp >> 2, r = 32 * (warp & 3) + lane;  // row of the tile
        const uint32_t o_s = (r >> 4) * 1024 + ((r >> 3) & 1) * 512 + chunk_at(r & 7, 0);  // chunk t at o_s ^ 16 t
        const uint32_t o_c = kStepSm + (r >> 4) * 512 + chunk_at(r & 7, 0) + ((r >> 3) & 1) * 8;
        const uint32_t t_lane = (uint32_t)(32 * (warp & 3)) << 16;
        bool ok = true;
        int i = 0;  // steps before this unit
        while (ok && units.next(w)) {
            const uint32_t B = GATED ? __ldg(v.base + 2 * w.e + ((r >> 4) & 1)) : __ldg(v.base + w.e);
            for (int ks = (kGroups - i % kGroups + grp) % kGroups; ks < ksteps; ks += kGroups) {
                const int q = i + ks, s = q % kSW, sa = q % kSA;
                if (!mbar_wait(&wfull[s], (q / kSW) & 1)) { ok = false; break; }
                const uint8_t *st = wring + s * kWStage;
                const uint32_t *mask = (const uint32_t *)(st + kStepRec);
                const uint32_t mw = mask[r >> 5];
                const bool verb = (mw >> lane) & 1u;
                const uint32_t run = verb ? verbatim_rank(mask, r) : 0u;
                // The 32 words are rebuilt before the wait for a slot of tensor memory, so that a slot is held for their
                // store alone.
                uint32_t p[32];
#pragma unroll
                for (int t = 0; t < 4; t++) {
                    const uint4 S = *(const uint4 *)(st + (o_s ^ (16u * t)));
                    const uint2 C = *(const uint2 *)(st + (o_c ^ (16u * t)));
                    uint32_t c[8];
                    rebuild_chunk(S, C, B, c);
                    if (mw) {
                        // a verbatim run among the warp's rows (the same word for every lane)
                        if (verb) {
                            uint4 E;
                            if (run < (uint32_t)kVCs) E = *(const uint4 *)(st + kVOff + run * 64 + 16 * t);
                            else E = __ldg((const uint4 *)(v.verb + ((uint64_t)mask[4] + run) * 64 + 16 * t));
                            rebuild_chunk_verbatim(S, E, c);
                        }
                        __syncwarp();
                    }
#pragma unroll
                    for (int k = 0; k < 8; k++) p[8 * t + k] = c[k];
                }
                // the stage's reads are done before the next copy into it (the async proxy) is asked for
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&wempty[s]);
                if (q >= kSA && !mbar_wait(&aempty[sa], ((q / kSA) & 1) ^ 1)) { ok = false; break; }
                tc_fence_after();
                __syncwarp();  // lanes leave the waits one by one, the store is the whole warp's
                tmem_st32(tmem + t_lane + kACol + 32 * sa, p);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR && rank == 1) arrive_first(&afull[sa]);
                    else mbar_arrive(&afull[sa]);
                }
            }
            i += ksteps;
        }
        if (!ok && lane == 0) atomicExch(v.status, (int)DEV_TIMEOUT);
    } else if (warp >= kEpiWarp0) {
        // ---------------------------------------------------------------------------------------- epilogue
        const int q = warp & 3;
        bool ok = true;
        int ns = 0;
        // 16 columns from c0 on into the output
        auto emit = [&](const float (&x)[16], int c0) {
            constexpr int NO = GATED ? 8 : 16;
            float f[NO];
            int first = c0;
            int64_t col;
            if constexpr (GATED) {
                const bool up = lane >= 16;
                first += up ? 8 : 0;
                float gate[8];
#pragma unroll
                for (int j = 0; j < 8; j++) {
                    const float mine = up ? x[8 + j] : x[j];
                    const float other = __shfl_xor_sync(0xFFFFFFFFu, up ? x[j] : x[8 + j], 16);
                    gate[j] = up ? other : mine;
                    f[j] = up ? mine : other;
                }
                if (!SUMS && a.c.out_bf16) {
#pragma unroll
                    for (int j = 0; j < 8; j++) f[j] = gated<false>(gate[j], f[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; j++) f[j] = gated<true>(gate[j], f[j]);
                }
                col = ((int64_t)w.tile * 4 + q) * 16 + (lane & 15);
            } else {
#pragma unroll
                for (int j = 0; j < 16; j++) f[j] = x[j];
                col = (int64_t)w.tile * kTileRows + 32 * q + lane;
            }
            const int m = w.real && col < v.N ? w.n - first : 0;
            const int64_t o = (int64_t)(w.r0 + first) * a.c.ldy + col;
            if (a.c.out_bf16) {
                __nv_bfloat16 *p = (__nv_bfloat16 *)a.c.y + o;
#pragma unroll
                for (int j = 0; j < NO; j++, p += a.c.ldy)
                    if (j < m) *p = __float2bfloat16_rn(f[j]);
            } else {
                float *p = (float *)a.c.y + o;
#pragma unroll
                for (int j = 0; j < NO; j++, p += a.c.ldy)
                    if (j < m) *p = f[j];
            }
            __syncwarp();
        };
        auto columns = [&](uint32_t acc, float (&x)[16]) {
            uint32_t u[16];
            tmem_ld16(acc, u);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; j++) x[j] = __uint_as_float(u[j]);
        };
        while (ok && units.next(w)) {
            for (int k0 = 0; k0 < ksteps; k0 += seg_steps, ns++) {
                const int buf = ns & 1;
                if (!mbar_wait(&accfull[buf], (ns >> 1) & 1)) { ok = false; break; }
                tc_fence_after();
                __syncwarp();  // lanes leave the wait one by one, the loads are the whole warp's
                const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + buf * kBN;
                const uint32_t run = tmem + ((uint32_t)(32 * q) << 16) + Sh::RunCol;  // this warp's alone
                for (int c0 = 0; c0 < w.n; c0 += 16) {
                    float x[16];
                    columns(acc + c0, x);
                    if constexpr (SUMS) {
                        if (k0) {
                            float y[16];
                            columns(run + c0, y);
#pragma unroll
                            for (int j = 0; j < 16; j++) x[j] += y[j];
                        }
                        if (k0 + seg_steps < ksteps) {
                            uint32_t u[16];
#pragma unroll
                            for (int j = 0; j < 16; j++) u[j] = __float_as_uint(x[j]);
                            tmem_st16(run + c0, u);
                            continue;
                        }
                    }
                    emit(x, c0);
                }
                if constexpr (SUMS) tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (PAIR && rank == 1) arrive_first(&accempty[buf]);
                    else mbar_arrive(&accempty[buf]);
                }
            }
        }
        if (!ok && lane == 0) atomicExch(v.status, (int)DEV_TIMEOUT);
    }
    tc_fence_before();
    if constexpr (PAIR) {
        // Neither CTA ends while products read its memory, or while word of them is on its way: of the second's barriers `done`
        // is the last to be told, after its accumulators, which its epilogue has seen.
        __syncthreads();
        if (rank == 1 && any && warp == kMmaWarp && !mbar_wait(done, 0) && lane == 0) atomicExch(v.status, (int)DEV_TIMEOUT);
        cluster_barrier();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        __syncwarp();
        if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
        else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <bool GATED, bool GATHER, typename Sh>
cudaError_t launch_one(const TcArgs &a, cudaStream_t st)
{
    auto kernel = group_tc_kernel<GATED, GATHER, Sh>;
    static OncePerDevice once;
    const cudaError_t e = allow_shared(once, kernel, Sh::smem);
    if (e != cudaSuccess) return e;
    // at least one row tile for each BN rows, at most one more for each expert
    const GroupCall &c = a.c;
    const int64_t row_tiles = (c.rows + Sh::BN - 1) / Sh::BN + std::min<int64_t>(c.v.experts, c.rows);
    const int64_t units = row_tiles * (Sh::PAIR ? (c.v.tiles + 1) / 2 : c.v.tiles);
    const int64_t grid = Sh::PAIR ? 2 * std::min<int64_t>(std::max(1, num_sms() / 2), units) : std::min<int64_t>(num_sms(), units);
    return launch_dependent(kernel, dim3((unsigned)grid), kThreads, Sh::smem, Sh::PAIR ? 2u : 0u, st, a);
}

template <typename Sh>
cudaError_t launch_shape(const TcArgs &a, cudaStream_t st)
{
    if (a.c.v.gated) return a.c.row_src ? launch_one<true, true, Sh>(a, st) : launch_one<true, false, Sh>(a, st);
    return a.c.row_src ? launch_one<false, true, Sh>(a, st) : launch_one<false, false, Sh>(a, st);
}

bool map_x(CUtensorMap *m, const GroupCall &c)
{
    auto fn = (PFN_cuTensorMapEncodeTiled_v12000)tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)c.v.K, (cuuint64_t)c.x_rows};
    cuuint64_t strides[1] = {(cuuint64_t)c.ldx * 2};
    cuuint32_t box[2] = {64, c.row_src ? 1u : 32u};
    cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t *>(c.x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool group_tc_supported(const GroupCall &c)
{
    // the map's row stride is below 2^40 bytes
    return c.x_rows > 0 && c.ldx < ((int64_t)1 << 39) && tensor_map_encoder() != nullptr;
}

int launch_group_tc(const GroupCall &c, void *stream)
{
    TcArgs a;
    memset(&a, 0, sizeof a);
    if (!map_x(&a.tm_x, c)) return cudaErrorInvalidValue;
    a.c = c;
    // An fp32 output of several segments is summed in tensor memory, by the shape that has room for it.  Adding the segments up
    // in the output instead, by the pairs of 192 rows, took 70 us against 64 for 512 tokens top 8 of 64 experts of [2048, 1408],
    // 278 against 218 for 4096, 212 against 134 for 333 tokens top 2 of 8 of [4096, 14336]; in the epilogue's registers, by
    // single CTAs of 64 rows, gated, 864 against 453 for 4096 tokens top 8 of 64 of [1408, 2048], 249 against 219 for 32 top 2
    // of 8 of [14336, 4096].
    if (group_sums(c)) return launch_shape<Shape<128, true, true>>(a, (cudaStream_t)stream);
    // Else pairs of CTAs, or single ones up to 24 rows an expert on average: 64 experts of [2048, 1408] take 51.4 us against
    // 54.0 at 16 rows each, 56.9 against 56.0 at 32, 74 against 59 at 64.
    if (c.rows <= 24 * (int64_t)c.v.experts) return launch_shape<Shape<64, false, false>>(a, (cudaStream_t)stream);
    return launch_shape<Shape<192, true, false>>(a, (cudaStream_t)stream);
}

}  // namespace uw
