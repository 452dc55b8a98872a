// k_attend_tc.cu - attention of many new tokens over a cache of keys and values in pages, on tcgen05 (sm_103a).
//
// An item is 256 query rows - tokens x query heads of one key head - as two tiles A and B of 128, against tiles of 128 keys.
// (Or 128 rows, where the sequences bring no more on average: tile A alone, with room for one more tile of keys or values.)
//   S = Q K^T   (128 x 128, operands in shared memory), P = 2^(scale2 S - m) by a warpgroup, a thread a row,
//   O += P V    (P in tensor memory, V from shared memory as it lies in the cache: keys x elements)
// Roles of the twelve warps (of eight, with one tile: A's four, then the same):
//   - 0-3 and 4-7: softmax, output and queries of tile A, of tile B.  A thread holds its row's 128 scores in registers, so a
//     row's maximum and sum take no exchange.  The output is rescaled only when a maximum has grown by more than 2^8 (then
//     by tensor memory loads and stores of the row): probabilities are at most 256 and keep their relative precision;
//   - 8: tensor copies of the pages' slots of one head, keys and values in turn, into a ring of 128-key tiles.  Values that
//     no row of the item sees are set to zero in shared memory when they have landed, as 0 x NaN is NaN;
//   - 9: the products of Q and K, A's and B's in turn; 10: those of P and V, by one thread each (one warp for both: 680 us
//     against 638 for 8191 tokens, at that step);
//   - 11: none, it makes up the third warpgroup, which gives registers to the other two.
// Tensor memory: O of A and B, one S, P of A and of B: 2 D + 128 + 2 x 64 columns.  One S is enough as a warpgroup takes its
// scores into registers at once, under the product in between, and P does not lie in S: every reuse waits on a barrier of
// what used it last.  The product of P and V starts when the first half of a tile's probabilities is there.
// P is rounded to bf16 as an operand (by 2^-8 of each at most; the sum of the powers is taken before that).
// Waits suspend the thread: polls of shared memory take turns that the operands of the products need (a spinning form took 874 us
// where this one took 638).
//
// Measured in a captured chain (as ordinary calls): 8191 tokens of 32 query heads over 8 key heads of 128, causal: 396 us (417), 1.39 PFLOP/s,
// not causal 704, 1.56; 509 tokens of 64 heads over 7171: 116 us (119), 1.07 PFLOP/s.  What an item costs beside its tiles (queries, the pipeline's ends,
// the output, a part's way through the workspace: 3 to 10 us) is what keeps the smaller ones from that.  The chain of a tile bounds a
// long one: scores 0.27 us, 0.15 until they are seen, 0.9 for softmax, 0.15, the second product 0.27; the tensor cores are busy half of
// the time (4095 tokens), the units for powers a quarter.  4 tokens x 8 heads over 131067: 109 us (110), 4.9 TB/s: 54 tiles of keys a CTA, 1.85 us each, the chain of one
// tile again, as an item of 128 rows has no other one to run beside it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "attend.cuh"
#include "dev_async.cuh"
#include "f32x2.cuh"
#include "launch.cuh"
#include "uw_internal.h"

namespace uw {

namespace {

using namespace dev;

constexpr int kTile = kKeys;
constexpr float kNegInf = -INFINITY;
constexpr float kGrow = 8.f;      // log2 of how far a maximum may grow before the output is rescaled

template <int D, int T>
struct Layout {
    static constexpr uint32_t half = kTile * 128;               // 64 elements of 128 rows or keys
    static constexpr uint32_t tile = half * (D / 64);           // a tile of queries, keys or values
    static constexpr int slots = (D == 128 ? 7 : 12) - T;
    static constexpr uint32_t bars = 8 * (3 * slots + 18);
    static constexpr size_t smem = 1024 + (T + slots) * tile + bars + 16;
    static_assert(smem <= 227 * 1024, "shared memory");
    // columns of tensor memory
    static constexpr uint32_t o = 0, s = 2 * D, p = s + 128;    // O of tile t at o + t D, P at p + 64 t
    static_assert(p + 128 <= 512, "tensor memory");
};

struct Args {
    CUtensorMap km, vm;
    AttendCall c;
    uint32_t q_xor, q_and;    // what turns a pair of query elements for a negative or zero scale
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void tma4d(uint32_t dst, const CUtensorMap *map, int x, int slot, int head, int page, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(slot), "r"(head), "r"(page), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]),
          "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
          "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]),
          "=r"(v[31])
        : "r"(taddr)
        : "memory");
}

// descriptor of values as the second operand: keys (the summed dimension) 128 bytes apart, 64 elements (columns of the result)
// in a row of the 128-byte swizzle, groups of eight keys 1024 bytes apart, blocks of 64 elements `half` bytes apart
__device__ __forceinline__ uint64_t values_desc(uint32_t addr, uint32_t half)
{
    uint64_t d = (uint64_t)((addr >> 4) & 0x3FFFu);
    d |= (uint64_t)(half >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// both barriers' phases; false after the limit of a wait
__device__ __forceinline__ bool wait_both(uint64_t *a, uint32_t pa, uint64_t *b, uint32_t pb)
{
    const bool x = mbar_poll(a, pa), y = mbar_poll(b, pb);
    if (x && y) return true;
    return mbar_wait_short(a, pa) && mbar_wait_short(b, pb);
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *(const uint32_t *)&v;
}

// the 128 threads of a tile of rows; the barrier is of whole warps
__device__ __forceinline__ void tile_sync(int t)
{
    __syncwarp();
    asm volatile("bar.sync %0, 128;" ::"r"(1 + t) : "memory");
}

// Joins a row's parts of an item that was cut, a thread a row: those of ranges r0 .. r0 + parts - 1.
template <int D, int kRows, typename Cur>
__device__ __forceinline__ void join_row(const AttendCall &a, const Cur &c, int r0, int parts, int r, int tok, int x)
{
    constexpr size_t kSlot = slot_floats<kRows, D>();
    auto part = [&](int i) { return a.part + (2 * (size_t)(r0 + i) + (i == 0 ? 1 : 0)) * kSlot; };
    float m = kNegInf, l = 0.f;
#pragma unroll 4
    for (int i = 0; i < parts; i++) m = fmaxf(m, __ldcg(part(i) + kRows * D + r));
    const float b = m == kNegInf ? 0.f : m;
#pragma unroll 4
    for (int i = 0; i < parts; i++) l += __ldcg(part(i) + kRows * D + kRows + r) * exp2_fast(__ldcg(part(i) + kRows * D + r) - b);
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
    const int h = c.head * a.group + x - tok * a.group;
    const int64_t row = c.w.q.first + tok;
    uint16_t *p = a.out + row * a.ldo + (int64_t)h * D;
#pragma unroll 1
    for (int q = 0; q < D; q += 64) {
        float o[64];
#pragma unroll
        for (int k = 0; k < 64; k++) o[k] = 0.f;
#pragma unroll 1
        for (int i = 0; i < parts; i++) {
            const float *s = part(i);
            float4 v[16];
#pragma unroll
            for (int k = 0; k < 16; k++) v[k] = __ldcg((const float4 *)s + ((q / 4 + k) * kRows + r));
            const float f = exp2_fast(__ldcg(s + kRows * D + r) - b);
#pragma unroll
            for (int k = 0; k < 16; k++) {
                o[4 * k] += v[k].x * f;
                o[4 * k + 1] += v[k].y * f;
                o[4 * k + 2] += v[k].z * f;
                o[4 * k + 3] += v[k].w * f;
            }
        }
#pragma unroll
        for (int k = 0; k < 64; k += 8)
            *(uint4 *)(p + q + k) = make_uint4(pack2(o[k] * inv, o[k + 1] * inv), pack2(o[k + 2] * inv, o[k + 3] * inv),
                                               pack2(o[k + 4] * inv, o[k + 5] * inv), pack2(o[k + 6] * inv, o[k + 7] * inv));
    }
    if (a.lse) a.lse[row * a.q_heads + h] = l == 0.f ? kNegInf : (m + log2f(l)) * 0.69314718f;
}

// T: tiles of 128 rows of an item, and warpgroups that have one.
template <int D, int T>
__global__ void __launch_bounds__(128 * (T + 1), 1) attend_tc_kernel(const __grid_constant__ Args g)
{
    using L = Layout<D, T>;
    constexpr int kRows = 128 * T;
    constexpr int kCopyWarp = 4 * T, kScoreWarp = kCopyWarp + 1, kValueWarp = kCopyWarp + 2;
    using Cur = Cursor<kRows, kItemTc>;
    constexpr int NS = L::slots;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const AttendCall &a = g.c;
    uint8_t *qs = smem_raw + ((1024u - (saddr(smem_raw) & 1023u)) & 1023u);  // [T] tiles
    uint8_t *ring = qs + T * L::tile;
    // Tile i of the ring (keys, values, keys, ...) is in slot i % NS, and has landed when full[i % 2 NS] has completed phase i / 2 NS.  A slot
    // of an odd ring holds keys and values in turn, which two warps wait for: with one barrier for both the one could ask for its tile's phase
    // while the other's before it is still open, and the parity would answer a turn early.  So each has its own, 2 NS being even.
    uint64_t *full = (uint64_t *)(ring + NS * L::tile);
    uint64_t *empty = full + 2 * NS;
    uint64_t *raw = empty + NS;                       // a tile whose values are put right before it counts as full
    uint64_t *qfull = raw + 1, *sfull = qfull + 2, *sfree = sfull + 2, *pfull = sfree + 1, *pvdone = pfull + 4, *ofree = pvdone + 2, *done = ofree + 2;
    uint32_t *tmem_slot = (uint32_t *)((uint8_t *)full + L::bars);
    volatile int *last = (volatile int *)(tmem_slot + 1);   // [2]: of each tile of rows
    const int warp = __shfl_sync(0xFFFFFFFFu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; i++) {
            mbar_init(&full[i], 1);
            mbar_init(&full[NS + i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(raw, 1);
        mbar_init(sfree, 4);
        mbar_init(&done[0], 1);
        mbar_init(&done[1], 1);
        for (int t = 0; t < 2; t++) {
            mbar_init(&qfull[t], 4);
            mbar_init(&sfull[t], 1);
            mbar_init(&pfull[2 * t], 4);
            mbar_init(&pfull[2 * t + 1], 4);
            mbar_init(&pvdone[t], 1);
            mbar_init(&ofree[t], 4);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
    if (warp == kScoreWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(tmem_slot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    pdl_trigger();
    pdl_wait();

    // this CTA's range
    const int range = blockIdx.x;
    const bool any = range < a.plan->ranges;
    const int64_t C = a.plan->per, ua = range * C, ub = min(ua + C, a.plan->units);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool ok = true;

    // 12 warps have 168 registers a thread at launch; a row of scores wants more: 256 x 208 + 128 x 88 is what 384 x 168 is
    if (warp >= 4 * T) {
        if constexpr (T == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (any && warp == kCopyWarp) {
            // ------------------------------------------------------------------------------ copies
            Cur c;
            c.set(a, a.begin[range], ua, ub);
            int n = 0;                        // tiles asked for: keys, values, keys, ...
            // values that are to be put right when they have landed
            bool fix = false;
            int fix_tile = 0, fix_lo = 0, fix_hi = 0;
            uint32_t raw_phase = 0;
            auto mend = [&] {
                if (!fix) return;
                fix = false;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait_short(raw, raw_phase & 1))) ok = false;
                raw_phase++;
                uint8_t *v = ring + fix_tile % NS * L::tile;
                for (int i = lane; i < kTile * (D / 8); i += 32) {
                    const int row = i / (D / 8), ch = i % (D / 8);
                    if (row >= fix_lo && row < fix_hi) continue;
                    *(uint4 *)(v + (ch >> 3) * L::half + row * 128 + ((ch & 7) ^ (row & 7)) * 16) = make_uint4(0, 0, 0, 0);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[fix_tile % (2 * NS)]);
                __syncwarp();
            };
            // a lane's copies: a box of slots, 64 elements each
            const int boxes = kTile / a.box, half = lane % (D / 64), bx0 = lane / (D / 64);
            constexpr int kPer = 32 / (D / 64);          // boxes of one round of lanes
            const uint32_t box_bytes = (uint32_t)a.box * 128u;
            for (; c.more() && ok; c.next(a)) {
                const int32_t *table = a.b.pages + (int64_t)c.s * a.b.ld_pages;
                for (int j = 0; j < c.cnt && ok; j++) {
                    const int key0 = (c.k.t0 + c.off + j) * kTile;
                    const bool odd = key0 < c.k.lo || key0 + kTile > c.k.hi;
                    for (int kv = 0; kv < 2 && ok; kv++) {
                        const int slot = n % NS;
                        if (n >= NS && !__all_sync(0xFFFFFFFFu, mbar_poll(&empty[slot], ((n / NS) & 1) ^ 1))) {
                            mend();
                            if (!__all_sync(0xFFFFFFFFu, mbar_wait_short(&empty[slot], ((n / NS) & 1) ^ 1))) { ok = false; break; }
                        }
                        const bool mended = kv && odd;
                        if (mended) mend();              // the one before
                        uint64_t *bar = mended ? raw : &full[n % (2 * NS)];
                        if (lane == 0) mbar_expect_tx(bar, L::tile);
                        __syncwarp();
                        for (int b0 = 0; b0 < boxes; b0 += kPer) {
                            const int bx = b0 + bx0;
                            if (bx < boxes) {
                                const int key = key0 + bx * a.box, pi = key / a.page_size;
                                const int page = key < c.w.keys ? table[pi] : -1;
                                tma4d(saddr(ring) + slot * L::tile + half * L::half + bx * box_bytes, kv ? &g.vm : &g.km, half * 64, key - pi * a.page_size, c.head,
                                      page, saddr(bar));
                            }
                        }
                        __syncwarp();
                        if (mended) {
                            fix = true;
                            fix_tile = n;
                            fix_lo = c.k.lo - key0;
                            fix_hi = c.k.hi - key0;
                        }
                        n++;
                    }
                }
            }
            mend();
            // the products' word that the last tiles are free arrives before the block ends
            for (int i = n > NS ? n - NS : 0; i < n && ok; i++) ok = __all_sync(0xFFFFFFFFu, mbar_wait_short(&empty[i % NS], (i / NS) & 1));
            if (!ok) {
                if (lane == 0) atomicExch(a.status, (int)DEV_TIMEOUT);
                __syncwarp();
                // what is on its way lands before the block ends (a tile that waits to be put right: above)
                for (int i = n > NS ? n - NS : 0; i < n; i++) mbar_wait_short(&full[i % (2 * NS)], (i / (2 * NS)) & 1);
            }
        } else if (any && warp == kScoreWarp) {
            // ------------------------------------------------------------------------------ products of queries and keys
            Cur c;
            c.set(a, a.begin[range], ua, ub);
            const bool leader = elect_one();
            constexpr uint32_t id = idesc_bf16(128, 128);
            const uint32_t q0 = saddr(qs), r0 = saddr(ring);
            int n = 0, qk = 0;                  // tiles of keys, products before this one
            int segs[2] = {0, 0};               // of each tile of rows: items begun
            for (; c.more() && ok; c.next(a)) {
                const int nt = c.cnt, both = T == 2 && c.rows(a) > 128;
                for (int j = 0; j < nt && ok; j++, n++) {
                    const int slot = (2 * n) % NS;
                    uint64_t *here = &full[(2 * n) % (2 * NS)];
                    const uint32_t turn = ((2 * n) / (2 * NS)) & 1;
                    for (int t = 0; t <= both && ok; t++) {
                        bool w = qk > 0 ? wait_both(here, turn, sfree, (qk - 1) & 1) : mbar_wait_short(here, turn);
                        if (j == 0) w = w && mbar_wait_short(&qfull[t], segs[t]++ & 1);
                        ok = __all_sync(0xFFFFFFFFu, w);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t qd = smem_desc_sw128(q0 + t * L::tile), kd = smem_desc_sw128(r0 + slot * L::tile);
                        if (leader) {
#pragma unroll
                            for (int k = 0; k < D / 16; k++) {
                                const uint32_t at = ((k >> 2) * L::half + (k & 3) * 32) >> 4;
                                mma_ss(tmem + L::s, qd + at, kd + at, id, k > 0);
                            }
                            mma_commit(&sfull[t]);
                            if (t == both) mma_commit(&empty[slot]);
                        }
                        __syncwarp();
                        qk++;
                    }
                }
            }
            if (!ok && lane == 0) atomicExch(a.status, (int)DEV_TIMEOUT);
            __syncwarp();
            // every product issued is complete before the tensor memory is freed
            if (leader) mma_commit(&done[0]);
            __syncwarp();
            if (!mbar_wait_short(&done[0], 0) && lane == 0) atomicExch(a.status, (int)DEV_TIMEOUT);
            __syncwarp();
        } else if (any && warp == kValueWarp) {
            // ------------------------------------------------------------------------------ products of probabilities and values
            Cur c;
            c.set(a, a.begin[range], ua, ub);
            const bool leader = elect_one();
            constexpr uint32_t id = idesc_bf16(128, D) | 1u << 16;  // the second operand's columns run along memory
            const uint32_t r0 = saddr(ring);
            int n = 0;
            int segs[2] = {0, 0}, pv[2] = {0, 0};
            for (; c.more() && ok; c.next(a)) {
                const int nt = c.cnt, both = T == 2 && c.rows(a) > 128;
                for (int j = 0; j < nt && ok; j++, n++) {
                    const int v = 2 * n + 1, slot = v % NS;
                    for (int t = 0; t <= both && ok; t++) {
                        bool w = wait_both(&full[v % (2 * NS)], (v / (2 * NS)) & 1, &pfull[2 * t], pv[t] & 1);
                        if (j == 0) {
                            if (segs[t] > 0) w = w && mbar_wait_short(&ofree[t], (segs[t] - 1) & 1);
                            segs[t]++;
                        }
                        ok = __all_sync(0xFFFFFFFFu, w);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t vd = values_desc(r0 + slot * L::tile, L::half);
                        const uint32_t od = tmem + L::o + t * D, pd = tmem + L::p + t * 64;
                        if (leader) {
#pragma unroll
                            for (int k = 0; k < kTile / 32; k++) mma_ts(od, pd + 8 * k, vd + k * (2048 >> 4), id, j > 0 || k > 0);
                        }
                        __syncwarp();
                        ok = __all_sync(0xFFFFFFFFu, mbar_wait_short(&pfull[2 * t + 1], pv[t] & 1));
                        if (!ok) break;
                        tc_fence_after();
                        if (leader) {
#pragma unroll
                            for (int k = kTile / 32; k < kTile / 16; k++) mma_ts(od, pd + 8 * k, vd + k * (2048 >> 4), id, 1);
                            mma_commit(&pvdone[t]);
                            if (t == both) mma_commit(&empty[slot]);
                        }
                        __syncwarp();
                        pv[t]++;
                    }
                }
            }
            if (!ok && lane == 0) atomicExch(a.status, (int)DEV_TIMEOUT);
            __syncwarp();
            if (leader) mma_commit(&done[1]);
            __syncwarp();
            if (!mbar_wait_short(&done[1], 0) && lane == 0) atomicExch(a.status, (int)DEV_TIMEOUT);
            __syncwarp();
        }
    } else {
        if constexpr (T == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        if (any) {
            // ------------------------------------------------------------------------------ softmax
            const int t = warp >> 2, row = threadIdx.x & 127;
            const uint32_t t_lane = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
            Cur c;
            c.set(a, a.begin[range], ua, ub);
            int steps = 0;                  // scores seen, also products of P and V asked for
            // Stores and loads of tensor memory follow it, which are the whole warp's: it ends as it began
            auto arrive = [&](uint64_t *b) {
                __syncwarp();
                if (lane == 0) mbar_arrive(b);
                __syncwarp();
            };
            auto wait = [&](uint64_t *b, uint32_t parity) {
                if (ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait_short(b, parity));
            };
            // an item's queries of this tile, 16 threads a row
            auto queries = [&](const Cur &q) {
                const int x0 = q.rt * kRows + 128 * t, xn = q.w.q.n * a.group;
                constexpr int kC = D / 8, kStep = 128 / kC;     // 16-byte pieces of a row, rows of a round
                const int ch = row % kC;
                int r = row / kC, tok = (int)(((uint32_t)x0 + r) / (uint32_t)a.group), h = (int)((uint32_t)x0 + r - (uint32_t)tok * a.group);
                const int dt = kStep / a.group, dh = kStep % a.group;
                const uint16_t *src = a.q + q.w.q.first * a.ldq + (int64_t)(q.head * a.group) * D + 8 * ch;
#pragma unroll 1
                for (int b = 0; b < 128 / kStep; b += 8) {
                    uint4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        v[i] = make_uint4(0, 0, 0, 0);
                        if (x0 + r + i * kStep < xn) v[i] = *(const uint4 *)(src + tok * a.ldq + h * D);
                        tok += dt;
                        h += dh;
                        if (h >= a.group) {
                            h -= a.group;
                            tok++;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; i++, r += kStep) {
                        v[i].x = (v[i].x & g.q_and) ^ g.q_xor;
                        v[i].y = (v[i].y & g.q_and) ^ g.q_xor;
                        v[i].z = (v[i].z & g.q_and) ^ g.q_xor;
                        v[i].w = (v[i].w & g.q_and) ^ g.q_xor;
                        *(uint4 *)(qs + t * L::tile + (ch >> 3) * L::half + r * 128 + ((ch & 7) ^ (r & 7)) * 16) = v[i];
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                arrive(&qfull[t]);
            };
            if (c.more() && c.rows(a) > 128 * t) queries(c);
            while (c.more()) {
                const int nt = c.cnt;
                const bool begins = c.begins(), ends = c.ends();
                Cur nx = c;
                nx.next(a);
                if (c.rows(a) <= 128 * t) {   // the item has no such tile
                    c = nx;
                    if (c.more() && c.rows(a) > 128 * t) queries(c);
                    continue;
                }
                // this thread's row, and the keys [from, upto) that it sees
                const int64_t x = (int64_t)c.rt * kRows + 128 * t + row;
                const bool in = x < (int64_t)c.w.q.n * a.group;
                const int tok = in ? (int)x / a.group : 0;
                const int64_t pos = (int64_t)c.w.q.len - c.w.q.n + tok;
                const int upto = !in ? 0 : a.causal ? (int)min(max(pos + 1, (int64_t)0), (int64_t)c.w.keys) : c.w.keys;
                const int from = a.window ? (int)max(pos - a.window + 1, (int64_t)0) : 0;
                float m = kNegInf;            // what the powers are relative to, in powers of 2
                Pair l2 = pair(0.f, 0.f);
                for (int j = 0; j < nt; j++) {
                    const int key0 = (c.k.t0 + c.off + j) * kTile;
                    wait(&sfull[t], steps & 1);
                    tc_fence_after();
                    uint32_t s[4][32];
#pragma unroll
                    for (int q = 0; q < 4; q++) tmem_ld32(t_lane + L::s + 32 * q, s[q]);
                    tmem_wait_ld();
                    tc_fence_before();
                    arrive(sfree);
                    if (__any_sync(0xFFFFFFFFu, key0 < from || key0 + kTile > upto)) {
                        const int lo = from - key0, hi = upto - key0;
#pragma unroll
                        for (int i = 0; i < 128; i++)
                            if (i < lo || i >= hi) s[i >> 5][i & 31] = __float_as_uint(kNegInf);
                    }
                    float mx[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
                    for (int i = 0; i < 128; i += 8)
#pragma unroll
                        for (int q = 0; q < 4; q++)
                            mx[q] = max3(mx[q], __uint_as_float(s[i >> 5][(i & 31) + 2 * q]), __uint_as_float(s[i >> 5][(i & 31) + 2 * q + 1]));
                    const float ms = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale2;
                    bool waited = steps == 0 || __all_sync(0xFFFFFFFFu, mbar_poll(&pvdone[t], (steps - 1) & 1));  // the product before
                    if (j == 0) m = ms;
                    else if (__any_sync(0xFFFFFFFFu, ms > m + kGrow)) {
                        // the output so far, in other powers
                        const float mn = fmaxf(m, ms), f = mn == kNegInf ? 1.f : exp2_fast(m - mn);
                        m = mn;
                        l2 = mul2(l2, pair(f, f));
                        if (!waited) wait(&pvdone[t], (steps - 1) & 1);
                        waited = true;
                        tc_fence_after();
#pragma unroll 1
                        for (int q = 0; q < D / 32; q++) {
                            uint32_t o[32];
                            tmem_ld32(t_lane + L::o + t * D + 32 * q, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32(t_lane + L::o + t * D + 32 * q, o);
                        }
                        tmem_wait_st();
                    }
                    const float base = m == kNegInf ? 0.f : m;
                    const Pair sc = pair(a.scale2, a.scale2), nb = pair(-base, -base);
                    Pair acc[2] = {l2, pair(0.f, 0.f)};
#pragma unroll
                    for (int h = 0; h < 2; h++) {        // each half's product starts when it is there
                        uint32_t p[32];
#pragma unroll
                        for (int i = 64 * h; i < 64 * h + 64; i += 2) {
                            float e0, e1;
                            unpair(fma2(pair(__uint_as_float(s[i >> 5][i & 31]), __uint_as_float(s[i >> 5][(i & 31) + 1])), sc, nb), e0, e1);
                            e0 = exp2_fast(e0);
                            e1 = exp2_fast(e1);
                            acc[(i >> 1) & 1] = add2(acc[(i >> 1) & 1], pair(e0, e1));
                            p[(i & 63) >> 1] = pack2(e0, e1);
                        }
                        if (h == 0) {
                            if (!waited) wait(&pvdone[t], (steps - 1) & 1);   // the product before has read P
                            tc_fence_after();
                        }
                        tmem_st32(t_lane + L::p + t * 64 + 32 * h, p);
                        tmem_wait_st();
                        tc_fence_before();
                        arrive(&pfull[2 * t + h]);
                    }
                    l2 = add2(acc[0], acc[1]);
                    steps++;
                }
                // the last scores are in: the products are done with the queries
                if (nx.more() && nx.rows(a) > 128 * t) queries(nx);
                wait(&pvdone[t], (steps - 1) & 1);
                tc_fence_after();
                float la, lb;
                unpair(l2, la, lb);
                const float l = la + lb;
                if (begins && ends) {
                    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
                    const int h = c.head * a.group + (in ? (int)x - tok * a.group : 0);
                    const int64_t r = c.w.q.first + tok;
                    uint16_t *o = a.out + r * a.ldo + (int64_t)h * D;
#pragma unroll 1
                    for (int q = 0; q < D / 32; q++) {
                        uint32_t v[32];
                        tmem_ld32(t_lane + L::o + t * D + 32 * q, v);
                        tmem_wait_ld();
                        if (in) {
#pragma unroll
                            for (int i = 0; i < 32; i += 8) {
                                uint4 w;
                                w.x = pack2(__uint_as_float(v[i]) * inv, __uint_as_float(v[i + 1]) * inv);
                                w.y = pack2(__uint_as_float(v[i + 2]) * inv, __uint_as_float(v[i + 3]) * inv);
                                w.z = pack2(__uint_as_float(v[i + 4]) * inv, __uint_as_float(v[i + 5]) * inv);
                                w.w = pack2(__uint_as_float(v[i + 6]) * inv, __uint_as_float(v[i + 7]) * inv);
                                *(uint4 *)(o + 32 * q + i) = w;
                            }
                        }
                        __syncwarp();     // rows are left out above, the next load is the whole warp's
                    }
                    if (in && a.lse) a.lse[r * a.q_heads + h] = l == 0.f ? kNegInf : (m + log2f(l)) * 0.69314718f;
                    __syncwarp();
                } else {
                    // pieces of four columns of all rows: a warp's stores are 512 bytes in a row
                    float *o = a.part + (2 * (size_t)range + (begins ? 1 : 0)) * slot_floats<kRows, D>();
                    const int r = 128 * t + row;
#pragma unroll 1
                    for (int q = 0; q < D / 32; q++) {
                        uint32_t v[32];
                        tmem_ld32(t_lane + L::o + t * D + 32 * q, v);
                        tmem_wait_ld();
                        if (in) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4) __stcg((uint4 *)(o + ((32 * q + i) / 4 * kRows + r) * 4), make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]));
                        }
                        __syncwarp();     // as above
                    }
                    if (in) {
                        __stcg(o + kRows * D + r, m);
                        __stcg(o + kRows * D + kRows + r, l);
                    }
                    __syncwarp();
                    tc_fence_before();
                    arrive(&ofree[t]);
                    // the part that comes last joins them all
                    const int r0 = c.first_range(C), parts = c.last_range(C) - r0 + 1;
                    __threadfence();
                    tile_sync(t);
                    if (row == 0) last[t] = atomicAdd(&a.arrived[2 * r0 + t], 1) == parts - 1;
                    __syncwarp();
                    tile_sync(t);
                    if (last[t] && in) {
                        __threadfence();
                        join_row<D, kRows>(a, c, r0, parts, r, tok, (int)x);
                    }
                    __syncwarp();
                    c = nx;
                    continue;
                }
                tc_fence_before();
                arrive(&ofree[t]);
                c = nx;
            }
            if (!ok && lane == 0) atomicExch(a.status, (int)DEV_TIMEOUT);
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kScoreWarp) {
        __syncwarp();
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <int D, int T>
cudaError_t launch_tc(const uw_kv_cache *c, const AttendCall &call, int ctas, cudaStream_t st)
{
    static OncePerDevice once;
    cudaError_t e = allow_shared(once, attend_tc_kernel<D, T>, Layout<D, T>::smem);
    if (e != cudaSuccess) return e;
    Args g;
    g.km = c->k128;
    g.vm = c->v128;
    g.c = call;
    g.c.box = c->box128;
    g.q_xor = call.scale2 < 0.f ? 0x80008000u : 0u;
    g.q_and = call.scale2 == 0.f ? 0u : 0xFFFFFFFFu;
    g.c.scale2 = call.scale2 == 0.f ? 1.f : std::fabs(call.scale2);
    if ((e = (cudaError_t)launch_attend_plan(g.c, 128 * T, ctas, st)) != cudaSuccess) return e;
    return launch_dependent(attend_tc_kernel<D, T>, dim3((unsigned)ctas), 128 * (T + 1), Layout<D, T>::smem, 0, st, g);
}

}  // namespace

int launch_attend_tc(const uw_kv_cache *c, const AttendCall &a, int rows, int ctas, void *stream)
{
    const cudaStream_t st = (cudaStream_t)stream;
    if (c->d.head_dim == 128) return rows == 128 ? launch_tc<128, 1>(c, a, ctas, st) : launch_tc<128, 2>(c, a, ctas, st);
    return rows == 128 ? launch_tc<64, 1>(c, a, ctas, st) : launch_tc<64, 2>(c, a, ctas, st);
}

}  // namespace uw
