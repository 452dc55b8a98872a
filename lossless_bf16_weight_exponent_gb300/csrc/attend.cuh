// attend.cuh - the call of uw_kv_attend as its kernels take it, and how its work is cut.
//
// An item is a tile of R query rows of a sequence (its new tokens' query heads that share a key head) against one key head;
// a unit is one of its tiles of 128 keys.  The work is a line: item after item - sequence, key head, tile of rows - each with
// kItem units of its own, for what it costs beside its keys, and then its tiles.  The line is cut into a range of as many units
// for each CTA wherever these end, so that all have as much to do whatever the lengths are.  A first, small kernel measures
// the line and writes down where each range begins.
// An item that lies in one range is stored by the CTA that has the range; of an item that is cut each CTA leaves its sums (the running
// maximum, the sum of powers, the unnormalised output) in the workspace, and the one that comes last joins them, in the line's
// order, so that the result does not depend on which that is.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dev_async.cuh"
#include "kv.cuh"

namespace uw {

struct AttendCall {
    KvBatch b;
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    int64_t ldq, ldo;
    int q_heads, kv_heads, group;     // group: query heads of a key head
    int page_size, pages, box;        // box: slots of a copy
    int causal, window;               // window 0: none
    float scale2;                     // scale * log2(e)
    // workspace
    struct PlanHead *plan;
    struct Start *begin;              // [ranges]
    int *arrived;                     // [2 ranges]: parts of an item that are there, by the range that it begins in (and the tile of rows)
    int64_t *line;                    // [sequences + 1], for more sequences than fit in shared memory
    float *part;                      // [ranges][2] places
    int *status;
};

// What the first kernel finds out.
struct PlanHead {
    int64_t units, per;               // of the line, of a range
    int ranges;
};

// where a range begins: the item that holds its first unit, where that begins in the line, and its sequence
struct Start {
    int64_t at;
    int s, head, i;                   // i: place of the tile of rows
    KvSeq q;
};

constexpr int kKeys = 128;            // keys of a tile

struct Seq {
    KvSeq q;
    int keys, row_tiles;              // keys: slots that the table reaches, at most its length
};

template <int R>
__device__ __forceinline__ Seq seq_of(const AttendCall &a, const KvSeq &q)
{
    Seq w;
    w.q = q;
    w.keys = min(w.q.len, a.b.capacity);
    w.row_tiles = (int)(((uint32_t)w.q.n * (uint32_t)a.group + (R - 1)) / R);
    return w;
}

template <int R>
__device__ __forceinline__ Seq seq_at(const AttendCall &a, int s) { return seq_of<R>(a, kv_seq(a.b, s)); }

// the keys [lo, hi) that some row of a tile of rows sees, and the tiles of keys [t0, t0 + nt) that hold them (one at least)
struct Span {
    int lo, hi, t0, nt;
};

template <int R>
__device__ __forceinline__ Span span_of(const AttendCall &a, int n, int len, int keys, int rt)
{
    // n x group and the tile's end are below 2^31 (the call's rows are limited)
    const uint32_t x0 = (uint32_t)rt * R, x1 = min((uint32_t)n * (uint32_t)a.group, x0 + R);
    const int i0 = (int)(x0 / (uint32_t)a.group), i1 = (int)((x1 - 1) / (uint32_t)a.group);
    const int p0 = len - n;
    Span r;
    r.hi = a.causal ? min(max(p0 + i1 + 1, 0), keys) : keys;
    r.lo = a.window ? (int)min(max((int64_t)p0 + i0 - a.window + 1, (int64_t)0), (int64_t)r.hi) : 0;
    r.t0 = r.lo / kKeys;
    r.nt = max(1, (r.hi + kKeys - 1) / kKeys - r.t0);
    return r;
}

// The i-th tile of rows of `tiles` in the line: from both ends in turn, as a causal sequence's first tiles see few keys and its
// last many, and a range should not be all short items.
__device__ __forceinline__ int tile_of(int i, int tiles) { return (i & 1) ? tiles - 1 - (i >> 1) : i >> 1; }

// An item of the line and which of its tiles of keys lie in the range [ua, ub): those [off, off + cnt).  Set, and moved on, to an
// item that has some there; more(): there was one.
template <int R, int kItem>
struct Cursor {
    Seq w;
    Span k;
    int64_t at, ua, ub;
    int s, head, i, rt, off, cnt;
    __device__ __forceinline__ void enter(const AttendCall &a)
    {
        rt = tile_of(i, w.row_tiles);
        k = span_of<R>(a, w.q.n, w.q.len, w.keys, rt);
        off = (int)max(ua - at - kItem, (int64_t)0);
        cnt = (int)(min(ub - at - kItem, (int64_t)k.nt)) - off;
    }
    __device__ __forceinline__ void set(const AttendCall &a, const Start &f, int64_t ua_, int64_t ub_)
    {
        at = f.at;
        ua = ua_;
        ub = ub_;
        s = f.s;
        head = f.head;
        i = f.i;
        w = seq_of<R>(a, f.q);
        enter(a);
        if (cnt <= 0) next(a);
    }
    __device__ __forceinline__ bool more() const { return at < ub; }
    __device__ __forceinline__ void next(const AttendCall &a)
    {
        do {
            at += k.nt + kItem;
            if (at >= ub) return;
            if (++i >= w.row_tiles) {
                i = 0;
                if (++head >= a.kv_heads) {
                    head = 0;
                    do {
                        if (++s >= a.b.sequences) {   // only where `starts` is not ascending
                            at = ub;
                            return;
                        }
                        w = seq_at<R>(a, s);
                    } while (!w.row_tiles);
                }
            }
            enter(a);
        } while (cnt <= 0);
    }
    __device__ __forceinline__ int rows(const AttendCall &a) const { return min(w.q.n * a.group - rt * R, R); }
    __device__ __forceinline__ bool begins() const { return off == 0; }
    __device__ __forceinline__ bool ends() const { return off + cnt == k.nt; }
    // the ranges that hold the item's first and last tile
    __device__ __forceinline__ int first_range(int64_t per) const { return (int)((at + kItem) / per); }
    __device__ __forceinline__ int last_range(int64_t per) const { return (int)((at + kItem + k.nt - 1) / per); }
};

// Partial sums of an item in the workspace: R rows of D, then R maxima (of 2^), then R sums.  Range r has two places: 2 r for
// the item that goes on from the range before, 2 r + 1 for the one that goes on in the next.
template <int R, int D>
__host__ __device__ constexpr size_t slot_floats() { return (size_t)R * (D + 2); }

namespace dev {

// The phase is complete, without waiting for it.
__device__ __forceinline__ bool mbar_poll(uint64_t *b, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok) : "r"(saddr(b)), "r"(parity) : "memory");
    return ok != 0;
}

// Until the phase is complete; false after 2^32 cycles (2 s).  The thread may be suspended for up to a millisecond at a time:
// polls take turns of shared memory that the tensor cores' operands need.
__device__ __forceinline__ bool mbar_sleep(uint64_t *b, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok)
                 : "r"(saddr(b)), "r"(parity), "r"(1000000u)
                 : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool mbar_wait_short(uint64_t *b, uint32_t parity)
{
    if (mbar_sleep(b, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_sleep(b, parity))
        if (clock64() - t0 > (1ll << 32)) return false;
    return true;
}

}  // namespace dev

// k_attend_tc.cu: items of 128 or 256 rows on tcgen05.  launch_attend_plan (k_attend.cu): the first kernel for them.
int launch_attend_tc(const uw_kv_cache *c, const AttendCall &a, int rows, int ctas, void *stream);
int launch_attend_plan(const AttendCall &a, int rows, int ctas, void *stream);
constexpr int kItemTc = 3;           // what an item of 128 or 256 rows costs beside its tiles of keys: queries, output, a pipeline that runs dry

}  // namespace uw
