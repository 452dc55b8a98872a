// attend.cuh - the call of uw_kv_attend as its kernels take it, and how its work is cut.
//
// The work is a line of units: tiles of keys for each item (a sequence's tile of query rows and a key head), item after item.
// CTA c of G has the units [U c / G, U (c + 1) / G), so all of them have as much to do whatever the lengths are.  An item that
// lies in one CTA's range is stored by it; of an item cut by a range's end each CTA leaves its sums (the running maximum,
// the sum of powers, the unnormalised output) in the workspace, and a second kernel joins them in the order of the CTAs.
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
    float *part;                      // [G][2] slots: sums, then maxima, then powers' sums
    struct Cut *cuts;                 // [G]
    int *status;
};

// what a CTA leaves about the item that begins in its range and goes on behind it
struct Cut {
    int64_t end, units;               // the item's last unit + 1; all units
    int valid, seq, item;
    int pad;
};

// a sequence's items for tiles of R query rows and K keys
template <int R, int K>
struct SeqWork {
    KvSeq q;
    int keys;                         // slots that the table reaches, at most its length
    int row_tiles, tile0, tiles;      // tiles of keys: [tile0, tile0 + tiles) for every item
    __device__ __forceinline__ int64_t units(const AttendCall &a) const { return (int64_t)row_tiles * a.kv_heads * tiles; }
};

template <int R, int K>
__device__ __forceinline__ SeqWork<R, K> seq_work(const AttendCall &a, int s)
{
    SeqWork<R, K> w;
    w.q = kv_seq(a.b, s);
    w.keys = min(w.q.len, a.b.capacity);
    w.row_tiles = (int)(((int64_t)w.q.n * a.group + R - 1) / R);
    const int64_t first = (int64_t)w.q.len - w.q.n - a.window + 1;  // the first key that the first token sees
    const int lo = a.window && first > 0 ? (int)min(first, (int64_t)w.keys) : 0;
    w.tile0 = lo / K;
    w.tiles = w.row_tiles ? max(1, (w.keys + K - 1) / K - w.tile0) : 0;
    return w;
}

// Partial sums of an item in the workspace: R rows of D, then R maxima (of 2^), then R sums.
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

// k_attend_tc.cu: items of 256 rows on tcgen05
size_t attend_tc_slot_floats(int D);
int launch_attend_tc(const uw_kv_cache *c, const AttendCall &a, int ctas, void *stream);

}  // namespace uw
