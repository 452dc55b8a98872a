// kv.cuh - a cache of keys and values in pages, and the new tokens of a step, as the kernels on it see them.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "uw_internal.h"

namespace uw {

// What the device knows of a step's sequences: clamped, so that no kernel leaves the call's tensors or the page table.
struct KvBatch {
    const int32_t *starts, *lengths, *pages;
    int64_t ld_pages;
    int32_t sequences, rows;
    int32_t capacity;         // slots of a row of the page table, at most 2^30
};

struct KvSeq {
    int first, n;             // rows of the call's tensors
    int len;                  // tokens, with the new ones (not clamped to the table)
};

__device__ __forceinline__ KvSeq kv_seq(const KvBatch &b, int s)
{
    KvSeq q;
    q.first = min(max(b.starts[s], 0), b.rows);
    q.n = max(min(max(b.starts[s + 1], 0), b.rows) - q.first, 0);
    q.len = max(b.lengths[s], 0);
    return q;
}

}  // namespace uw

struct uw_kv_cache {
    uw_kv_desc d;
    int device;
    int *status;              // device
    // boxes of one head: 64 elements by so many slots, the largest power of 2 up to 16 and up to 128 that divides a page
    CUtensorMap k16, v16, k128, v128;
    int box16, box128;
};

namespace uw {

uw_status check_kv_batch(const uw_kv_cache *c, const uw_kv_batch *b, int64_t rows, KvBatch *out, const char *who);
uw_status check_kv_device(const uw_kv_cache *c, const char *who);

}  // namespace uw
