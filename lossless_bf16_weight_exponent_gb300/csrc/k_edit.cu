// k_edit.cu - penalties for repeated tokens, biases and grammar masks on rows of logits (sm_103a).
//
// A CTA has a slice of one row's vocabulary, whose logits it asks for first.  It looks through the row's whole history (from L2,
// which all slices of the row share) and counts, for each token of its slice, in a word of shared memory: bits 0-23 how often
// it was generated, bit 31 that it is in the prompt.  The additions are of whole numbers, so their order does not matter.  A token
// that the row's biases name is edited by the thread of its first entry, which adds the others in the list's order (bit 30
// tells the rest to pass it over).  Then one pass over the slice: a word of 0 and an allowed token leave a logit as it is.
// (A list of the tokens with edits, made as the words are counted and gone through behind a pass that looks at no word, was slower
// in fp32: 70 us against 56, for its atomics with answers and its scattered stores.)
// Out of place a logit is read and written once, unless a 16-byte piece is masked out as a whole, which is not read.  In
// place a piece in which nothing changes is neither read nor written.
// Bound by issue slots (79 % busy) beside memory: 256 rows of 128256 fp32, each with 1500 to 3000 tokens of history and every second one masked, take 57.2 us
// (4.7 TB/s; 48.8 without histories, which every slice of a row looks through; in place 50); 1 row 5.0 us with 8 biases, 3.9 without; 96
// rows of 32003 bf16 with 300 biases each, their rows not aligned, 18.3 us (11.7 without biases; 8.5 of 32000 without, aligned; in place 14.7).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "launch.cuh"
#include "uw_internal.h"

using namespace uw;

namespace {

constexpr int kThreads = 512;
constexpr int kSlice = 8192;   // tokens of a CTA at most: 32 KB of counts
constexpr int kMaxBias = 4096;
constexpr int kPlaceBits = 13;
static_assert(kSlice == 1 << kPlaceBits, "a token's place in the slice, and above it that of an entry in 4096");
constexpr uint32_t kSeen = 1u << 31, kBias = 1u << 30, kCount = (1u << 24) - 1;

struct EditArgs {
    uw_logit_edits e;
    const void *logits;
    void *out;
    int64_t vocab, ld, ld_out;
    int slice;                // tokens of a CTA, a multiple of 32
};

template <bool F32>
__device__ __forceinline__ float value_of(const void *p, int64_t i)
{
    if constexpr (F32) return ((const float *)p)[i];
    else return __uint_as_float((uint32_t)((const uint16_t *)p)[i] << 16);
}

template <bool F32>
__device__ __forceinline__ void put(void *p, int64_t i, float x)
{
    if constexpr (F32) ((float *)p)[i] = x;
    else ((__nv_bfloat16 *)p)[i] = __float2bfloat16_rn(x);
}

struct Row {
    float rep, inv, up, freq, pres;
    // x / rep is (x inv) up, with up a power of 2 for which inv is an ordinary number: 1 / rep alone is infinite for a rep below
    // 2^-126 and short of bits for one above 2^126, where the quotient is neither.
    __device__ __forceinline__ void repetition(float x)
    {
        rep = x;
        up = fabsf(x) < 0x1p-126f ? 0x1p64f : fabsf(x) > 0x1p126f ? 0x1p-64f : 1.f;
        inv = 1.f / (x * up);
    }
};

// The penalties; without a branch by token, as a few tokens of most warps have some.  The quotient is a product with the reciprocal, a
// rounding of fp32 more (256 rows of 128256 take 57.2 us; 89.5 with a division, 55.9 without the power of 2).
__device__ __forceinline__ float edited(float x, uint32_t w, const Row &r)
{
    const uint32_t c = w & kCount;
    const bool over = x > 0.f;
    const float y = x * (over ? r.inv : r.rep) * (over ? r.up : 1.f);
    x = (w & (kSeen | kCount)) ? y : x;
    const float d = r.freq * (float)c + r.pres;
    return c ? x - d : x;
}

// W: logits of a piece (8 of bf16, 4 of fp32 inputs; 1: rows without 16-byte alignment).  Four CTAs an SM, for which a few
// registers go to memory, hide more of a CTA's phases from one another: 256 rows of 128256 fp32, half of them masked, took 55.9 us
// against 64.7 with two (57.2 now, with the penalties' power of 2).
template <bool F32, bool OUT32, int W, bool PLACE>
__global__ void __launch_bounds__(kThreads, 4) edit_kernel(const EditArgs a)
{
    constexpr uint32_t kAll = (1u << W) - 1;
    constexpr int U = kSlice / (kThreads * W);            // pieces of a thread
    constexpr int kWords = W == 1 ? 1 : 4;                // of a piece as loaded
    extern __shared__ uint32_t words[];
    __shared__ int counts[kThreads / 32];
    const int64_t row = blockIdx.y;
    const int64_t v0 = (int64_t)blockIdx.x * a.slice;
    const int n = (int)min((int64_t)a.slice, a.vocab - v0);
    const int whole = n / W * W;
    pdl_trigger();
    for (int i = threadIdx.x; i < n; i += kThreads) words[i] = 0;
    pdl_wait();
    // what the row's edits are, then its mask, history and logits, each as soon as it can be asked for
    const int64_t which = a.e.allowed ? (a.e.mask_rows ? a.e.mask_rows[row] : row) : -1;
    int len = 0, prompt = 0, n_bias = 0;
    if (a.e.tokens) {
        len = (int)min((int64_t)max(a.e.lengths[row], 0), a.e.max_tokens);
        if (a.e.prompt_lengths) prompt = a.e.prompt_lengths[row];
    }
    if (a.e.bias_ids) {
        n_bias = (int)a.e.max_bias;
        if (a.e.bias_lengths) n_bias = min(max(a.e.bias_lengths[row], 0), n_bias);
    }
    Row r;
    r.repetition(a.e.repetition ? a.e.repetition[row] : 1.f);
    r.freq = a.e.frequency ? a.e.frequency[row] : 0.f;
    r.pres = a.e.presence ? a.e.presence[row] : 0.f;
    const uint32_t *mask = which >= 0 && which < a.e.mask_count ? a.e.allowed + which * a.e.ld_allowed + v0 / 32 : nullptr;
    const int32_t *tokens = a.e.tokens + row * a.e.ld_tokens;
    int32_t id[8];                    // of the history, eight of a thread on their way
    auto history = [&](int i0) {
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int i = i0 + j * kThreads + threadIdx.x;
            id[j] = i < len ? tokens[i] : -1;
        }
    };
    history(0);
    const uint8_t *in = (const uint8_t *)a.logits + (row * a.ld + v0) * (F32 ? 4 : 2);
    uint8_t *out = (uint8_t *)a.out + (row * a.ld_out + v0) * (OUT32 ? 4 : 2);
    auto at = [&](int u) { return (u * kThreads + (int)threadIdx.x) * W; };
    // the slice's logits are on their way while the history is looked through
    uint32_t ok[U] = {}, raw[U][kWords];
    auto fetch = [&](int u) {
#pragma unroll
        for (int q = 0; q < kWords; q++) raw[u][q] = 0;
        if (at(u) >= whole || !ok[u]) return;
        if constexpr (W == 1) {
            if constexpr (F32) raw[u][0] = ((const uint32_t *)in)[at(u)];
            else raw[u][0] = (uint32_t)((const uint16_t *)in)[at(u)] << 16;
        } else {
            const uint4 v = *(const uint4 *)(in + (int64_t)at(u) * (F32 ? 4 : 2));
            raw[u][0] = v.x;
            raw[u][1] = v.y;
            raw[u][2] = v.z;
            raw[u][3] = v.w;
        }
    };
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int p = at(u);
        ok[u] = p >= whole ? 0u : mask ? (mask[p >> 5] >> (p & 31)) & kAll : kAll;
    }
    if (!PLACE) {
#pragma unroll
        for (int u = 0; u < U; u++) fetch(u);
    }
    const float *bias = a.e.bias + row * a.e.max_bias;
    __syncthreads();
    for (int i0 = 0; i0 < len; i0 += 8 * kThreads) {
        if (i0) history(i0);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const int64_t v = (int64_t)id[j] - v0;
            if (v < 0 || v >= n) continue;
            if (i0 + j * kThreads + (int)threadIdx.x >= prompt) atomicAdd(&words[v], 1u);
            else atomicOr(&words[v], kSeen);
        }
    }
    __syncthreads();
    if (n_bias) {
        // The entries of the slice's tokens, in the list's order: the token's place in the slice below its place in the list
        uint32_t *list = words + a.slice;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        int m = 0;
        for (int i0 = 0; i0 < n_bias; i0 += kThreads) {
            const int i = i0 + threadIdx.x;
            const int64_t p = i < n_bias ? (int64_t)a.e.bias_ids[row * a.e.max_bias + i] - v0 : -1;
            const bool here = p >= 0 && p < n;
            const unsigned among = __ballot_sync(0xFFFFFFFFu, here);
            if (lane == 0) counts[warp] = __popc(among);
            __syncthreads();
            int front = 0, all = 0;
            for (int k = 0; k < kThreads / 32; k++) {
                front += k < warp ? counts[k] : 0;
                all += counts[k];
            }
            if (here) list[m + front + __popc(among & ((1u << lane) - 1u))] = (uint32_t)p | (uint32_t)i << kPlaceBits;
            m += all;
            __syncthreads();
        }
        // A token with biases is one thread's, that of its first entry, from its logit to its output; the pass below leaves it out.
        for (int k = threadIdx.x; k < m; k += kThreads) {
            const uint32_t e = list[k];
            const int p = (int)(e & (kSlice - 1));
            const bool allowed = !mask || ((mask[p >> 5] >> (p & 31)) & 1u);
            float x = value_of<F32>(in, p);
            const float own = bias[e >> kPlaceBits];
            int before = 0, after = 0;                     // other entries of the token
#pragma unroll 4
            for (int j = 0; j < m; j++) {
                const bool same = ((list[j] ^ e) & (kSlice - 1)) == 0;
                before += same && j < k;
                after += same && j > k;
            }
            if (before) continue;
            x = edited(x, words[p], r) + own;
            for (int j = k + 1; after; j++) {
                if ((list[j] ^ e) & (kSlice - 1)) continue;
                x += bias[list[j] >> kPlaceBits];
                after--;
            }
            if (!allowed) x = -INFINITY;
            put<OUT32>(out, p, x);
            words[p] |= kBias;          // the others' threads do not look at this token's word
        }
        __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int p = at(u);
        if (p >= whole) break;
        uint32_t w[W], any = 0;
        if constexpr (W == 1) {
            any = w[0] = words[p];
        } else {
#pragma unroll
            for (int q = 0; q < W; q += 4) {
                const uint4 v = *(const uint4 *)(words + p + q);
                w[q] = v.x;
                w[q + 1] = v.y;
                w[q + 2] = v.z;
                w[q + 3] = v.w;
                any |= v.x | v.y | v.z | v.w;
            }
        }
        if (PLACE) {
            if (!any && ok[u] == kAll) continue;
            fetch(u);
        }
        float x[W];
#pragma unroll
        for (int q = 0; q < W; q++) {
            if constexpr (F32 || W == 1) x[q] = __uint_as_float(raw[u][q]);
            else x[q] = __uint_as_float((q & 1) ? raw[u][q / 2] & 0xFFFF0000u : raw[u][q / 2] << 16);
            if (any) x[q] = edited(x[q], w[q], r);
            if (!((ok[u] >> q) & 1u)) x[q] = -INFINITY;
        }
        if (W == 1 || (any & kBias)) {
#pragma unroll
            for (int q = 0; q < W; q++)
                if (!(w[q] & kBias)) put<OUT32>(out, p + q, x[q]);
            continue;
        }
        if constexpr (W > 1) {
            uint8_t *o = out + (int64_t)p * (OUT32 ? 4 : 2);
            if constexpr (OUT32) {
#pragma unroll
                for (int q = 0; q < W; q += 4) *(float4 *)(o + 4 * q) = make_float4(x[q], x[q + 1], x[q + 2], x[q + 3]);
            } else {
                uint32_t h[W / 2];
#pragma unroll
                for (int q = 0; q < W; q += 2) {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(x[q], x[q + 1]);
                    h[q / 2] = *(const uint32_t *)&v;
                }
                if constexpr (W == 8) *(uint4 *)o = make_uint4(h[0], h[1], h[2], h[3]);
                else *(uint2 *)o = make_uint2(h[0], h[1]);
            }
        }
    }
    // the rest of a row that is not a number of pieces
    const int p = whole + threadIdx.x;
    if (p < n) {
        const uint32_t w = words[p];
        const bool allowed = !mask || ((mask[p >> 5] >> (p & 31)) & 1u);
        if (!(w & kBias) && (!PLACE || w || !allowed)) put<OUT32>(out, p, allowed ? edited(value_of<F32>(in, p), w, r) : -INFINITY);
    }
}

template <bool F32, bool OUT32, int W, bool PLACE>
cudaError_t launch_one(const EditArgs &a, dim3 grid, cudaStream_t st)
{
    auto kernel = edit_kernel<F32, OUT32, W, PLACE>;
    static OncePerDevice once;
    const cudaError_t e = allow_shared(once, kernel, (kSlice + kMaxBias) * 4);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, grid, kThreads, (size_t)a.slice * 4 + (a.e.bias_ids ? (size_t)a.e.max_bias * 4 : 0), 0, st, a);
}

template <bool F32, bool OUT32>
cudaError_t launch_types(const EditArgs &a, int64_t rows, bool wide, bool place, cudaStream_t st)
{
    constexpr int W = F32 ? 4 : 8;
    const dim3 grid((unsigned)((a.vocab + a.slice - 1) / a.slice), (unsigned)rows);
    if constexpr (F32 == OUT32) {
        if (place) return wide ? launch_one<F32, OUT32, W, true>(a, grid, st) : launch_one<F32, OUT32, 1, true>(a, grid, st);
    }
    return wide ? launch_one<F32, OUT32, W, false>(a, grid, st) : launch_one<F32, OUT32, 1, false>(a, grid, st);
}

bool aligned(const void *p, unsigned n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace

extern "C" uw_status uw_edit_logits(const uw_logit_edits *e, const void *logits, uw_out_dtype dtype, int64_t rows, int64_t vocab, int64_t ld,
                                    void *out, uw_out_dtype out_dtype, int64_t ld_out, uw_stream stream)
{
    clear_error();
    if (!e) return fail(UW_ERR_INVALID_ARG, "uw_edit_logits: NULL edits");
    if (ld == 0) ld = vocab;
    if (ld_out == 0) ld_out = vocab;
    const int64_t most = (int64_t)1 << 40;
    if (rows < 0 || rows > ((int64_t)1 << 31) - 1024 || vocab < 1 || vocab > (1 << 24) || ld < vocab || ld_out < vocab || ld > most || ld_out > most)
        return fail(UW_ERR_SHAPE, "uw_edit_logits: rows=%lld vocab=%lld ld=%lld ld_out=%lld", (long long)rows, (long long)vocab, (long long)ld, (long long)ld_out);
    if ((dtype != UW_OUT_F32 && dtype != UW_OUT_BF16) || (out_dtype != UW_OUT_F32 && out_dtype != UW_OUT_BF16))
        return fail(UW_ERR_INVALID_ARG, "uw_edit_logits: bad dtype");
    const bool f32 = dtype == UW_OUT_F32, o32 = out_dtype == UW_OUT_F32;
    EditArgs a{*e, logits, out, vocab, ld, ld_out, 0};
    if (a.e.tokens) {
        if (!a.e.lengths) return fail(UW_ERR_INVALID_ARG, "uw_edit_logits: tokens without lengths");
        if (a.e.ld_tokens == 0) a.e.ld_tokens = a.e.max_tokens;
        if (a.e.max_tokens < 0 || a.e.max_tokens >= (1 << 24) || (rows > 1 && a.e.ld_tokens < a.e.max_tokens) || a.e.ld_tokens > most)
            return fail(UW_ERR_SHAPE, "uw_edit_logits: max_tokens=%lld ld_tokens=%lld", (long long)a.e.max_tokens, (long long)a.e.ld_tokens);
    } else if (a.e.repetition || a.e.frequency || a.e.presence) {
        return fail(UW_ERR_INVALID_ARG, "uw_edit_logits: penalties without tokens");
    }
    if (!a.e.repetition && !a.e.frequency && !a.e.presence) a.e.tokens = nullptr;  // nothing looks at them
    if (!a.e.bias_ids != !a.e.bias) return fail(UW_ERR_INVALID_ARG, "uw_edit_logits: bias_ids and bias go together");
    if (a.e.max_bias < 0 || a.e.max_bias > kMaxBias) return fail(UW_ERR_SHAPE, "uw_edit_logits: max_bias=%lld", (long long)a.e.max_bias);
    const int64_t words = (vocab + 31) / 32;
    if (a.e.allowed) {
        if (a.e.ld_allowed == 0) a.e.ld_allowed = words;
        if (a.e.mask_count < 0 || a.e.ld_allowed < words || a.e.ld_allowed > most)
            return fail(UW_ERR_SHAPE, "uw_edit_logits: mask_count=%lld ld_allowed=%lld", (long long)a.e.mask_count, (long long)a.e.ld_allowed);
    }
    for (const void *p : {(const void *)a.e.tokens, (const void *)a.e.lengths, (const void *)a.e.prompt_lengths, (const void *)a.e.repetition,
                          (const void *)a.e.frequency, (const void *)a.e.presence, (const void *)a.e.bias_ids, (const void *)a.e.bias,
                          (const void *)a.e.bias_lengths, (const void *)a.e.allowed, (const void *)a.e.mask_rows})
        if (!aligned(p, 4)) return fail(UW_ERR_INVALID_ARG, "uw_edit_logits: a pointer is not 4-byte aligned");
    if (!aligned(logits, f32 ? 4 : 2) || !aligned(out, o32 ? 4 : 2)) return fail(UW_ERR_INVALID_ARG, "uw_edit_logits: logits or out not aligned to their elements");
    if (rows == 0) return UW_OK;
    if (!logits || !out) return fail(UW_ERR_INVALID_ARG, "uw_edit_logits: logits or out NULL");
    const bool place = logits == out && f32 == o32 && (ld == ld_out || rows == 1);
    if (!place && rows_overlap({logits, ld * (f32 ? 4 : 2), vocab * (f32 ? 4 : 2)}, {out, ld_out * (o32 ? 4 : 2), vocab * (o32 ? 4 : 2)}, rows))
        return fail(UW_ERR_INVALID_ARG, "uw_edit_logits: out overlaps logits (it may be logits itself, with their type and ld)");
    if (place && !a.e.tokens && !a.e.bias_ids && !a.e.allowed) return UW_OK;
    // rows of 16-byte pieces; out's pieces are of as many logits
    const int W = f32 ? 4 : 8;
    const bool wide = aligned(logits, 16) && aligned(out, W * (o32 ? 4 : 2) >= 16 ? 16 : 8) && (rows == 1 || (ld % W == 0 && ld_out % W == 0));
    // A slice of 8192 tokens (32 KB of counts); smaller ones for few rows, so that the GPU is full.
    a.slice = kSlice;
    while (a.slice > 1024 && rows * ((vocab + a.slice - 1) / a.slice) < 2 * num_sms()) a.slice /= 2;
    for (int64_t r0 = 0; r0 < rows; r0 += 65535) {  // the grid's second dimension
        const int64_t n = std::min<int64_t>(rows - r0, 65535);
        EditArgs b = a;
        b.logits = (const uint8_t *)a.logits + r0 * ld * (f32 ? 4 : 2);
        b.out = (uint8_t *)a.out + r0 * ld_out * (o32 ? 4 : 2);
        if (b.e.tokens) {
            b.e.tokens += r0 * a.e.ld_tokens;
            b.e.lengths += r0;
            if (b.e.prompt_lengths) b.e.prompt_lengths += r0;
        }
        if (b.e.repetition) b.e.repetition += r0;
        if (b.e.frequency) b.e.frequency += r0;
        if (b.e.presence) b.e.presence += r0;
        if (b.e.bias_ids) {
            b.e.bias_ids += r0 * a.e.max_bias;
            b.e.bias += r0 * a.e.max_bias;
            if (b.e.bias_lengths) b.e.bias_lengths += r0;
        }
        if (b.e.allowed && b.e.mask_rows) b.e.mask_rows += r0;
        else if (b.e.allowed) {
            b.e.allowed += r0 * a.e.ld_allowed;
            b.e.mask_count = std::max<int64_t>(a.e.mask_count - r0, 0);
        }
        const cudaError_t x = f32 ? (o32 ? launch_types<true, true>(b, n, wide, place, (cudaStream_t)stream) : launch_types<true, false>(b, n, wide, place, (cudaStream_t)stream))
                                  : (o32 ? launch_types<false, true>(b, n, wide, place, (cudaStream_t)stream) : launch_types<false, false>(b, n, wide, place, (cudaStream_t)stream));
        if (x != cudaSuccess) return fail(UW_ERR_CUDA, "uw_edit_logits: launch: %s", cudaGetErrorString(x));
    }
    return UW_OK;
}
