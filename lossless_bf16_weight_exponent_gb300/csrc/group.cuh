// group.cuh - the compressed form of a uw_group and its rebuild, shared by the grouped kernels.
//
// A group's matrices are cut into virtual rows: of one matrix its rows; of a gated expert 16 rows of the gate matrix,
// the 16 rows of the up matrix that belong to them, the next 16 of the gate matrix, and so on, so that a kernel that
// holds 32 virtual rows holds both factors of 16 outputs.  16 virtual rows x 64 weights of K are a granule, eight
// granules (128 rows) a tile, and a tile's 64 weights of K a step.  A step is one run of 12320 bytes: 8 KB of
// sign+mantissa bytes (granule after granule), 4 KB of 4-bit exponent distances, and a record of 32 bytes, so that one
// bulk copy brings it.  Steps follow each other along K, tiles along N, experts last, so a tile is one stream of memory
// whatever N is.
//
// Within a granule, rows are (half, g) = (row / 8, row % 8) and the 64 weights of a row four chunks t of 16.  With place
// p = 4 g + (t ^ (g / 2)):
//   sign+mantissa: 16 bytes of (half, t, g) at 512 half + 16 p
//   distances:      8 bytes of (half, t, g) at 16 p + 8 half
// The matrix-vector kernel's lane 4 g + t loads its part of a granule (the tensor instruction's rows g and g + 8) with
// three 16-byte loads, eight neighbouring lanes one line of 128 bytes; and where 32 threads own a row each and read
// chunk t of it from shared memory, the exchange of chunks by g / 2 keeps them off each other's banks.
//
// A chunk's words are packed so that a pair of bf16 weights (2q, 2q + 1) takes about four instructions to rebuild.
// With P the pair's sign and mantissa bits in place (mask 807F807F) and D its two distances in place of the
// exponents' low bits (mask 07800780):
//   sign+mantissa word j = P(2j) | P(2j + 1) with the bytes of each half exchanged: the two masks are disjoint
//   distance word i      = D(4i) | D(4i + 1) << 4 | D(4i + 2) >> 4 | D(4i + 3) rotated right by 8
// and the pair is P + D + B, B the matrix's lowest exponent in both exponent fields; no sum carries out of a field,
// as the lowest exponent is at most 240 and a distance at most 15.  No table is needed (a palette of 16 arbitrary
// exponents takes a shared-memory lookup per pair, as the single-matrix kernels do).
//
// Verbatim runs: a step's record is {mask[4] (bit r: row r's run is verbatim), index of its first run, count}; the
// runs' exponent bytes are kept in (expert, tile, step, row) order, 64 each, in the order of K.
#pragma once

#include <cstdint>

#include "dev_async.cuh"

namespace uw {

constexpr int kGran = 16;                 // rows of a granule
constexpr int kTileRows = 128;            // virtual rows of a tile
constexpr int kStepW = 64;                // weights of K per step
constexpr uint32_t kStepSm = 8192;        // a step: sign+mantissa bytes, distances, record
constexpr uint32_t kStepRec = 12288;
constexpr uint32_t kStepBytes = kStepRec + 32;
constexpr int kMaxExperts = 1024;

struct StepRec {
    uint32_t mask[4];
    uint32_t first, count, pad[2];
};
static_assert(sizeof(StepRec) == 32 && kStepBytes % 16 == 0, "step record");

// device view of a group
struct GroupView {
    const uint8_t *steps;     // [experts][tiles][ksteps][kStepBytes]
    const uint8_t *verb;      // [n_verbatim][64]
    const uint32_t *base;     // [experts][1 or 2]: a matrix's lowest exponent, in both exponent fields of a pair
    int *status;
    int64_t N, K;
    int experts, gated, tiles, ksteps, granules;  // granules: virtual granules that hold rows of the matrix
};

namespace dev {

// byte of a granule's sign+mantissa half, and of its distances, where chunk t of row g (or g + 8) begins
__host__ __device__ __forceinline__ constexpr uint32_t chunk_at(int g, int t) { return 64u * g + 16u * (t ^ (g >> 1)); }

__device__ __forceinline__ const StepRec *step_rec(const uint8_t *steps, int64_t step)
{
    return (const StepRec *)(steps + step * kStepBytes + kStepRec);
}

// the eight pairs of a chunk: sign+mantissa words S, distance words C, lowest exponent B
__device__ __forceinline__ void rebuild_chunk(const uint4 &S, const uint2 &C, uint32_t B, uint32_t (&p)[8])
{
    constexpr uint32_t mp = 0x807F807Fu, md = 0x07800780u;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const uint32_t s = word_of(S, j), c = j < 2 ? C.x : C.y;
        const uint32_t d0 = (j & 1) ? (c << 4) & md : c & md;
        const uint32_t d1 = (j & 1) ? __funnelshift_l(c, c, 8) & md : (c >> 4) & md;
        p[2 * j] = (s & mp) + d0 + B;
        p[2 * j + 1] = (prmt(s, 0u, 0x2301u) & mp) + d1 + B;
    }
}

// the same from the chunk's 16 exponent bytes E
__device__ __forceinline__ void rebuild_chunk_verbatim(const uint4 &S, const uint4 &E, uint32_t (&p)[8])
{
    constexpr uint32_t mp = 0x807F807Fu, me = 0x7F807F80u;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const uint32_t s = word_of(S, j), e = word_of(E, j);
        p[2 * j] = (s & mp) | ((prmt(e, 0u, 0x4140u) << 7) & me);
        p[2 * j + 1] = (prmt(s, 0u, 0x2301u) & mp) | ((prmt(e, 0u, 0x4342u) << 7) & me);
    }
}

// silu(gate) * up by e^-|gate|, which does not overflow, so that a far negative gate keeps its small product, and the quotient's
// divisor is within [1, 2].  An fp32 output takes expf (within an ulp; the quotient is within two): 4096 tokens top 8 of 64 of
// [1408, 2048] 496 us against 488 with the fast power, and 573 with the division rounded too.  For a bf16 output, whose
// rounding is 2^-9, the fast power's 2^-16 at most is far below it.
template <bool F32>
__device__ __forceinline__ float gated(float gate, float up)
{
    const float e = F32 ? expf(-fabsf(gate)) : __expf(-fabsf(gate));
    return gate * __fdividef(gate < 0.f ? e : 1.f, 1.f + e) * up;
}

// the rank of row r's run among a step's verbatim runs
__device__ __forceinline__ uint32_t verbatim_rank(const uint32_t *mask, int r)
{
    uint32_t n = __popc(mask[r >> 5] & ((1u << (r & 31)) - 1u));
    for (int i = 0; i < (r >> 5); i++) n += __popc(mask[i]);
    return n;
}

}  // namespace dev

// one grouped product (k_group_gemv.cu, k_group_tc.cu); the launchers return cudaError_t as int
struct GroupCall {
    GroupView v;
    const uint16_t *x;
    int64_t x_rows, ldx;
    const int32_t *row_src, *offsets;
    int64_t rows;
    void *y;
    int64_t ldy;
    int out_bf16;
};
int launch_group_gemv(const GroupCall &c, void *stream);
constexpr int kSegSteps = 8;  // steps of a segment: tcgen05 sums of 512 products, which fp32 additions join for an fp32 output
inline bool group_sums(const GroupCall &c) { return !c.out_bf16 && c.v.ksteps > kSegSteps; }
bool group_tc_supported(const GroupCall &c);
int launch_group_tc(const GroupCall &c, void *stream);

}  // namespace uw
