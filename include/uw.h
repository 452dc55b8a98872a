/*
 * uw.h - C ABI of the lossless BF16 exponent codec with fused decode+matmul.
 *
 * Method: Cloudflare blog post "Unweight" (lossless compression of BF16 model
 * weights, decompressed on-chip inside the matrix multiply).  Each BF16 weight
 * is split into a raw sign+mantissa byte and an exponent byte; the exponent
 * byte is coded against a per-matrix palette of the 16 most frequent exponents
 * (4-bit codes) or with a length-limited canonical Huffman code; any run of 64
 * weights holding an exponent outside the palette is stored verbatim.
 *
 * Conventions for every entry point:
 *   - Every call returns a uw_status; nothing is thrown across the ABI.  On an
 *     error, uw_last_error() returns a message for the calling thread.
 *   - Device pointers are CUDA device addresses on the current device; host
 *     pointers are ordinary process memory.  The caller owns every buffer it
 *     passes (weights, blob, X, Y, workspace); the library owns only what a
 *     uw_matrix holds.
 *   - Device work is enqueued on the given stream (NULL = legacy default
 *     stream) and is asynchronous unless stated otherwise.  No entry point
 *     falls back to the CPU: without a CUDA device they return UW_ERR_CUDA.
 *   - Shapes: W is [N, K] row-major with K % 64 == 0 (a block is 64 weights of
 *     one row); X is [B, K] row-major bf16; Y is [B, N] row-major.  Device
 *     pointers to X, Y and workspaces must be 16-byte aligned.
 *   - Errors found by device kernels (a Huffman stream that overruns its
 *     chunk) are latched in a per-matrix status word and reported by uw_check
 *     and by the next uw_decode / uw_matmul on that matrix.
 */
#ifndef UW_H
#define UW_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t, declared without the CUDA headers. */
typedef struct CUstream_st *uw_stream;

typedef enum {
    UW_OK = 0,
    UW_ERR_INVALID_ARG = 1,   /* null pointer, misaligned pointer, bad option value */
    UW_ERR_SHAPE = 2,         /* K % 64 != 0, negative sizes, B < 0, size overflow */
    UW_ERR_UNSUPPORTED = 3,   /* strategy not available for this matrix / batch */
    UW_ERR_CORRUPT = 4,       /* blob failed validation, or a device decoder found a bad stream */
    UW_ERR_NO_MEMORY = 5,     /* host or device allocation failed */
    UW_ERR_WORKSPACE = 6,     /* workspace smaller than uw_workspace_size reports */
    UW_ERR_CUDA = 7,          /* a CUDA runtime call failed (message in uw_last_error) */
    UW_ERR_TIMEOUT = 8,       /* a bounded device wait expired */
    UW_ERR_BUFFER_TOO_SMALL = 9 /* host output buffer too small; required size returned */
} uw_status;

typedef enum { UW_CODEC_PALETTE = 0, UW_CODEC_HUFFMAN = 1 } uw_codec;

/*
 * Execution strategies: the four pipelines of the "Unweight" post (section on
 * the four execution pipelines), and a fifth that decodes inside the GEMV:
 *   FULL_DECODE        rebuild the whole BF16 matrix into the workspace, then a
 *                      plain BF16 GEMV/GEMM (the post uses cuBLAS; here a
 *                      hand-written kernel).
 *   EXP_ONLY           a preprocess kernel writes only the exponent bytes into
 *                      the workspace; the fused kernel joins them with the raw
 *                      sign+mantissa bytes.
 *   PALETTE_TRANSCODE  a preprocess kernel turns the Huffman stream into 4-bit
 *                      palette codes in the workspace; the fused kernel rebuilds
 *                      BF16 from them.
 *   DIRECT_PALETTE     no preprocessing: the fused kernel reads resident 4-bit
 *                      codes (palette codec, or a Huffman matrix loaded with its
 *                      palette form).
 *   HUFFMAN_DIRECT     no preprocessing and no palette form: one GEMV kernel
 *                      decodes the Huffman stream itself (the lookup table in
 *                      shared memory, as in the post's section on the decode
 *                      kernels) and multiplies the rebuilt weights straight away.
 *                      Huffman codec only, code lengths <= 12, chunk_weights a
 *                      divisor of K of at most 2048, 1 <= B <= 8; runs on
 *                      UW_KERNEL_GEMV with split_k 0/1 and variant 0 (plain
 *                      loads) or 1 (each work unit also prefetched into L2 in
 *                      bulk one unit ahead).  It goes beyond the post's four
 *                      pipelines.
 *   AUTO               the autotuned choice for (matrix, B), else a default:
 *                      DIRECT_PALETTE when the palette form is resident, else
 *                      HUFFMAN_DIRECT where it applies, else PALETTE_TRANSCODE.
 */
typedef enum {
    UW_STRAT_AUTO = 0,
    UW_STRAT_FULL_DECODE = 1,
    UW_STRAT_EXP_ONLY = 2,
    UW_STRAT_PALETTE_TRANSCODE = 3,
    UW_STRAT_DIRECT_PALETTE = 4,
    UW_STRAT_HUFFMAN_DIRECT = 5
} uw_strategy;

typedef enum { UW_OUT_F32 = 0, UW_OUT_BF16 = 1 } uw_out_dtype;

/*
 * What uw_load keeps on the device for a Huffman blob (a palette blob always
 * keeps its 4-bit codes and has no stream):
 *   UW_RESIDENT_HUFFMAN  the Huffman stream alone (the smallest form; the
 *                        Huffman-fed pipelines and HUFFMAN_DIRECT run on it)
 *   UW_RESIDENT_BOTH     the stream and the 4-bit palette form
 *   UW_RESIDENT_PALETTE  the 4-bit palette form alone: the stream is transcoded
 *                        at load time (the post's direct-palette form) and then
 *                        dropped, so PALETTE_TRANSCODE and HUFFMAN_DIRECT are not
 *                        available
 * Matching the post's results section, the choice trades footprint against
 * speed: the stream is about 10.8 bits per weight on Gaussian weights, the
 * palette form about 12.1.
 */
typedef enum { UW_RESIDENT_HUFFMAN = 0, UW_RESIDENT_BOTH = 1, UW_RESIDENT_PALETTE = 2 } uw_resident;

/* Matmul kernel families. */
typedef enum {
    UW_KERNEL_AUTO = 0,
    UW_KERNEL_GEMV = 1,      /* matrix-vector kernels for small B (see uw_plan.variant) */
    UW_KERNEL_TC = 2         /* tcgen05 tensor-core GEMM, W rebuilt in shared memory, fp32 in TMEM */
} uw_kernel;

typedef struct {
    uint32_t codec;          /* uw_codec */
    uint32_t chunk_weights;  /* Huffman chunk size in weights: multiple of 64, >= 64 (default 256) */
    uint32_t max_code_len;   /* Huffman length limit, 4..15 (default 12) */
} uw_encode_opts;

/* One execution plan: what uw_matmul runs for a given (matrix, B). */
typedef struct {
    int32_t strategy;        /* uw_strategy, never AUTO inside a stored plan */
    int32_t kernel;          /* uw_kernel */
    int32_t split_k;         /* K-splits (>= 1); 0 = kernel's default */
    int32_t variant;         /* kernel-specific launch shape; 0 = default.  UW_KERNEL_GEMV:
                              *   0, 2..5: bulk-copy GEMV, fp32 FMA on CUDA cores, B <= 2 (0: 8 consumer warps,
                              *            2 CTAs/SM; 2: 16 warps, 1 CTA/SM; 3: 8 warps, 1 CTA/SM in half the
                              *            shared memory; 4, 5: as 0, 2 with 64 weights per lane)
                              *   1:       plain-load GEMV, any B (batch groups of up to 8)
                              *   6, 7:    GEMV on the tensor pipe (mma.sync, fp32 accumulate), B <= 16,
                              *            K a multiple of 256 (6: K-slices of 4096 weights up to B = 8;
                              *            7: of 2048)
                              *   8:       GEMV on the tensor pipe, B <= 64, K a multiple of 256: one CTA per
                              *            SM walks an even share of the 128-row x 256-weight units, each warp
                              *            owning 8 rows (split_k ignored)
                              * UW_KERNEL_TC: 0, 1: one CTA per 128-row tile and K-slice, rebuilt tiles in shared
                              *   memory; 4: one CTA per SM over an even share of the 128-row x 256-weight units,
                              *   each 64-weight step rebuilt into shared memory (B <= 512, K a multiple of 256,
                              *   4-bit codes, split_k ignored); other values run as 0
                              * a shape that does not fit the matrix or B runs the nearest one that does */
} uw_plan;

typedef struct {
    int64_t N, K;
    uint32_t codec;
    uint32_t n_pal;
    uint8_t palette[16];
    uint8_t code_len[16];
    uint64_t n_blocks, n_verbatim, n_chunks, total_bits;
    uint64_t blob_bytes;     /* size of the serialized blob */
    uint64_t device_bytes;   /* device memory held by the uw_matrix */
    int32_t has_palette_form;/* 4-bit codes resident (DIRECT_PALETTE available) */
    int32_t chunk_weights, max_code_len;
    int32_t has_huffman_stream; /* the Huffman stream is resident (PALETTE_TRANSCODE, HUFFMAN_DIRECT available) */
} uw_info;

typedef struct uw_matrix uw_matrix;

/*
 * uw_encode - encode W[N,K] (host bf16 bit patterns, row-major) into a blob.
 *   Passages: BF16 anatomy (sign+mantissa byte kept raw), exponent statistics
 *   (top-16 palette), Huffman coding of the exponent byte, verbatim 64-weight
 *   runs.  Host-only, pure and deterministic: the bytes are a function of
 *   (W, opts) alone.  opts == NULL means palette codec.
 *   out == NULL: only *out_size is written (required size).  out != NULL and
 *   out_cap < required: UW_ERR_BUFFER_TOO_SMALL with *out_size = required.
 *   Errors: UW_ERR_SHAPE (K % 64, negative sizes), UW_ERR_INVALID_ARG (bad
 *   options), UW_ERR_UNSUPPORTED (Huffman stream of 2^32 bits or more).
 */
uw_status uw_encode(const uint16_t *w_host, int64_t N, int64_t K, const uw_encode_opts *opts,
                    void *out, size_t out_cap, size_t *out_size);

/*
 * uw_load - validate a blob fully on the host (magic, version, sizes, section
 *   bounds and alignment, bitmap/prefix/verbatim consistency, code lengths and
 *   Kraft sum, chunk offsets) and copy it to device memory owned by the new
 *   uw_matrix.  `resident` (uw_resident) says what stays on the device for a
 *   Huffman blob; any form with the palette codes runs the post's load-time
 *   transcode of the stream into 4-bit codes.  Blocks the host until the
 *   upload on `stream` is done, so the caller may free `blob` on return.
 *   uw_get_info reports the device bytes the matrix holds.
 *   Errors: UW_ERR_INVALID_ARG (resident out of range), UW_ERR_CORRUPT
 *   (validation), UW_ERR_NO_MEMORY, UW_ERR_CUDA.
 */
uw_status uw_load(const void *blob, size_t size, int resident, uw_stream stream, uw_matrix **out);

/*
 * uw_blob_validate - the host-side checks of uw_load without any device work
 *   (usable on a machine without a GPU).  info may be NULL.
 *   Errors: UW_ERR_CORRUPT with the first failed check in uw_last_error().
 */
uw_status uw_blob_validate(const void *blob, size_t size, uw_info *info);

/* uw_free - release a uw_matrix and its device memory.  As with cudaFree (which it calls, and which waits for
 * work still running on the device), no work that reads the matrix may be enqueued after it.  NULL is a no-op. */
void uw_free(uw_matrix *m);

/* uw_get_info - header facts and memory footprint of a loaded matrix. */
uw_status uw_get_info(const uw_matrix *m, uw_info *out);

/*
 * uw_decode - rebuild W[N,K] bf16 (bit-exact, the post's lossless claim) into
 *   caller-owned device memory w_dev (N*K*2 bytes, 16-byte aligned).
 *   Asynchronous on `stream`.  Errors: UW_ERR_INVALID_ARG, UW_ERR_CORRUPT (a
 *   device error latched by an earlier call), UW_ERR_CUDA.
 */
uw_status uw_decode(const uw_matrix *m, uint16_t *w_dev, uw_stream stream);

/*
 * uw_workspace_size - device workspace bytes uw_matmul needs for (m, B,
 *   strategy) (AUTO: the plan AUTO would pick; an explicit strategy: that
 *   strategy with the kernel and launch shape AUTO would pair with it at this B).
 *   0 is a valid answer.  The workspace holds a preprocess output, an fp32
 *   accumulator [B,N] and 24 bytes per 128 rows of W; its contents need no
 *   initialisation (the tensor-core kernel tags the cells it shares between
 *   its CTAs with a per-launch epoch, and clears them before it ends, so a
 *   CUDA graph that replays the call finds them clear).  A call owns its
 *   workspace until `stream` has passed it: calls that may overlap take
 *   separate workspaces.  If a call ends with UW_ERR_TIMEOUT in uw_check, a
 *   graph replay of it on the same workspace may find stale cells.
 */
uw_status uw_workspace_size(const uw_matrix *m, int64_t B, uw_strategy strategy, size_t *bytes);

/*
 * uw_matmul - Y[B,N] = X[B,K] . W^T with W decoded on-chip (the post's
 *   reconstructive matmul; fp32 accumulation).  x_dev: [B,K] bf16 device;
 *   y_dev: [B,N] fp32 or bf16 (RNE) device; workspace: device scratch of at
 *   least uw_workspace_size bytes (may be NULL if that size is 0).  B == 0 is a
 *   no-op.  Asynchronous on `stream`.
 *   Errors: UW_ERR_INVALID_ARG, UW_ERR_SHAPE, UW_ERR_UNSUPPORTED (e.g.
 *   DIRECT_PALETTE without resident codes), UW_ERR_WORKSPACE, UW_ERR_CORRUPT,
 *   UW_ERR_CUDA.
 */
/*   AUTO runs the autotuned plan for B's bucket, else the default plan; an explicit
 *   strategy runs with the default kernel and launch shape for that strategy and B. */
uw_status uw_matmul(const uw_matrix *m, const uint16_t *x_dev, int64_t B, void *y_dev, uw_out_dtype out_dtype,
                    uw_strategy strategy, void *workspace, size_t ws_bytes, uw_stream stream);

/* uw_matmul_plan - as uw_matmul, with an explicit plan (strategy, kernel, split, variant). */
uw_status uw_matmul_plan(const uw_matrix *m, const uint16_t *x_dev, int64_t B, void *y_dev, uw_out_dtype out_dtype,
                         const uw_plan *plan, void *workspace, size_t ws_bytes, uw_stream stream);

/* uw_plan_workspace_size - workspace bytes for an explicit plan. */
uw_status uw_plan_workspace_size(const uw_matrix *m, int64_t B, const uw_plan *plan, size_t *bytes);

/* uw_plan_for - the plan AUTO runs for (m, B): the autotuned entry for B's
 *   bucket if one exists, else a default rule. */
uw_status uw_plan_for(const uw_matrix *m, int64_t B, uw_plan *out);

/*
 * uw_matmul_host - end-to-end form of uw_matmul with HOST X and Y: copies
 *   x_host ([B,K] bf16) to the device, runs the plan AUTO picks, copies Y back
 *   into y_host and synchronises `stream` before returning.  workspace must be
 *   a device buffer of at least uw_host_workspace_size bytes (it also holds
 *   the device copies of X and Y).  Pinned host memory gives the fastest copies.
 */
uw_status uw_matmul_host(const uw_matrix *m, const uint16_t *x_host, int64_t B, void *y_host,
                         uw_out_dtype out_dtype, void *workspace, size_t ws_bytes, uw_stream stream);
uw_status uw_host_workspace_size(const uw_matrix *m, int64_t B, uw_out_dtype out_dtype, size_t *bytes);

/*
 * uw_matmul_host_async - uw_matmul_host without the final synchronisation: the
 *   copy of X, the matmul and the copy of Y back are enqueued on `stream` and
 *   the call returns.  x_host must stay unchanged, and y_host unread, until
 *   the stream has passed the copy back (synchronise the stream or an event
 *   recorded after the call); the workspace belongs to the call until then.
 *   With pinned host buffers and two streams, one call's copies overlap the
 *   other's matmul.  Errors as uw_matmul_host.
 */
uw_status uw_matmul_host_async(const uw_matrix *m, const uint16_t *x_host, int64_t B, void *y_host,
                               uw_out_dtype out_dtype, void *workspace, size_t ws_bytes, uw_stream stream);

/*
 * uw_matmul_noalloc - uw_matmul with the palette-transcode pipeline
 *   (UW_STRAT_PALETTE_TRANSCODE on the GEMV kernel) that allocates nothing and
 *   takes no workspace.  The Unweight post has no counterpart to this entry
 *   point; it exists for callers that cannot call cudaMalloc - an engine whose
 *   allocator reserved all device memory at start-up, or a latency-critical
 *   path that must not take the device synchronisation cudaMalloc / cudaFree may
 *   imply.  Its scratch (the transcoded 4-bit codes, plus the fp32 accumulator a
 *   K-split may need) is a library-owned static device array of 36 MiB, held on
 *   every GPU that loads the library until the process exits.
 *   m must be a Huffman-coded matrix; x_dev, y_dev, B and out_dtype are as in
 *   uw_matmul.  The array's device address is looked up (cudaGetSymbolAddress)
 *   by the first call in each CUDA context - the device's primary context, or
 *   one a driver-API caller made current - and cached under that context's
 *   unique id, so a call after cudaDeviceReset looks it up again.  Make the
 *   first call in a context before any stream capture.  All calls share the
 *   one array and it keeps the last call's contents (the accumulator is
 *   cleared on the stream before each use): calls whose GPU work overlaps
 *   (different streams, or different threads without ordering) race on it.
 *   Errors: UW_ERR_WORKSPACE when N*K/2 plus B*N*4 plus 24 bytes per 128 rows
 *   (each rounded up to 256 bytes, with 64 bytes of padding on the codes)
 *   exceeds the 36 MiB array;
 *   UW_ERR_UNSUPPORTED for a palette-codec matrix; otherwise as uw_matmul.
 */
uw_status uw_matmul_noalloc(const uw_matrix *m, const uint16_t *x_dev, int64_t B, void *y_dev, uw_out_dtype out_dtype,
                            uw_stream stream);

/*
 * uw_autotune - for each batch size in batches[0..n_batches), time the
 *   candidate plans on this GPU (CUDA events on `stream`, several repetitions,
 *   median) by coordinate descent over strategy, kernel, split and variant (the
 *   post's autotuner: measure real throughput, vary one choice at a time until
 *   nothing improves), and store the fastest in the matrix's tune table, keyed
 *   by batch bucket.  workspace must hold uw_workspace_size for every candidate
 *   (uw_autotune_workspace_size).  Synchronous.  Writes scratch outputs only
 *   into the workspace.  It also allocates, for the duration of the call, a
 *   device buffer of twice the L2 size that it rewrites before each timed
 *   launch, so candidates are timed with their weights coming from HBM (if
 *   that allocation fails, timing proceeds without it).
 */
uw_status uw_autotune(uw_matrix *m, const int64_t *batches, int n_batches, void *workspace, size_t ws_bytes,
                      uw_stream stream);
uw_status uw_autotune_workspace_size(const uw_matrix *m, const int64_t *batches, int n_batches, size_t *bytes);

/*
 * uw_tune_save / uw_tune_load - the tune table as text, one line per batch
 *   bucket: "B strategy kernel split_k variant us".  save: buf == NULL returns
 *   the length in *len.  load replaces the table; it rejects malformed lines
 *   with UW_ERR_INVALID_ARG and leaves the table unchanged.
 */
uw_status uw_tune_save(const uw_matrix *m, char *buf, size_t cap, size_t *len);
uw_status uw_tune_load(uw_matrix *m, const char *text);

/* One matmul of a sequence: Y[B,N] = X[B,K] . W^T for the loaded matrix m; x and y are device pointers as in
 * uw_matmul, out_dtype a uw_out_dtype; flags 0 or UW_STEP_CONCURRENT. */
typedef struct {
    const uw_matrix *m;
    const uint16_t *x;
    void *y;
    int32_t out_dtype;
    int32_t flags;
} uw_step;

/* The step may run at the same time as the steps before it back to the last step without the flag: it reads
 * nothing those steps write and writes nothing they read or write (an MLP's up projection beside its gate
 * projection: both read the layer's input).  Such a run forms a group.  The flag permits overlap; a schedule
 * with UW_SEQ_GROUPS runs each group's matmuls on streams of their own (the first four members on four streams,
 * any further member after the member four places before it), any other schedule runs them in order. */
#define UW_STEP_CONCURRENT 1

/*
 * uw_sequence_run - run n matmuls in order at batch B (the post's section on scheduling hard and easy layers).
 *   A step is "hard" when its matrix holds only its Huffman stream (UW_RESIDENT_HUFFMAN): its 4-bit palette codes
 *   are transcoded on `side_stream` into one of two slots of the workspace (double buffering), as soon as the
 *   slot's previous matmul is done, so the transcode of the next hard step runs while the main stream works on
 *   the steps before it.  Its matmul on `stream` waits for that transcode and reads the codes (the direct-palette
 *   kernels).  Steps whose matrix holds its palette form run their AUTO plan.  Asynchronous: everything is enqueued
 *   at once and ordered by events; `stream` ends joined with `side_stream`, so the call can be captured into one
 *   CUDA graph from `stream`.  `side_stream` must differ from `stream` when a step is hard.  The workspace
 *   (uw_sequence_workspace_size bytes, 256-byte aligned) belongs to the sequence until `stream` has passed it.
 *   The first call in a thread on a device creates the events the calls use; make it before any stream capture.
 *   The steps' x and y must not overlap a later step's inputs unless the caller wants that chaining: steps run in
 *   order on `stream`, except that under a UW_SEQ_GROUPS schedule a group of steps joined by UW_STEP_CONCURRENT
 *   runs on `stream` and on streams the library keeps per thread and device (forked from and joined back to
 *   `stream` with events, so a graph captured from `stream` holds them).  Each member of a group has its own part
 *   of the workspace (the size covers both forms).  With the transcode schedule a hard step always waits for the
 *   steps before it (the flag is not applied to it).
 *   Errors: UW_ERR_INVALID_ARG, UW_ERR_WORKSPACE, UW_ERR_CUDA, or a step's uw_matmul error.
 */
/*   decode_sms: the post's decode-vs-matmul SM split.  0: every launch sizes its grid for all SMs.  d > 0: the
 *   main stream's persistent matmul grids are sized for the device's SMs minus d, and each transcode is a
 *   persistent grid of d SMs' worth of CTAs, so the two run side by side.  UW_SEQ_DIRECT (-1): no side-stream
 *   transcode; every step runs its own AUTO plan on `stream` (a hard step at B <= 8: the Huffman-direct GEMV;
 *   `side_stream` is not used).  Any of these plus UW_SEQ_GROUPS: the same schedule with the groups of
 *   UW_STEP_CONCURRENT steps overlapped.  Must lie in [-1, SMs) or in UW_SEQ_GROUPS + [-1, SMs).
 */
#define UW_SEQ_DIRECT (-1)
#define UW_SEQ_GROUPS 65536
uw_status uw_sequence_workspace_size(const uw_step *steps, int n, int64_t B, size_t *bytes);
uw_status uw_sequence_run(const uw_step *steps, int n, int64_t B, void *workspace, size_t ws_bytes, uw_stream stream,
                          uw_stream side_stream, int decode_sms);

/*
 * uw_sequence_tune - time uw_sequence_run over these steps (same arguments) for the direct schedule and a range of
 *   decode SM splits (UW_SEQ_DIRECT, 0, 8, 16, ..., 96; CUDA events on `stream`, median of three runs after two),
 *   each also with UW_SEQ_GROUPS when a step carries UW_STEP_CONCURRENT, and return the fastest in *decode_sms
 *   (the post's tuning of the decoder's share of the SMs).  Synchronous; runs the sequence 5 times per
 *   candidate, writing the steps' outputs.
 */
uw_status uw_sequence_tune(const uw_step *steps, int n, int64_t B, void *workspace, size_t ws_bytes, uw_stream stream,
                           uw_stream side_stream, int *decode_sms);

/* ------------------------------------------------------------------------------------------------------------
 * Operators around the compressed products of a mixture-of-experts decoder: the router, the experts' grouped
 * products on compressed weights, the norms and residual around a block, and the log probabilities on the head's
 * logits.  A token's way: uw_block_norm; uw_matmul for the router's logits; uw_route; uw_group_matmul for gate and
 * up, and for down; uw_block_norm, which joins the token's expert rows; uw_matmul for the head; uw_token_logprobs.
 * Sizes that only the device knows (rows per expert) are read there: no call waits for the GPU, so every call can be
 * captured into a CUDA graph.  uw_out_dtype names the type of inputs here too.
 * ------------------------------------------------------------------------------------------------------------ */

/*
 * uw_group - the weight matrices of `experts` experts, all [N, K], compressed without loss in the form the grouped
 *   kernels read: per weight a sign+mantissa byte and 4 bits of exponent (its distance from the lowest of 16
 *   consecutive exponents, chosen per matrix to cover the most weights), per 64 weights of a row that hold an
 *   exponent outside those 16 the 64 exponent bytes.  With up matrices the group is gated: an expert's product is
 *   silu(W x) * (W_up x), both products in one pass.
 */
typedef struct uw_group uw_group;

typedef struct {
    int64_t N, K;            /* per matrix: N outputs, K inputs */
    int32_t experts;
    int32_t gated;           /* made with up matrices */
    uint64_t n_verbatim;     /* 64-weight runs stored with their exponent bytes */
    uint64_t device_bytes;   /* device memory held by the group */
} uw_group_info;

/*
 * uw_group_create - a group from loaded matrices (any codec or resident form): w[0..experts), and w_up[0..experts)
 *   for a gated group (NULL: not gated).  The group holds its own copy; the matrices may be freed afterwards.
 *   Decodes one matrix at a time into a temporary N*K*2-byte device buffer.  Synchronous.
 * uw_group_create_dense - the same from bf16 weights on the device: w_dev [experts, N, K] row-major, 16-byte
 *   aligned, and w_up_dev (NULL: not gated).
 *   Errors: UW_ERR_INVALID_ARG (NULL, alignment, experts outside 1..1024, a matrix of another device),
 *   UW_ERR_SHAPE (K % 64, N or K < 1 or above 2^31 - 256, matrices of different shapes, 2^32 or more verbatim
 *   runs), UW_ERR_CORRUPT, UW_ERR_NO_MEMORY, UW_ERR_CUDA.
 */
uw_status uw_group_create(const uw_matrix *const *w, const uw_matrix *const *w_up, int experts, uw_stream stream,
                          uw_group **out);
uw_status uw_group_create_dense(const uint16_t *w_dev, const uint16_t *w_up_dev, int experts, int64_t N, int64_t K,
                                uw_stream stream, uw_group **out);

/* uw_group_free - release a group and its device memory (as uw_free).  NULL is a no-op. */
void uw_group_free(uw_group *g);
uw_status uw_group_get_info(const uw_group *g, uw_group_info *out);

/* uw_group_decode - rebuild one expert's matrix bit-exactly into w_dev [N, K] bf16 (16-byte aligned); up != 0: its
 *   up matrix.  Asynchronous.  Errors: UW_ERR_INVALID_ARG, UW_ERR_UNSUPPORTED (up of a group that is not gated),
 *   UW_ERR_CUDA. */
uw_status uw_group_decode(const uw_group *g, int expert, int up, uint16_t *w_dev, uw_stream stream);

/*
 * uw_group_matmul - for every expert e and every row r in [offsets[e], offsets[e + 1]):
 *     y[r, :] = W_e x[s]           or, gated,   y[r, :] = silu(W_e x[s]) * (W_up_e x[s])
 *   with s = row_src[r], or s = r when row_src is NULL (fp32 accumulation, one rounding to the output type).
 *   x_dev: [x_rows, K] bf16, rows ldx elements apart (ldx 0: K; a multiple of 8).  y_dev: [rows, N] fp32 or bf16,
 *   rows ldy elements apart (0: N).  offsets_dev: int32 [experts + 1], ascending, on the device; rows of y outside
 *   [offsets[0], offsets[experts]) are not written.  Offsets are clamped to [0, rows]; a row whose source lies
 *   outside [0, x_rows) counts as zeros, so an expert's rows may be padded with a source of -1.  An expert may have
 *   any number of rows, none included.  A row's result is the same bits in every run with the same `rows`, and does not
 *   depend on what the other experts' rows hold nor how they are shared out; another `rows` may choose another kernel,
 *   whose sums have another order.
 *   No workspace.  Asynchronous on `stream`.
 *   Errors: UW_ERR_INVALID_ARG (NULL, x or y not 16-byte aligned, bad dtype, another current device than the group's),
 *   UW_ERR_SHAPE (negative sizes, rows or x_rows above 2^31 - 1024, ldx < K or not a multiple of 8, ldy < N),
 *   UW_ERR_CUDA.
 */
uw_status uw_group_matmul(const uw_group *g, const uint16_t *x_dev, int64_t x_rows, int64_t ldx,
                          const int32_t *row_src_dev, const int32_t *offsets_dev, int64_t rows, void *y_dev,
                          int64_t ldy, uw_out_dtype out_dtype, uw_stream stream);

/* uw_group_check - as uw_check, for a group: UW_ERR_TIMEOUT if a bounded wait of a kernel on it expired. */
uw_status uw_group_check(const uw_group *g, uw_stream stream);

/* How uw_route turns a token's logits into weights. */
typedef enum {
    UW_SCORE_SOFTMAX = 0,    /* softmax over all experts */
    UW_SCORE_SIGMOID = 1,    /* 1 / (1 + e^-logit), each expert by itself */
    UW_SCORE_CHOOSES = 16    /* added to either: the experts are chosen by score + bias, in place of logit + bias */
} uw_score;

typedef struct {
    int32_t experts;         /* 1..1024 */
    int32_t topk;            /* 1..min(16, experts) */
    int32_t score;           /* uw_score, with or without UW_SCORE_CHOOSES */
    int32_t renormalize;     /* divide a token's chosen weights by their sum (a sum of 0 leaves zeros) */
    float scale;             /* multiplies the weights */
    const float *bias;       /* device fp32 [experts], for the choice alone; NULL: none.  It is added to the logits, or, with
                              * UW_SCORE_CHOOSES, to the scores, as routers with a load-balancing correction have it */
} uw_router;

/*
 * uw_route - choose each token's experts and the order of the grouped products' rows.
 *   logits_dev: [tokens, experts] of `dtype`, rows ld elements apart (0: experts).  Token t takes the topk experts
 *   with the largest logit + bias, or score + bias (in fp32; equal ones by the lower index; NaN counts above +inf):
 *     ids     int32 [tokens, topk]  the experts, largest first
 *     weights fp32  [tokens, topk]  score [/ the sum over the chosen] * scale
 *     offsets int32 [experts + 1]   rows of expert e are [offsets[e], offsets[e + 1])
 *     row_src int32 [tokens * topk] the token of each row; rows are ordered by (expert, token)
 *     pos     int32 [tokens, topk]  the row of each (token, choice)
 *   A row of logits that is all -inf has scores 0, and without a bias takes experts 0..topk-1.
 *   workspace: uw_route_workspace_size bytes of device scratch, 16-byte aligned (0 for a few tokens; needs no
 *   initialisation).  Asynchronous.  The result does not depend on the run.
 *   Errors: UW_ERR_INVALID_ARG, UW_ERR_SHAPE (tokens < 0, tokens * topk above 2^31 - 1024, ld < experts),
 *   UW_ERR_WORKSPACE, UW_ERR_CUDA.
 */
uw_status uw_route_workspace_size(const uw_router *r, int64_t tokens, size_t *bytes);
uw_status uw_route(const uw_router *r, const void *logits_dev, uw_out_dtype dtype, int64_t tokens, int64_t ld,
                   int32_t *ids, float *weights, int32_t *offsets, int32_t *row_src, int32_t *pos, void *workspace,
                   size_t ws_bytes, uw_stream stream);

/* What uw_block_norm does with each row; the pointers are device addresses, 16-byte aligned. */
typedef struct {
    int64_t dim;             /* elements of a row, 1..65536 */
    const uint16_t *post_weight; /* bf16 [dim]: the block's output is normed with it; NULL: it is not */
    const uint16_t *gate;    /* bf16 [ceil(rows / gate_every), dim]: multiplies the block's output; NULL: none */
    int64_t gate_every;      /* consecutive rows that share a row of the gate (rows or more: one row for all) */
    const uint16_t *pre_weight;  /* bf16 [dim]: weight of the norm that makes u (NULL: no u) */
    float res_scale, out_scale, eps;
    int32_t res_dtype;       /* uw_out_dtype of h and h_out */
    int32_t block_dtype;     /* uw_out_dtype of y */
} uw_norm;

/*
 * uw_block_norm - what stands between one block's output and the next block's input, for each row t:
 *     o = y[t], or sum over j < topk of weights[t, j] y[pos[t, j]]    (a pos outside [0, y_rows) adds nothing)
 *     o = post_weight * o / sqrt(mean(o^2) + eps)                     with a post_weight
 *     o = gate[t / gate_every] * o                                    with a gate
 *     h_out[t] = res_scale * h[t] + out_scale * o
 *     u[t] = pre_weight * h_out[t] / sqrt(mean(h_out[t]^2) + eps)     with a pre_weight; h_out before its rounding
 *   All in fp32, one rounding per output.  h, h_out: [rows, dim] of res_dtype; y of block_dtype: [rows, dim], or
 *   [y_rows, dim] with topk > 0; u: bf16 [rows, dim].  y NULL: no block output (o = 0), for a model's first norm.
 *   h NULL: no residual.  h_out NULL: not stored.  h_out may be h; u may be y where y is bf16 and topk 0.  Rows are dim elements
 *   apart; any dim is taken, multiples of 8 (16-byte rows) are fast.  Asynchronous.
 *   Errors: UW_ERR_INVALID_ARG (NULL or misaligned pointers, bad dtypes, u without pre_weight or the reverse,
 *   nothing to write, topk outside 0..16, gate_every < 1 with a gate), UW_ERR_SHAPE, UW_ERR_CUDA.
 */
uw_status uw_block_norm(const uw_norm *n, int64_t rows, const void *h, void *h_out, const void *y, int64_t y_rows,
                        const int32_t *pos, const float *weights, int topk, uint16_t *u, uw_stream stream);

/*
 * uw_token_logprobs - log probabilities of given tokens under softmax(logits / temperature), with the entropy of
 *   each row's distribution and its most probable tokens, in one call on logits as uw_matmul of a head leaves them.
 *   logits_dev: [rows, vocab] of `dtype`, rows ld elements apart (0: vocab).
 *     logprob [rows] fp32: of token targets[r]; 0 where targets[r] < 0 (no token given), NaN where it is >= vocab
 *     entropy [rows] fp32 in nats
 *     top_ids int32, top_logprobs fp32 [rows, n_top]: the n_top largest logits, largest first, equal ones by the
 *     lower index (NaN counts above +inf)
 *   targets/logprob, entropy and top_ids/top_logprobs are each optional (NULL).  Logits of -inf are tokens masked
 *   out: probability 0.  A row with nothing but -inf has log probabilities -inf and entropy 0; a row with a NaN or
 *   +inf has NaN.  0 <= n_top <= min(32, vocab).  No workspace.  Asynchronous; the result does not depend on the run.
 *   Errors: UW_ERR_INVALID_ARG (NULL, misaligned to the element, temperature not finite and > 0, bad n_top, logprob
 *   without targets or the reverse), UW_ERR_SHAPE (vocab outside 1..2^24, ld < vocab), UW_ERR_CUDA.
 */
uw_status uw_token_logprobs(const void *logits_dev, uw_out_dtype dtype, int64_t rows, int64_t vocab, int64_t ld,
                            float temperature, const int32_t *targets, float *logprob, float *entropy, int n_top,
                            int32_t *top_ids, float *top_logprobs, uw_stream stream);

/* ------------------------------------------------------------------------------------------------------------
 * Attention between the qkv product and the output product, over keys and values kept in pages; and the edits of
 * logits in front of uw_token_logprobs.  A token's way: uw_matmul for q, k and v; uw_kv_append, which rotates q and k
 * and stores k and v; uw_kv_attend; uw_matmul for the output; and behind the head's uw_matmul uw_edit_logits, then
 * uw_token_logprobs.  Lengths are read on the device: no call waits for the GPU.
 * ------------------------------------------------------------------------------------------------------------ */

/* Which elements of a head are turned together: i and i + dim / 2, or 2 i and 2 i + 1. */
typedef enum {
    UW_ROTARY_HALF = 0,
    UW_ROTARY_INTERLEAVED = 1
} uw_rotary_layout;

/* How the frequencies base^(-2 i / dim) are scaled for contexts longer than those of training.  In brackets the published method, and
 * what a model's configuration usually calls it. */
typedef enum {
    UW_ROTARY_PLAIN = 0,     /* not (rotary position embedding; "default") */
    UW_ROTARY_LINEAR = 1,    /* all divided by factor (position interpolation; "linear") */
    UW_ROTARY_STRETCHED = 2, /* base multiplied by factor^(dim / (dim - 2)): the lowest frequency divided by factor (NTK-aware scaling of
                              * the base, with a fixed factor; "dynamic" at one length, with that length's factor) */
    UW_ROTARY_BANDS = 3,     /* by the turns made over `original` positions: divided by factor up to `low`, kept from `high` on,
                              * between the two a mixture that is linear in the turns (frequency bands; "llama3", with its
                              * low_freq_factor and high_freq_factor, usually 1 and 4) */
    UW_ROTARY_RAMP = 4       /* the same ends, linear in the index i between the indices (rounded outwards) that make `high` and
                              * `low` turns; cos and sin are multiplied by 0.1 ln(factor) + 1 (factor > 1) (YaRN; "yarn", with its
                              * beta_slow as `low` and beta_fast as `high`, usually 1 and 32) */
} uw_rotary_scaling;

/*
 * uw_rotary_frequencies - host: freq[0..dim/2), in radians a position, and the factor on cos and sin (*scale; may be
 *   NULL).  factor, low, high, original: as the scaling uses them (others are ignored).
 *   Errors: UW_ERR_INVALID_ARG (NULL, base not finite and > 1, factor not finite and >= 1, low or high not finite, low < 0,
 *   high <= low, for a ramp low <= 0, original < 1, unknown scaling), UW_ERR_SHAPE (dim not a multiple of 16 in 16..128).
 */
uw_status uw_rotary_frequencies(int dim, double base, uw_rotary_scaling scaling, double factor, double low, double high,
                                int64_t original, double *freq, float *scale);

typedef struct {
    int32_t dim;             /* elements of a head that are turned, the first ones: a multiple of 16, 16..head_dim */
    int32_t layout;          /* uw_rotary_layout */
    const double *freq;      /* device [dim / 2], radians a position */
    float scale;             /* multiplies cos and sin */
} uw_rotary;

/*
 * uw_kv_cache - keys and values of many sequences in pages of page_size slots, a page being an index into k and v.  The
 *   element i of a head's key in a page's slot is at k[page * page_stride + slot * slot_stride + head * head_stride + i], its
 *   value at the same place in v: [pages, page_size, kv_heads, head_dim] and [pages, kv_heads, page_size, head_dim] are
 *   both taken, k and v may be halves of one tensor.  The caller owns the memory and which sequence holds which page.
 */
typedef struct uw_kv_cache uw_kv_cache;

typedef struct {
    uint16_t *k, *v;         /* device, bf16, 16-byte aligned */
    int64_t pages;           /* 1..2^31 - 1 */
    int64_t page_stride, slot_stride, head_stride; /* elements, multiples of 8, at least head_dim, below 2^39 (one of a dimension
                              * of size 1 is ignored) */
    int32_t page_size;       /* slots: a multiple of 8, 8..65536 */
    int32_t kv_heads;        /* 1..1024 */
    int32_t head_dim;        /* 64 or 128 */
} uw_kv_desc;

/*
 * uw_kv_create - a handle on such memory for the current device: two words of device memory and the copies'
 *   descriptions.  Errors: UW_ERR_INVALID_ARG (NULL, alignment, strides), UW_ERR_SHAPE, UW_ERR_UNSUPPORTED (head_dim, or a
 *   driver without tensor maps), UW_ERR_NO_MEMORY, UW_ERR_CUDA.
 */
uw_status uw_kv_create(const uw_kv_desc *d, uw_kv_cache **out);
void uw_kv_free(uw_kv_cache *c);

/* The new tokens of a step: sequence s brings the rows [starts[s], starts[s + 1]) of the call's tensors and holds lengths[s]
 * tokens with them, so its i-th new token is at position lengths[s] - (starts[s + 1] - starts[s]) + i.  Device pointers;
 * starts ascending, clamped to [0, rows]; a sequence may bring none.  pages[s * ld_pages + p] is the page of its positions
 * [p page_size, (p + 1) page_size), for p below max_pages; entries behind its length are not read. */
typedef struct {
    int32_t sequences;       /* 1..65536 */
    const int32_t *starts;   /* [sequences + 1] */
    const int32_t *lengths;  /* [sequences] */
    const int32_t *pages;
    int64_t ld_pages;        /* 0: max_pages */
    int64_t max_pages;       /* 1..2^30 / page_size */
} uw_kv_batch;

/*
 * uw_kv_append - rotate the new tokens' queries and keys, store their keys and values in the cache.
 *   q: [rows, q_heads, head_dim], k and v: [rows, kv_heads, head_dim] of `dtype` (as uw_matmul leaves them: fp32 or bf16), rows
 *   ldq, ldk, ldv elements apart (0: dense; multiples of 8), so that all three may be columns of one product's output.
 *   q_out: bf16 [rows, q_heads, head_dim], rows ldq_out apart; it may be q itself (bf16, with the same stride) and else shares
 *   nothing with q, k or v, though rows may lie between theirs.  Either q and q_out or k and v may be NULL.
 *   r NULL: nothing is turned.  positions: int32 [rows], what the angles go by; NULL: the position in the cache.
 *   The angle position * freq is reduced in 64 bits; products in fp32, one rounding to bf16.  A token whose position in the
 *   cache is negative or past the table, or whose page is outside [0, pages), is not stored.  Rows outside
 *   [starts[0], starts[sequences]) are left as they were.  Two rows with one slot (a page that two
 *   sequences write to): each eight elements there are one of the two's, not all of the same one.  Asynchronous.
 *   Errors: UW_ERR_INVALID_ARG (NULL, alignment: 16 bytes for q, k, v, q_out and 4 for the rest, 8 for freq; another current
 *   device than the cache's; bad dtype or layout; q_out overlapping q, k or v), UW_ERR_SHAPE, UW_ERR_CUDA.
 */
uw_status uw_kv_append(const uw_kv_cache *c, const uw_kv_batch *b, const uw_rotary *r, int64_t rows, uw_out_dtype dtype,
                       const void *q, int64_t ldq, int q_heads, const void *k, int64_t ldk, const void *v, int64_t ldv,
                       const int32_t *positions, uint16_t *q_out, int64_t ldq_out, uw_stream stream);

/*
 * uw_kv_attend - for every new token t and query head h, with the keys k_j and values v_j of h's key head
 *   h / (q_heads / kv_heads) in t's sequence:
 *     out[t, h] = sum_j p_j v_j,  p = softmax over j of (scale * q[t, h] . k_j),  lse[t, h] = ln sum_j exp(scale * q[t, h] . k_j)
 *   over the positions j of its sequence's length that it may see: causal != 0: j <= position, and with window > 0
 *   position - j < window; else all.  A row that sees nothing gets zeros and an lse of -inf.
 *   q, out: bf16 [rows, q_heads, head_dim], rows ldq and ldo elements apart (0: dense; multiples of 8), which share nothing, though
 *   rows may lie between one another.  lse: fp32 [rows, q_heads] or NULL.  Sums in fp32; probabilities are rounded to bf16 in front of the second product, as its operand.
 *   A page outside [0, pages) reads as zeros.  Slots behind a sequence's length may hold anything; a key or value of the
 *   sequence itself that is not finite spoils the rows that see it, and may spoil others of its sequence that do not.
 *   Rows outside [starts[0], starts[sequences]) are left as they were.  The same call gives the same bits in every run; how a
 *   sequence's keys are cut, and so the last bits, depends on the whole batch's lengths.
 *   workspace: uw_kv_attend_workspace_size bytes, 16-byte aligned; needs no initialisation.  Calls that may run at the
 *   same time need one each.  Asynchronous.
 *   Errors: UW_ERR_INVALID_ARG (NULL, alignment, scale not finite, window < 0, a window without causal, out
 *   overlapping q, another current device than the cache's), UW_ERR_SHAPE (rows, q_heads not a multiple of kv_heads or above 64 kv_heads, strides),
 *   UW_ERR_WORKSPACE, UW_ERR_CUDA.
 */
/* For a call of these sequences, rows and query heads; it does not shrink as rows grow. */
uw_status uw_kv_attend_workspace_size(const uw_kv_cache *c, int sequences, int64_t rows, int q_heads, size_t *bytes);
uw_status uw_kv_attend(const uw_kv_cache *c, const uw_kv_batch *b, int64_t rows, const uint16_t *q, int64_t ldq, int q_heads,
                       float scale, int causal, int64_t window, uint16_t *out, int64_t ldo, float *lse, void *workspace,
                       size_t ws_bytes, uw_stream stream);

/* uw_kv_check - as uw_check, for a cache: UW_ERR_TIMEOUT if a bounded wait of a kernel on it expired. */
uw_status uw_kv_check(const uw_kv_cache *c, uw_stream stream);

/*
 * What uw_edit_logits does to each row; every pointer is a device address or NULL (that edit is left out).  tokens holds a
 * row's prompt and, behind it, what was generated: row r's tokens are tokens[r * ld_tokens + i], i < lengths[r], the first
 * prompt_lengths[r] (NULL: 0) of them the prompt's.  Lengths are clamped to [0, max_tokens], ids outside the vocabulary are
 * passed over.
 */
typedef struct {
    const int32_t *tokens;
    int64_t ld_tokens, max_tokens; /* ld_tokens 0: max_tokens */
    const int32_t *lengths;        /* [rows]; needed with tokens */
    const int32_t *prompt_lengths; /* [rows] */
    const float *repetition;       /* [rows], > 0: logits of tokens in the prompt or generated, divided by it above 0, else multiplied */
    const float *frequency;        /* [rows]: times the number of times the token was generated, subtracted */
    const float *presence;         /* [rows]: subtracted once if it was generated */
    const int32_t *bias_ids;       /* [rows, max_bias], with bias: added to these tokens' logits, a token's several entries in order */
    const float *bias;
    const int32_t *bias_lengths;   /* [rows], clamped to [0, max_bias]; NULL: max_bias */
    int64_t max_bias;              /* 0..4096; rows of bias and bias_ids are max_bias apart */
    const uint32_t *allowed;       /* [mask_count, ld_allowed] words: a token v whose bit v % 32 of word v / 32 is 0 becomes -inf */
    int64_t ld_allowed, mask_count; /* ld_allowed 0: ceil(vocab / 32) */
    const int32_t *mask_rows;      /* [rows]: which row of allowed; outside [0, mask_count): none.  NULL: row r's own (r < mask_count) */
} uw_logit_edits;

/*
 * uw_edit_logits - penalties for repeated tokens, biases and grammar masks, in this order, on each row of logits:
 *     x = repetition; x -= frequency * count; x -= presence; x += bias; -inf where not allowed
 *   in fp32 (the quotient by `repetition` is a product with its reciprocal, within 2^-23; both penalties are taken off as one
 *   sum), then rounded to out_dtype.
 *   logits: [rows, vocab] of `dtype`, rows ld elements apart (0: vocab); out: of out_dtype, rows ld_out apart.  out may be
 *   logits itself with the same type and ld; then only logits that change are written, and without a mask only those are
 *   read.  NaN stays NaN unless it is masked.  Elements behind vocab are left as they were.  No workspace.  Asynchronous; the
 *   result does not depend on the run.
 *   Errors: UW_ERR_INVALID_ARG (NULL, misaligned to the element, tokens without lengths, bias_ids without bias or the reverse,
 *   penalties without tokens, out overlapping logits in part), UW_ERR_SHAPE (vocab outside 1..2^24, ld, ld_out < vocab,
 *   max_tokens outside 0..2^24 - 1, max_bias), UW_ERR_CUDA.
 */
uw_status uw_edit_logits(const uw_logit_edits *e, const void *logits, uw_out_dtype dtype, int64_t rows, int64_t vocab,
                         int64_t ld, void *out, uw_out_dtype out_dtype, int64_t ld_out, uw_stream stream);

/* uw_check - synchronise `stream` and report (then clear) the matrix's device status word. */
uw_status uw_check(const uw_matrix *m, uw_stream stream);

/* Human-readable name of a status code (static storage). */
const char *uw_status_string(uw_status s);

/* Last error message of the calling thread ("" if none). */
const char *uw_last_error(void);

/* Library build string (version, target architecture). */
const char *uw_version(void);

#ifdef __cplusplus
}
#endif

#endif /* UW_H */
