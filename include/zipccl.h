/*
 * zipccl.h -- C ABI of the GB300 (sm_103a) ZipCCL BF16 exponent-coding path.
 *
 * The operations follow "ZipCCL: Efficient Lossless Data Compression of
 * Communication Collectives for Accelerating LLM Training":
 *   - abstract, technique (1) and the shd-paper summary's key design: BF16
 *     communication tensors are near-Gaussian, so the 8-bit exponent is
 *     entropy-coded with a code derived from the Gaussian density, with no
 *     online statistics;  Fig. 6 caption: sign and mantissa stay raw and a
 *     value shrinks to about 11 bits;
 *   - abstract, technique (2): GPU compressor/decompressor kernels with a
 *     communication-aware data layout -- here one self-contained compressed
 *     chunk per destination rank, back to back in one buffer;
 *   - Fig. 3 and Fig. 5 captions: the receive side of zipcclReduceScatter
 *     decompresses the peers' chunks and reduces them.
 * The stream format (v1) is defined by this library; the pages fix none.
 *
 * Conventions for every call:
 *   - Pointers named d_* are device memory on the current CUDA device, owned
 *     by the caller.  The library allocates and frees nothing on the device.
 *   - d_* base pointers must be 16-byte aligned.
 *   - `stream` is a cudaStream_t passed as void*.  Calls are asynchronous and
 *     stream-ordered; they never synchronize unless the name says so.
 *   - Argument errors are returned synchronously, before any launch.
 *   - Data-dependent errors (a corrupt stream, a look-back that timed out)
 *     are recorded by the kernels in a status word at the start of the
 *     workspace; zipccl_get_device_status reads it and reports the last
 *     call made on that workspace, so read it after the call you want to
 *     check.  A compress call clears it first; a decompress or
 *     decompress_reduce call does not clear anything but tags its errors
 *     with a 56-bit number of its own, so that an earlier call's code (or
 *     whatever the memory held) never reads as its status.  No
 *     initialisation of a workspace is needed.  On such an error outputs
 *     are undefined but every access stays inside the caller's buffers.
 *   - A workspace must not be shared by calls that may run concurrently.
 */
#ifndef ZIPCCL_H
#define ZIPCCL_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ZIPCCL_OK = 0,
    ZIPCCL_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size, sum mismatch */
    ZIPCCL_ERR_CAPACITY = 2,    /* output or workspace smaller than required */
    ZIPCCL_ERR_CORRUPT = 3,     /* stream fails validation (device status) */
    ZIPCCL_ERR_VERSION = 4,     /* stream written by another format version */
    ZIPCCL_ERR_TIMEOUT = 5,     /* a bounded device wait gave up (device status) */
    ZIPCCL_ERR_CUDA = 6         /* a CUDA runtime call failed */
} zipccl_status;

/* Format version written and read by this library (1). */
int zipccl_format_version(void);

/* Static, human-readable name of a status code. */
const char *zipccl_status_string(int status);

/*
 * Passage: abstract, technique (3) (collectives fall back to uncompressed
 * operation) -- read as a per-tile raw fallback, so the expansion is bounded.
 * Exact worst-case compressed size of a chunk layout: every tile stored with
 * raw exponents (bounded expansion).  chunk_elems: host array of n_chunks
 * element counts.  *out_bytes receives the bound.  Host only.
 */
zipccl_status zipccl_max_compressed_bytes(const uint64_t *chunk_elems, uint32_t n_chunks,
                                          uint64_t *out_bytes);

/*
 * Workspace sizes, one call per operation (each sizes only what its kernels
 * use): compress needs per-chunk code tables and per-tile records, the
 * decoders per-chunk decode tables.  Host only.
 */
/* Workspace bytes needed by zipccl_compress for this chunk layout. */
zipccl_status zipccl_compress_workspace_bytes(const uint64_t *chunk_elems, uint32_t n_chunks,
                                              uint64_t *out_bytes);

/* Workspace bytes needed by zipccl_decompress for n elements in n_chunks chunks. */
zipccl_status zipccl_decompress_workspace_bytes(uint64_t n, uint32_t n_chunks, uint64_t *out_bytes);

/* Workspace bytes needed by zipccl_decompress_reduce for k peers. */
zipccl_status zipccl_reduce_workspace_bytes(uint32_t k, uint64_t *out_bytes);

/*
 * Passages: abstract, technique (1) (exponent coding from the Gaussian law,
 * no expensive online statistics) and technique (2) (GPU compressor with a
 * communication-aware data layout); shd-paper key-design paragraph
 * (frequent exponents get short codes); Fig. 6 caption (about 11 bits per
 * value: sign and mantissa raw).
 * Compress n BF16 words (d_in, bit patterns as uint16) split into n_chunks
 * per-destination chunks: chunk c is the next chunk_elems[c] words (host
 * array, sum == n, n_chunks >= 1, each chunk < 2^31 words; empty chunks are
 * allowed and produce a header-only chunk).
 * sigma_hint: host array of n_chunks floats or NULL.  A value > 0 fixes the
 * Gaussian scale of that chunk's code; otherwise the scale is taken from a
 * fixed sample of the chunk's exponents (no histogram pass).
 * d_out receives the chunks back to back, each a self-contained stream that
 * can be sent alone; out_capacity must be >= zipccl_max_compressed_bytes.
 * d_chunk_offsets (device, n_chunks + 1 uint64) receives each chunk's byte
 * offset in d_out and, last, the total size.  d_ws: workspace of at least
 * zipccl_compress_workspace_bytes bytes.
 * The tiles are coded by one persistent kernel whose CTAs (one per SM) must
 * all be resident at once, so it is issued as a cooperative launch; where the
 * device or context cannot make that launch the call returns ZIPCCL_ERR_CUDA.
 * The first call on a device sets the kernel's shared-memory limit and reads
 * its occupancy; later calls reuse them.
 */
zipccl_status zipccl_compress(const uint16_t *d_in, uint64_t n, const uint64_t *chunk_elems,
                              uint32_t n_chunks, const float *sigma_hint, void *d_out,
                              uint64_t out_capacity, uint64_t *d_chunk_offsets, void *d_ws,
                              uint64_t ws_bytes, void *stream);

/*
 * Passages: abstract (the compressor and decompressor kernels overlap
 * compression with memory access through a pipeline); Fig. 5 caption
 * (minimize kernel launch overhead, overlap compression with memory access);
 * abstract, technique (2) (communication-aware layout: one chunk per
 * destination rank).
 * zipccl_compress that also writes every chunk into d_send, the buffer a
 * transport would send from, and posts each chunk as soon as it is complete
 * while later chunks are still being coded.  In the same kernel: each tile's
 * image leaves shared memory by two TMA stores, one to d_out and one to the
 * same offset in d_send (the send costs HBM writes, no reads); the store
 * warps count the stored tiles of each chunk (release at GPU scope); one
 * warp in the first CTA, the stand-in for the proxy that hands chunks to
 * the network, waits for each chunk's count in chunk order (acquire, bounded
 * by 2 s) and posts it: it writes %globaltimer into d_chunk_ready[c].
 * d_chunk_ready[n_chunks] receives the kernel's start on the same clock.
 * The exchange itself is outside this library.
 *   d_send: device, 16-byte aligned, not d_out, send_capacity >=
 *     zipccl_max_compressed_bytes; afterwards d_send[0, offsets[n_chunks])
 *     equals d_out over the same range.
 *   d_chunk_ready: device, n_chunks + 1 uint64, 8-byte aligned, or NULL.
 * A wait that gives up records ZIPCCL_ERR_TIMEOUT; an error of the coding
 * warps ends the posting; read either with zipccl_get_device_status.  Other
 * arguments as zipccl_compress.
 */
zipccl_status zipccl_compress_send(const uint16_t *d_in, uint64_t n, const uint64_t *chunk_elems,
                                   uint32_t n_chunks, const float *sigma_hint, void *d_out,
                                   uint64_t out_capacity, uint64_t *d_chunk_offsets, void *d_send,
                                   uint64_t send_capacity, uint64_t *d_chunk_ready, void *d_ws,
                                   uint64_t ws_bytes, void *stream);

/*
 * Passages: Fig. 6 caption (the decompressor restores each value from its
 * raw sign/mantissa byte and its decoded exponent); pith summary (lossless:
 * every byte restored).
 * Decompress n_chunks chunks from d_stream into n BF16 words at d_out,
 * bit-identical to the compressed input.  d_chunk_offsets (device,
 * n_chunks + 1) are the offsets compress wrote; the stream must hold
 * d_chunk_offsets[n_chunks] bytes.  The chunks' element counts are read from
 * their headers and must sum to n (else ZIPCCL_ERR_CORRUPT in the device
 * status).  d_ws: at least zipccl_decompress_workspace_bytes bytes.
 */
zipccl_status zipccl_decompress(const void *d_stream, const uint64_t *d_chunk_offsets,
                                uint32_t n_chunks, uint16_t *d_out, uint64_t n, void *d_ws,
                                uint64_t ws_bytes, void *stream);

/*
 * Passages: Fig. 3 and Fig. 5 captions (zipcclReduceScatter: the receiver
 * decompresses the peers' chunks and reduces them).
 * Receive side of a reduce-scatter: d_peer_chunks is a host array of k
 * (1 <= k <= 16) device pointers, in rank order, each to one compressed
 * chunk of n elements and peer_chunk_bytes[p] bytes (host array; every read
 * of peer p stays inside those bytes, so a truncated or corrupt chunk gives
 * ZIPCCL_ERR_CORRUPT instead of a read past it).
 * d_out[i] = bf16_rne(((x0[i] + x1[i]) + x2[i]) ... + x_{k-1}[i]) with every
 * addition in fp32 (round to nearest even, subnormals kept); a NaN result is
 * written as 0x7FC0.  d_ws: at least zipccl_reduce_workspace_bytes bytes.
 */
zipccl_status zipccl_decompress_reduce(const void *const *d_peer_chunks,
                                       const uint64_t *peer_chunk_bytes, uint32_t k, uint64_t n,
                                       uint16_t *d_out, void *d_ws, uint64_t ws_bytes,
                                       void *stream);

/*
 * Passages: none; this call has no counterpart in the paper.
 * zipccl_decompress_reduce for callers that may not allocate device memory
 * at the point of the call: code that runs inside a device allocator's own
 * hook or callback (allocating there would re-enter the allocator), and
 * processes whose device memory is all reserved up front by a caching
 * allocator, where a new allocation would fail or force the cache to be
 * emptied.  Same kernels, same results; the workspace is a scratch area
 * compiled into this library (one per device) instead of a caller buffer, and
 * no call allocates or frees anything.  The paper has no counterpart to this
 * call: it serves only such callers.
 *   - The scratch holds ZIPCCL_NOALLOC_SCRATCH_BYTES bytes per device, the
 *     workspace of k = ZIPCCL_NOALLOC_MAX_PEERS (16) peers.  k == 0 or
 *     k > 16 returns ZIPCCL_ERR_INVALID_ARG before anything is launched.
 *   - The first call on a device, made with that device current, does a
 *     one-time set-up: it looks up the scratch's device address, which may
 *     load this library's kernels onto the device.  Make that first call
 *     before any stream capture begins.  A failed lookup returns
 *     ZIPCCL_ERR_CUDA.  The address is kept for the life of the process:
 *     do not call this after cudaDeviceReset on that device, or from a
 *     context other than the device's primary context; the library's module,
 *     and the scratch with it, may then sit at another address.
 *   - Each call first clears the scratch's 256-byte status header on
 *     `stream` (cudaMemsetAsync); the rest of the scratch is written before
 *     it is read, so nothing else must start at zero.
 *   - One scratch per device is shared by every call on that device: calls
 *     that may overlap (other streams, host threads, or processes sharing the
 *     context) race on it and must be ordered by the caller, e.g. on one
 *     stream.
 *   - d_scratch (may be NULL) receives the scratch's device address; pass it
 *     to zipccl_get_device_status to read the device status of the call.
 */
#define ZIPCCL_NOALLOC_MAX_PEERS 16
#define ZIPCCL_NOALLOC_SCRATCH_BYTES (256u + 1024u + 16u * 4096u)
zipccl_status zipccl_decompress_reduce_noalloc(const void *const *d_peer_chunks,
                                               const uint64_t *peer_chunk_bytes, uint32_t k,
                                               uint64_t n, uint16_t *d_out, void **d_scratch,
                                               void *stream);

/*
 * Synchronizes `stream`, then returns the status the kernels of the last call
 * on this workspace recorded (ZIPCCL_OK, ZIPCCL_ERR_CORRUPT,
 * ZIPCCL_ERR_VERSION, ZIPCCL_ERR_TIMEOUT), or ZIPCCL_ERR_CUDA.
 */
zipccl_status zipccl_get_device_status(const void *d_ws, void *stream);

/*
 * Self-test of the bounded device waits: which = 0 runs the compressor's
 * look-back for a tile whose predecessor never publishes its state; which =
 * 1 waits for an mbarrier phase that never completes (the wait used for the
 * decoders' payload copies); which = 2 runs the compress-and-send sender's
 * wait for a chunk whose tiles are never stored (no encoder runs).  The wait
 * gives up after its limit (2 s) and the kernel records ZIPCCL_ERR_TIMEOUT
 * in the workspace status, read with zipccl_get_device_status; nothing
 * faults and the context stays usable.  d_ws: 256-byte aligned, at least
 * 272 bytes (which 0, 1) or 336 bytes (which 2).  Asynchronous on `stream`.
 */
zipccl_status zipccl_selftest_bounded_wait(int which, void *d_ws, uint64_t ws_bytes, void *stream);

/*
 * Measurement hook, for timing the encode kernel on its own.  While a pair
 * of events is set, every zipccl_compress and zipccl_compress_send call
 * records ev_before (a cudaEvent_t) on its stream immediately before it
 * launches its encode kernel and ev_after immediately after, so that
 * cudaEventElapsedTime(ev_before, ev_after) is that kernel's duration (the
 * select kernel before it excluded).  The events belong to the caller, who
 * creates them with timing enabled; two NULLs turn the hook off.  One NULL
 * and one event: ZIPCCL_ERR_INVALID_ARG.  The setting is process-wide and
 * meant for a benchmark driving calls from one host thread.
 */
zipccl_status zipccl_profile_encode_events(void *ev_before, void *ev_after);

/*
 * Cost model of the switch between compressed and plain exchange ("ZipCCL:
 * Efficient Lossless Data Compression of Communication Collectives for
 * Accelerating LLM Training", abstract, technique (3): collectives switch
 * between compressed and uncompressed operation from workload and system
 * characteristics).  Host only; nothing is launched.
 *
 * zipccl_predict_chunk_bytes: the size in bytes of the stream of one chunk
 * of n values drawn from N(0, sigma^2) and compressed with a sigma hint of
 * `sigma`: the format's header, tile table and tile headers, the raw
 * sign/mantissa plane, and per tile an exponent region of
 * ceil(n_t * E / 32) words plus the segment table, E being the expected code
 * bits of one exponent under that code (closed-form masses); raw exponent
 * bytes where those are not larger.  out_bits_per_value (nullable): 8 x
 * bytes / n.  sigma <= 0, not finite, or n above the per-chunk limit give
 * ZIPCCL_ERR_INVALID_ARG.
 *
 * zipccl_choose_compressed: with link, compress and decompress throughputs
 * in GB/s of their input, sending n values raw takes 2n / link; compressed,
 * 2n / compress + bytes / link + 2n / decompress (stages in sequence, bytes
 * as predicted above).  *use_compressed = 1 when raw time / compressed time
 * > 1 + margin; predicted_speedup (nullable) receives that ratio.
 * Non-positive throughputs or a negative margin give ZIPCCL_ERR_INVALID_ARG.
 */
zipccl_status zipccl_predict_chunk_bytes(uint64_t n, float sigma, uint64_t *out_bytes, double *out_bits_per_value);
zipccl_status zipccl_choose_compressed(uint64_t n, float sigma, double link_gbs, double compress_gbs,
                                       double decompress_gbs, double margin, int *use_compressed,
                                       double *predicted_speedup);

/*
 * The code this library uses for scale phase r = q mod 16 (0..15), frozen
 * in format v1: the window start relative to floor(q/16) + 127 and the 16
 * code lengths (symbols 0..14 = window exponents, 15 = escape).  Host only.
 */
zipccl_status zipccl_codebook_phase(int phase, int *base_offset, uint8_t *lens16);

/*
 * Passages: abstract, technique (1); shd-paper key-design paragraph (the
 * code comes from the Gaussian density).
 * The same table as zipccl_codebook_phase, derived again from the
 * closed-form masses at sigma = 2^(phase/16) (exact dynamic program over
 * Kraft sums, libm erf/erfc).  The library codes only with the frozen
 * tables of format v1; this call lets a test check that they still equal
 * their derivation.  Host only.
 */
zipccl_status zipccl_codebook_rebuild_phase(int phase, int *base_offset, uint8_t *lens16);

/*
 * ---------------------------------------------------------------- operators around the exchange
 *
 * What makes and what uses the exchanged tensors in training of
 * mixture-of-experts models: routing (which token goes to which expert), the
 * plan of the experts' chunks, dispatch and combine (to and from the rows
 * that zipccl_compress packs, one chunk per expert), and the optimizer step
 * between zipccl_decompress_reduce (gradient shard) and zipccl_compress
 * (parameters).  The conventions above hold, with these differences:
 *   - pointers need only the alignment of their element type; 16-byte
 *     aligned rows and tensors are the fast path;
 *   - the calls record no device status (but for zipccl_moe_status): every
 *     index read from device memory is checked against its range, and what is
 *     out of range takes no part, as each call says;
 *   - only zipccl_moe_plan and zipccl_moe_layer need a workspace;
 *   - results overlap neither inputs nor each other, but for what a call names.
 * Sums, softmax statistics, weights and states are computed in 32 bits; a
 * result of a 16-bit type is rounded once, to nearest even.  No call's
 * result depends on timing: no atomics on results, sums in a fixed order.
 */
typedef enum {
    ZIPCCL_TYPE_F32 = 0,
    ZIPCCL_TYPE_BF16 = 1,
    ZIPCCL_TYPE_F16 = 2
} zipccl_type;

typedef enum { ZIPCCL_SCORE_SOFTMAX = 0, ZIPCCL_SCORE_SIGMOID = 1 } zipccl_score;
typedef enum { ZIPCCL_GROUP_MAX = 0, ZIPCCL_GROUP_TOP2 = 1 } zipccl_group_score;

typedef struct {
    uint32_t top_k;       /* experts of a token: 1 .. min(32, groups_kept * experts / groups) */
    int32_t score;        /* zipccl_score */
    int32_t renormalize;  /* divide the chosen scores by their sum */
    float scale;          /* factor on the weights */
    uint32_t groups;      /* 1 .. 32, a divisor of the expert count; consecutive experts form a group */
    uint32_t groups_kept; /* groups a token may choose from: 1 .. groups */
    int32_t group_score;  /* zipccl_group_score: a group's largest choice score, or the sum of its two largest */
} zipccl_route_options;

/*
 * Experts and weights of every token.  With l the logits of a token (a
 * +infinite one counts as the largest finite float):
 *   score    s_e = exp(l_e) / sum exp(l)   or   1 / (1 + exp(-l_e))
 *   choice   c_e = s_e + bias_e (d_bias: experts floats, or NULL: 0)
 *   groups   the groups_kept best by their group score (equal: lower group)
 *   experts  the top_k largest c_e in the kept groups, in descending order
 *            (equal: lower expert)
 *   weight   scale * s_e, or scale * s_e / sum of the chosen s
 * Where neither a bias nor group sums enter, the logits choose: the order of the
 * scores without their rounding.
 * The bias takes part in the choice only.  An expert whose logit is -infinite
 * or NaN, or whose c_e is, is not eligible and takes no part in the softmax
 * (the latter: in the choice); d_mask (tokens bytes, or NULL) excludes the
 * tokens whose byte is 0.  Where fewer than top_k experts are eligible the
 * remaining ids are -1 with weight 0; chosen scores that sum to 0 give
 * weights 0.
 *   d_logits: [tokens][experts] of `type`, rows row_stride >= experts values
 *     apart, 1 <= experts <= 1024;  d_weights: [tokens][top_k] float;
 *     d_ids: [tokens][top_k] int32.  tokens * top_k < 2^31.
 */
zipccl_status zipccl_moe_route(const void *d_logits, int type, uint64_t row_stride, uint64_t tokens,
                               uint32_t experts, const zipccl_route_options *options,
                               const float *d_bias, const uint8_t *d_mask, float *d_weights,
                               int32_t *d_ids, void *stream);

/*
 * Gradient of zipccl_moe_route by the logits, for the same logits, options
 * and the ids it chose (distinct for a token; ids outside the experts take no
 * part): d_grad_logits [tokens][experts] of `type`, contiguous, fully
 * written.  The choice itself has no gradient, nor has the bias.
 */
zipccl_status zipccl_moe_route_backward(const float *d_grad_weights, const void *d_logits, int type,
                                        uint64_t row_stride, uint64_t tokens, uint32_t experts,
                                        const zipccl_route_options *options, const int32_t *d_ids,
                                        void *d_grad_logits, void *stream);

/*
 * Chunk layout of `pairs` = tokens * top_k token-expert pairs with experts
 * d_ids: chunk e holds the pairs of expert e in the order of d_ids.
 *   d_counts [experts]: rows of each chunk;
 *   d_offsets [experts + 1]: first row of each chunk, and the rows in all;
 *   d_slots [pairs]: row of each pair.  A pair whose id is outside
 *     0 .. experts-1 is dropped: its slot is -1 - row, with a row of its own
 *     after the last chunk's, so that pairs and rows stay one to one.
 * pairs < 2^31, experts <= 1024.  d_ws: 256-byte aligned, at least
 * zipccl_moe_plan_workspace_bytes bytes (0 for few pairs: NULL is allowed).
 */
zipccl_status zipccl_moe_plan_workspace_bytes(uint64_t pairs, uint32_t experts, uint64_t *out_bytes);
zipccl_status zipccl_moe_plan(const int32_t *d_ids, uint64_t pairs, uint32_t experts,
                              int32_t *d_counts, int32_t *d_offsets, int32_t *d_slots, void *d_ws,
                              uint64_t ws_bytes, void *stream);

/*
 * Rows of the experts' chunks: d_rows[slot] = d_x[token] for each pair; the
 * rows of dropped pairs are zeros.  d_x: [tokens][hidden] of `type`, rows
 * row_stride values apart (0: the same row for all); d_slots:
 * [tokens][top_k], top_k <= 32; d_rows: [tokens * top_k][hidden].  A slot
 * outside the rows is skipped.
 * The backward call sums: d_grad_x[token] = sum over the token's pairs of
 * d_grad_rows[slot], dropped pairs left out.
 */
zipccl_status zipccl_moe_dispatch(const void *d_x, int type, uint64_t row_stride, uint64_t tokens,
                                  uint32_t top_k, uint64_t hidden, const int32_t *d_slots,
                                  void *d_rows, void *stream);
zipccl_status zipccl_moe_dispatch_backward(const void *d_grad_rows, int type, uint64_t tokens,
                                           uint32_t top_k, uint64_t hidden, const int32_t *d_slots,
                                           void *d_grad_x, void *stream);

/*
 * The experts' rows back at their tokens: d_y[token] = d_residual[token] +
 * sum over the token's pairs of weight * d_rows[slot].  Dropped pairs (and
 * slots outside the rows) take no part, whatever their rows hold; a token
 * without pairs gets its residual, or 0.  d_weights: [tokens][top_k] or NULL
 * (1); d_residual: [tokens][hidden] or NULL (0), may be d_y.
 * The backward call: d_grad_rows[slot] = weight * d_grad_y[token] (0 for
 * dropped pairs) and, unless NULL, d_grad_weights = <d_grad_y[token],
 * d_rows[slot]> (0 for dropped pairs).
 */
zipccl_status zipccl_moe_combine(const void *d_rows, int type, uint64_t tokens, uint32_t top_k,
                                 uint64_t hidden, const int32_t *d_slots, const float *d_weights,
                                 const void *d_residual, void *d_y, void *stream);
zipccl_status zipccl_moe_combine_backward(const void *d_grad_y, const void *d_rows, int type,
                                          uint64_t tokens, uint32_t top_k, uint64_t hidden,
                                          const int32_t *d_slots, const float *d_weights,
                                          void *d_grad_rows, float *d_grad_weights, void *stream);

/*
 * One AdamW step, in place, over n_tensors tensors (host array) in as few
 * launches as their records fit.  With g the gradient (times *d_grad_scale,
 * a device float, unless NULL):
 *   m = beta1 m + (1 - beta1) g          v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^step) *
 *       m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * (a divisor below 2^-126 counts as 2^-126, one of NaN makes p NaN; the quotient
 * is a product with the divisor's reciprocal, good to 1 ulp) and, where d_copy is
 * set, d_copy = bf16(p).
 * param_type: F32 or BF16 (then p is rounded at every step);  grad_type: F32
 * or BF16.
 * state_bits 32: d_exp_avg and d_exp_avg_sq hold m and v as floats.
 * state_bits 8: they hold m and sqrt(v) as E4M3 bytes (4 exponent, 3 mantissa
 * bits) times one float scale for each block of ZIPCCL_ADAMW_BLOCK
 * consecutive values of a tensor, in d_avg_scale and d_sq_scale
 * (ceil(n / ZIPCCL_ADAMW_BLOCK) each).  The new scale is the block's largest
 * finite magnitude over 448 (at least 2^-126); a positive sqrt(v) is never
 * stored as 0, so that no step is divided by eps alone; what is not finite is
 * stored as NaN, in its own place only.  The step itself uses the new m and v
 * before they are rounded.  Zero bytes and any finite scale are a valid start.
 * 0 <= beta1, beta2 < 1; lr, eps, weight_decay >= 0; step >= 1.  The options
 * are launch parameters: a captured graph replays them unchanged.
 */
#define ZIPCCL_ADAMW_BLOCK 256u
typedef struct {
    void *d_param;
    const void *d_grad;
    void *d_exp_avg;
    void *d_exp_avg_sq;
    void *d_copy;       /* nullable: BF16 copy of the new parameters */
    float *d_avg_scale; /* state_bits 8 only */
    float *d_sq_scale;  /* state_bits 8 only */
    uint64_t n;
} zipccl_adamw_tensor;

typedef struct {
    double lr, beta1, beta2, eps, weight_decay;
    uint64_t step; /* 1 for the first */
} zipccl_adamw_options;

zipccl_status zipccl_adamw_step(const zipccl_adamw_tensor *tensors, uint32_t n_tensors, int param_type,
                                int grad_type, int state_bits, const zipccl_adamw_options *options,
                                const float *d_grad_scale, void *stream);

/*
 * ---------------------------------------------------------------- what the experts compute
 *
 * 8-bit blocks.  A block of values x with the largest finite magnitude a has
 * the scale 2^e, e the smallest whole number from -127 on with a <= 448 * 2^e,
 * and the codes E4M3(x * 2^-e), to nearest even: the scaling is exact, so the
 * code is the only rounding.  A value that is not finite has the code of NaN,
 * in its own place only.  Scales are bytes e + 127 (E8M0: 255 is NaN, as a
 * block's scale may be set by others).  Codes: rows code_stride bytes apart, a
 * multiple of 16, from a 16-byte aligned start.  At most 2^31 - 1 rows and
 * 2^22 columns.
 *
 * zipccl_moe_quantize: blocks of ZIPCCL_FP8_BLOCK consecutive values of a
 *   row.  d_x [rows][cols] of `type`, rows row_stride values apart; d_scales
 *   [rows][ceil(cols / 128)].
 * zipccl_moe_quantize_columns: blocks of 128 consecutive rows of a chunk in
 *   one column; chunk e is the rows d_offsets[e] .. d_offsets[e + 1] - 1, as
 *   zipccl_moe_plan gives them (d_offsets NULL, experts 1: all rows).  d_scales
 *   [rows / 128 + experts][cols]: chunk by chunk, ceil(rows of the chunk / 128)
 *   each, then zero bytes; rows behind the last chunk have codes of zero.  With
 *   d_row_codes and d_row_scales (or NULL) also what zipccl_moe_quantize gives,
 *   from the same reading.
 * zipccl_moe_quantize_weights: blocks of 128 x 128.  d_w [experts][rows][cols],
 *   contiguous; d_codes [experts][rows] rows; d_scales [experts]
 *   [ceil(rows / 128)][ceil(cols / 128)].
 */
#define ZIPCCL_FP8_BLOCK 128u
zipccl_status zipccl_moe_quantize(const void *d_x, int type, uint64_t row_stride, uint64_t rows, uint64_t cols,
                                  uint8_t *d_codes, uint64_t code_stride, uint8_t *d_scales, void *stream);
zipccl_status zipccl_moe_quantize_columns(const void *d_x, int type, uint64_t row_stride, uint64_t rows,
                                          uint64_t cols, const int32_t *d_offsets, uint32_t experts,
                                          uint8_t *d_codes, uint64_t code_stride, uint8_t *d_scales,
                                          uint8_t *d_row_codes, uint64_t row_code_stride,
                                          uint8_t *d_row_scales, void *stream);
zipccl_status zipccl_moe_quantize_weights(const void *d_w, int type, uint32_t experts, uint64_t rows,
                                          uint64_t cols, uint8_t *d_codes, uint64_t code_stride,
                                          uint8_t *d_scales, void *stream);

/*
 * Products of the experts' chunks with their matrices, operands in 8-bit
 * blocks, chunks as d_offsets [experts + 1] gives them (NULL with experts 1:
 * all rows; offsets are taken from 0 on, never falling and within the rows,
 * whatever the memory holds).  With x, w, g the values that the codes and
 * scales stand for:
 *   ZIPCCL_MATMUL_FORWARD   out[m][n] = sum_k x[m][k] w[e][n][k]
 *       a: rows [rows][inner] by rows; b: weights [experts][outer][inner];
 *       out [rows][outer]
 *   ZIPCCL_MATMUL_BACKWARD  out[m][k] = sum_n g[m][n] w[e][n][k]
 *       a: gradients [rows][outer] by rows; b: the same weights;
 *       out [rows][inner]
 *   ZIPCCL_MATMUL_WEIGHTS   out[e][n][k] = sum of g[m][n] x[m][k] over the
 *       chunk's rows; a: gradients [rows][outer] by columns; b: rows
 *       [rows][inner] by columns; out [experts][outer][inner]
 * Rows behind the last chunk are zeros in `out`, as are the gradients of the
 * weights of an empty chunk.  inner and outer are 1 at least.  out: rows
 * out_stride values apart, the WEIGHTS form's matrices `outer` rows apart; out_type
 * F32, BF16 or F16, rounded once from 32 bits.
 * Sums are held in 32 bits on the tensor cores, in a fixed order.  An instruction
 * adds 32 terms and cuts off what lies below the sum's last place, where float
 * additions would round: a sum of n terms is off by (n / 32 + 1) 2^-22 of their
 * magnitudes' sum at most, and one whose terms have one sign comes out small, by n
 * 2^-29 of itself at most (measured: 1.5e-6 for 4,096 terms, 9.9e-6 for 16,384).
 * A wait inside a kernel of this call or of zipccl_moe_layer that runs out (2 s
 * and 4 us for each 128 terms of a sum; not to be expected) leaves its results undefined and sets a word of the current
 * device that zipccl_moe_status reads and clears: ZIPCCL_OK or ZIPCCL_ERR_TIMEOUT
 * (synchronizes `stream`).
 */
typedef enum { ZIPCCL_MATMUL_FORWARD = 0, ZIPCCL_MATMUL_BACKWARD = 1, ZIPCCL_MATMUL_WEIGHTS = 2 } zipccl_matmul_form;

typedef struct {
    const uint8_t *d_codes;  /* 16-byte aligned */
    const uint8_t *d_scales; /* contiguous, laid out as the quantizing call leaves them */
    uint64_t stride;         /* bytes between rows of codes, a multiple of 16 */
} zipccl_fp8_blocks;

zipccl_status zipccl_moe_matmul(int form, const zipccl_fp8_blocks *a, const zipccl_fp8_blocks *b,
                                uint64_t rows, uint64_t inner, uint64_t outer, const int32_t *d_offsets,
                                uint32_t experts, void *d_out, int out_type, uint64_t out_stride, void *stream);
zipccl_status zipccl_moe_status(void *stream);

/*
 * A whole mixture-of-experts layer for up to ZIPCCL_LAYER_MAX_TOKENS tokens, in
 * two kernels.  With x a token's row:
 *   logits = router x, in 32 bits; weights and ids as zipccl_moe_route gives for
 *     them (options, d_bias, d_mask: the same)
 *   h_k    = act(gate x) * (up x), where gate and up are the first and the last
 *     `inner` rows of expert k's matrix in d_up; ungated: act(up x)
 *   y      = d_residual + sum over the token's experts of weight_k * down_k h_k
 * Sums are held in 32 bits.  A 16- or 8-bit operand takes part exactly, a 32-bit
 * one and h with 21 bits at least.  A token without experts gets its residual, or 0: a
 * logit that is NaN or -inf takes no part in the choice, so a token with a NaN has
 * none.  What something infinite or NaN takes part in, by the experts chosen, is
 * infinite or NaN.
 *   d_x [tokens][hidden] of `type`, rows x_stride values apart (0: all the same,
 *     else hidden at least);
 *     d_router [experts][hidden] of router_type: `type` or F32;
 *     d_up [experts][gated ? 2 inner : inner][hidden], d_down [experts][hidden]
 *     [inner]: of `type` (weight_bits those of the type), or 8-bit blocks
 *     (weight_bits 8, scales as zipccl_moe_quantize_weights leaves them); rows
 *     up_stride and down_stride values apart;
 *     d_residual, d_y [tokens][hidden], d_residual may be d_y;
 *     d_weights, d_ids [tokens][top_k], written.
 * act: SILU v / (1 + exp(-v)); GELU v (1 + erf(v / sqrt 2)) / 2; RELU max(v, 0).
 * d_ws: 256-byte aligned, zipccl_moe_layer_workspace_bytes bytes; nothing in it
 * has to be set, and nothing is kept in it.  Calls that may run at the same time
 * (on two streams, in two graphs) need workspaces of their own.
 */
#define ZIPCCL_LAYER_MAX_TOKENS 32u
typedef enum { ZIPCCL_ACTIVATION_SILU = 0, ZIPCCL_ACTIVATION_GELU = 1, ZIPCCL_ACTIVATION_RELU = 2 } zipccl_activation;

typedef struct {
    const void *d_x, *d_router, *d_up, *d_down;
    const void *d_residual;                      /* nullable */
    const uint8_t *d_up_scales, *d_down_scales;  /* weight_bits 8 only */
    const float *d_bias;                         /* nullable */
    const uint8_t *d_mask;                       /* nullable */
    void *d_y;
    float *d_weights;
    int32_t *d_ids;
    uint64_t tokens, hidden, inner, x_stride, up_stride, down_stride;
    uint32_t experts;
    int32_t type, router_type, weight_bits, gated, activation;
} zipccl_moe_layer_args;

zipccl_status zipccl_moe_layer_workspace_bytes(uint64_t tokens, uint32_t top_k, uint64_t inner, uint64_t *out_bytes);
zipccl_status zipccl_moe_layer(const zipccl_moe_layer_args *args, const zipccl_route_options *options, void *d_ws,
                               uint64_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ZIPCCL_H */
