/*
 * streamscan.h -- C ABI of libstreamscan.so: device-wide prefix sums and
 * order-preserving stream compaction on one NVIDIA GB300 (sm_103a).
 *
 * Definitions ("Prefix sum and other parallel patterns", Definitions):
 *   inclusive  out[i] = in[0] + ... + in[i]
 *   exclusive  out[i] = in[0] + ... + in[i-1],  out[0] = 0
 * e.g. in = [3,1,7,0,4,1,6,3] gives inclusive [3,4,11,11,15,16,22,25] and
 * exclusive [0,3,4,11,11,15,16,22].
 *
 * Conventions shared by every call:
 *   - Pointers named in/out/keys/flags/d_count/d_carry_* are DEVICE
 *     pointers owned by the caller (e.g. from torch, cudaMalloc).  Pointers
 *     named h_* are HOST pointers.  The library never frees caller memory.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Device
 *     calls only enqueue work and return; results are ready when the stream
 *     reaches them.  Calls on one stream run in order; calls on different
 *     streams are independent (each (device, stream) pair has its own
 *     workspace).
 *   - int32 and uint32 sums wrap modulo 2^32 (two's complement for int32).
 *     fp32 sums use IEEE round-to-nearest adds in an order the caller does
 *     not control; the last bits of an fp32 result may differ from run to
 *     run, because a tile adds its predecessors' published sums in whatever
 *     grouping the look-back found.
 *   - 16-byte aligned in/out take the vectorised path; any 4-byte aligned
 *     pointers are accepted and take a slower element-wise path.
 *   - Argument errors are found before anything is enqueued and return
 *     SS_ERR_INVALID_ARG (ss_last_error_detail() says why).  Launch
 *     failures return SS_ERR_CUDA.  Errors found on the device (a look-back
 *     wait that ran out) are recorded in the stream's status word and
 *     returned by the next ss_stream_status() call on that stream; the
 *     outputs of the failing call are then undefined.
 *   - n == 0 is a valid no-op (the compactions still write *d_count = 0).
 *   - The library owns a small per-(device, stream) workspace (tile
 *     descriptors, a tile counter, the status word), about 8 bytes per 4096
 *     elements, grown on demand with stream-ordered allocation and freed
 *     by ss_shutdown().  Size it before capturing a stream into a CUDA
 *     graph by making one call of the largest n on that stream first; a
 *     captured graph may then be replayed any number of times up to 2^29
 *     (the device-side launch epoch separates the replays).
 */
#ifndef STREAMSCAN_H
#define STREAMSCAN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t, declared here so that the header needs no CUDA
 * include. */
typedef struct CUstream_st *ss_stream_t;

typedef enum ss_status {
    SS_OK = 0,
    SS_ERR_INVALID_ARG = 1,      /* bad pointer, size or overlap */
    SS_ERR_CUDA = 2,             /* a CUDA runtime call or launch failed */
    SS_ERR_LOOKBACK_TIMEOUT = 3, /* a tile's look-back wait ran out */
    SS_ERR_NO_MEMORY = 4,        /* workspace allocation failed */
    SS_ERR_UNSUPPORTED = 5       /* no usable device, or bad enum value */
} ss_status;

typedef enum ss_dtype { SS_I32 = 0, SS_U32 = 1, SS_F32 = 2 } ss_dtype;

/* Algorithms for ss_scan().  SS_ALGO_LOOKBACK is the product path; the
 * others are the measured ablations. */
typedef enum ss_algo {
    SS_ALGO_LOOKBACK = 0,            /* single pass, decoupled look-back, 2n traffic */
    SS_ALGO_REDUCE_THEN_SCAN = 1,    /* three kernels, 3n traffic */
    SS_ALGO_RTS_BLELLOCH = 2,        /* same, third kernel a Blelloch tree, unpadded */
    SS_ALGO_RTS_BLELLOCH_PAD32 = 3,  /* same, tree padded i + i/32 */
    SS_ALGO_RTS_BLELLOCH_PAD2 = 4    /* same, tree padded i + i/32 + i/1024 */
} ss_algo;

/*
 * Device-wide scans, single pass with decoupled look-back ("Prefix sum and
 * other parallel patterns", A device-level scan: scan then propagate --
 * each block looks back at the states earlier blocks published, "local sum
 * only" or "inclusive prefix available").
 *   in   device, n elements, read once.
 *   out  device, n elements, written once.  out == in is allowed (in-place);
 *        any other overlap is SS_ERR_INVALID_ARG.
 *   n    element count, 0 <= n < 2^31 * 4096.
 */
ss_status scan_inclusive_i32(const int32_t *in, int32_t *out, size_t n, ss_stream_t stream);
ss_status scan_exclusive_i32(const int32_t *in, int32_t *out, size_t n, ss_stream_t stream);
ss_status scan_inclusive_u32(const uint32_t *in, uint32_t *out, size_t n, ss_stream_t stream);
ss_status scan_exclusive_u32(const uint32_t *in, uint32_t *out, size_t n, ss_stream_t stream);
ss_status scan_inclusive_f32(const float *in, float *out, size_t n, ss_stream_t stream);
ss_status scan_exclusive_f32(const float *in, float *out, size_t n, ss_stream_t stream);

/*
 * Scans with 64-bit sums ("Parallel Prefix Sum (Scan) for NVIDIA T4
 * (sm_75)", Key Features: 64-bit indexing for large arrays; the sum of many
 * 32-bit counts needs 64 bits).  Same definitions and method as the 32-bit
 * scans, with 16-byte tile descriptors.
 *   u32_u64  uint32 in, uint64 out: the exact sums (no wrap below 2^64).
 *   i32_i64  (ss_scan_wide only) int32 in, int64 out: the exact sums.
 *   i64      int64 in and out, wrapping modulo 2^64 (uint64 data gives the
 *            same bits).
 *   f64      fp64 in and out, IEEE round-to-nearest adds in an order the
 *            caller does not control (as for fp32).
 *   in   device, n elements, aligned to the element size (16-byte aligned
 *        in and out take the bulk-copy path; for f64, the tensor-copy path).
 *   out  device, n 8-byte elements.  out == in is allowed for i64 and f64;
 *        any other overlap is SS_ERR_INVALID_ARG.
 *   n    0 <= n < 2^31 * 8192.
 */
typedef enum ss_wide_type {
    SS_WIDE_U32_U64 = 0,
    SS_WIDE_I32_I64 = 1,
    SS_WIDE_I64 = 2,
    SS_WIDE_F64 = 3
} ss_wide_type;
ss_status scan_inclusive_u32_u64(const uint32_t *in, uint64_t *out, size_t n, ss_stream_t stream);
ss_status scan_exclusive_u32_u64(const uint32_t *in, uint64_t *out, size_t n, ss_stream_t stream);
ss_status scan_inclusive_i64(const int64_t *in, int64_t *out, size_t n, ss_stream_t stream);
ss_status scan_exclusive_i64(const int64_t *in, int64_t *out, size_t n, ss_stream_t stream);
ss_status scan_inclusive_f64(const double *in, double *out, size_t n, ss_stream_t stream);
ss_status scan_exclusive_f64(const double *in, double *out, size_t n, ss_stream_t stream);
ss_status ss_scan_wide(ss_wide_type type, int inclusive, const void *in, void *out, size_t n,
                       ss_stream_t stream);

/*
 * Order-preserving stream compaction in one pass: out receives, in index
 * order, every keys[i] whose flags[i] != 0, and *d_count the number kept
 * ("Prefix sum and other parallel patterns", Stream compaction and
 * Exercise 1: out[pos[i]] = in[i] with pos the exclusive scan of the 0/1
 * keep flags, count = pos[n-1] + flags[n-1]; fused so that the flags' scan
 * and the positions never reach device memory).
 *   keys     device, n uint32.
 *   flags    device, n uint8; any nonzero byte keeps the element.
 *   out      device, room for n uint32 (only the first *d_count written);
 *            must not overlap keys or flags.
 *   d_count  device, one uint64, written by the call.
 *   n        0 <= n < 2^32.
 */
ss_status compact_u32(const uint32_t *keys, const uint8_t *flags, uint32_t *out,
                      uint64_t *d_count, size_t n, ss_stream_t stream);

/*
 * Order-preserving compaction with a built-in predicate instead of a flag
 * array: out receives, in index order, every in[i] with in[i] > 0, and
 * *d_count the number kept ("Prefix sum and other parallel patterns",
 * Stream compaction, compact.cu's predicate v > 0, and Exercise 1's flags
 * in[i] > 0 fused into the scan's passes).  The predicate is evaluated in
 * the element type: for fp32, NaN, +0.0 and -0.0 are dropped and +inf is
 * kept; for int32 it is signed; for uint32 it means nonzero.  Kept elements
 * are copied bit for bit.
 *   in       device, n elements of `dtype`, read once.
 *   out      device, room for n elements (only the first *d_count written);
 *            must not overlap in.
 *   d_count  device, one uint64, written by the call.
 *   n        0 <= n < 2^32.
 * Errors as compact_u32.
 */
ss_status compact_positive_f32(const float *in, float *out, uint64_t *d_count, size_t n, ss_stream_t stream);
ss_status ss_compact_positive(ss_dtype dtype, const void *in, void *out, uint64_t *d_count, size_t n,
                              ss_stream_t stream);

/*
 * Unordered compaction (the measured ablation): the same kept elements and
 * count as compact_u32 / ss_compact_positive, but in no fixed order.  Each
 * warp claims room for its kept elements with one atomic add on *d_count
 * and writes them at the claimed offset plus their rank inside the warp
 * ("Prefix sum and other parallel patterns", Stream compaction: the
 * warp-aggregated atomic, ballot and popc).  Within each 512-element batch
 * of a warp the order is kept; the order of the batches depends on the
 * timing of the atomics.  Needs no workspace and no look-back.  *d_count is
 * zeroed on the stream first, then counted up by the kernel.  Arguments and
 * errors as the ordered calls.
 */
ss_status ss_compact_u32_unordered(const uint32_t *keys, const uint8_t *flags, uint32_t *out,
                                   uint64_t *d_count, size_t n, ss_stream_t stream);
ss_status ss_compact_positive_unordered(ss_dtype dtype, const void *in, void *out, uint64_t *d_count,
                                        size_t n, ss_stream_t stream);

/*
 * Batched scans: every row of a row-major rows x cols matrix scanned on its
 * own, the sum starting from zero at each row (for example the cumulative
 * sum over each row's sorted probabilities in top-p sampling, "Prefix sum
 * and other parallel patterns", In LLMs: MoE token dispatch, last
 * paragraph).  Same element types, wraparound and fp32 rules as the flat
 * scans.
 *   in    device, rows * cols elements, row r at in + r * cols.
 *   out   device, same shape; out == in is allowed, any other overlap is
 *         SS_ERR_INVALID_ARG.
 *   rows, cols  either may be 0 (a no-op); rows * cols < 2^31 * 4096, and
 *         for rows longer than 2048 elements rows * ceil(cols / 4096) < 2^31.
 * Rows longer than 2048 elements use row-aligned tiles with the decoupled
 * look-back (the per-stream workspace); shorter rows take one warp each;
 * rows of 2^21 elements or more run as one flat scan each.
 */
ss_status ss_scan_rows(ss_dtype dtype, int inclusive, const void *in, void *out, size_t rows, size_t cols,
                       ss_stream_t stream);

/*
 * Segmented scans: every segment [offsets[s], offsets[s+1]) of a flat array
 * scanned on its own, from zero; the general form of ss_scan_rows, for rows
 * of different lengths.  Same element types, wraparound and fp32 rules as the
 * flat scans.
 *   in, out       device, n elements each; out == in is allowed, any other
 *                 overlap is SS_ERR_INVALID_ARG.
 *   d_offsets     device, num_segments + 1 uint64: offsets[0] = 0,
 *                 non-decreasing, offsets[num_segments] = n (empty segments
 *                 are fine).  Only the starts offsets[0 .. num_segments-1]
 *                 are read, and the scan restarts at each start below n (so
 *                 with offsets as described the result is the definition
 *                 above).
 *   num_segments  0 means one segment, the whole array.
 * Two launches on the stream: a pass that marks the segment starts in a
 * workspace bitmask (n / 8 bytes), then the single-pass scan with a
 * segmented add, in which a tile holding a segment start publishes its
 * inclusive prefix at once.
 */
ss_status ss_scan_segments(ss_dtype dtype, int inclusive, const void *in, void *out, size_t n,
                           const uint64_t *d_offsets, size_t num_segments, ss_stream_t stream);

/*
 * MoE token counts and expert offsets aligned to GEMM tiles ("Prefix sum and
 * other parallel patterns", In LLMs: MoE token dispatch, steps 1-2, and
 * Exercise 2: a histogram of the router's expert ids, then an exclusive
 * prefix sum for each expert's start, each expert's segment rounded up to a
 * multiple of the tile size):
 *   counts[e]    = number of i < m with topk_ids[i] == e
 *   offsets[0]   = 0,  offsets[e+1] = offsets[e] + align * ceil(counts[e] / align)
 * An id outside [0, num_experts) is counted nowhere.
 *   topk_ids     device, m int32 (a row-major num_tokens x top_k array, flat).
 *   m            number of ids, 0 <= m < 2^31.
 *   num_experts  E, 1 <= E <= 16384.
 *   align        tile size, 1 <= align <= 2^20 (1 gives the plain exclusive
 *                scan of the counts); m + E * (align - 1) must fit 32 bits.
 *   d_counts     device, E uint32, written.
 *   d_offsets    device, E + 1 uint32, written (offsets[E] = padded total).
 * One kernel launch; no allocation after the stream's first call with this
 * E and grid size.  Arrays must not overlap.
 */
ss_status ss_moe_counts_offsets(const int32_t *topk_ids, size_t m, int32_t num_experts, uint32_t align,
                                uint32_t *d_counts, uint32_t *d_offsets, ss_stream_t stream);

/*
 * A paged key-value cache, with the attention of one new token per sequence
 * that reads it and the eviction that compacts it.
 *
 * The pool (ss_kv_pages): num_pages pages, each holding page_size tokens of
 * every key-value head.  Element d of the key of head h at slot s of page p
 * is k[p * page_stride + h * head_stride + s * slot_stride + d] (strides in
 * elements; [page][head][slot][dim] and [page][slot][head][dim] are both
 * strides of this), and the same offset in v.  An SS_E4M3 cache holds
 * value / scale: k_scale and v_scale are device arrays of kv_heads floats
 * (NULL: 1), and must be NULL for the 16-bit types.  An SS_E2M1 cache packs
 * two elements to a byte, the lower index in the low half, and holds beside them
 * a scale for every 16 elements: element d is e2m1(code d) * e4m3(k_block[((p *
 * kv_heads + h) * page_size + s) * head_dim / 16 + d / 16]) * k_scale[h], and the
 * same in v (k_block and v_block: device, contiguous, 16-byte aligned; read for
 * this type only).  `weight` (device,
 * contiguous [page][head][slot] floats, NULL: none) holds the attention that
 * each cached token has gathered.
 *
 * The sequences (ss_kv_table): position i of sequence b lives at slot
 * i % page_size of page pages[b * row_stride + i / page_size].  lens[b] is
 * its length; entries of `pages` past the length are not read.  max_len is
 * an upper bound on the lengths known to the host (0: max_pages *
 * page_size); it sizes launches and scratch.
 *
 * Shared rules:
 *   - head_dim is at most 256 and head_dim * element size a multiple of 16
 *     bytes, as are the strides (those of an extent of 1 are not looked at); an
 *     SS_E2M1 cache has a head_dim of 64, 128 or 256;
 *     k, v, the rows of new tokens, q and out are 16-byte aligned.
 *   - Lengths and page numbers are device data, checked on the device: a
 *     length below 0 or above max_len (or max_pages * page_size) is clamped,
 *     a page number outside [0, num_pages) is not followed, and either is
 *     reported by the next ss_stream_status() as SS_ERR_INVALID_ARG with the
 *     sequence in *failing_tile; the outputs of that sequence are then
 *     undefined, and nothing outside the arrays is touched.
 *   - batch == 0 is a no-op.  Results do not change from run to run.
 *   - attend and evict keep scratch in the stream's workspace, sized by
 *     batch, heads and max_len and grown by half at least.  With weights that
 *     is 4 bytes a score: of all sequences, or of as many as 2 GB hold, but of
 *     one at least.  As for the other calls, make one call of the largest size
 *     before capturing a stream into a graph: calls of no more sequences,
 *     key-value heads and positions, all else alike (also the query heads per
 *     key-value head, weights and `kept`), then need no more.  A call whose
 *     scratch would have to grow while its stream is being captured (or that
 *     is the first on that stream) returns SS_ERR_NO_MEMORY and enqueues
 *     nothing; one that makes it grow later leaves a captured graph its own.
 *     Graphs captured from one stream share its scratch, and are replayed one
 *     after the other.
 */
typedef enum ss_elem { SS_BF16 = 0, SS_F16 = 1, SS_E4M3 = 2, SS_E2M1 = 3, SS_ELEM_F32 = 4 } ss_elem;

typedef struct ss_kv_pages {
    ss_elem type;
    int32_t kv_heads;
    int32_t head_dim;
    int32_t page_size;
    int64_t num_pages;
    void *k;
    void *v;
    int64_t page_stride;
    int64_t head_stride;
    int64_t slot_stride;
    const float *k_scale;
    const float *v_scale;
    float *weight;
    uint8_t *k_block;
    uint8_t *v_block;
} ss_kv_pages;

typedef struct ss_kv_table {
    const int32_t *pages;
    int64_t row_stride;
    int32_t max_pages;
    int32_t batch;
    int32_t *lens;
    int32_t max_len;
} ss_kv_table;

/*
 * Appends new tokens' keys and values.  Sequence b has the new tokens
 * offsets[b] .. offsets[b+1] - 1 of k_new and v_new (offsets NULL: one token
 * each, token b), and lens[b] already counts them: they become its last
 * positions, in order.  Token t's row of head h starts at k_new + t *
 * token_stride + h * head_stride (elements of `type`, SS_BF16 or SS_F16;
 * the strides serve a fused projection's output in place).  The cache holds
 * `type`, or SS_E4M3: each element is then x / scale[h] (fp32 division)
 * clamped to [-448, 448] and rounded to the nearest e4m3, ties to even; NaN
 * stays NaN.  Or it holds SS_E2M1: with y = x * (1 / scale[h]) (both fp32), a
 * block's scale is max |y| / 6 as the nearest e4m3, at most 448 (NaN where an
 * element is NaN), and a code that of y over its block's scale, the nearest of 0,
 * 0.5, 1, 1.5, 2, 3, 4 and 6 with y's sign (0 where the scale is 0), ties to the
 * even code, in fp32.  The new slots' weights become 0 (where weight is not NULL).
 *   offsets  device, batch + 1 int32, offsets[0] = 0, non-decreasing, or NULL.
 *   tokens   offsets[batch]; batch where offsets is NULL.  tokens *
 *            kv_heads < 2^31.
 * No two sequences may share a page that is appended to.
 */
ss_status ss_kv_append(const ss_kv_pages *cache, const ss_kv_table *seqs, ss_elem type, const void *k_new,
                       const void *v_new, int64_t token_stride, int64_t head_stride, const int32_t *offsets,
                       size_t tokens, ss_stream_t stream);

/*
 * Page tables and slot maps from the lengths that sequences grow by.  Sequence
 * b has lens[b] tokens (none where restart[b] is not 0: another request takes
 * its place) and gets counts[b] more.  The pages that it needs beyond those that
 * it holds come from the front of a ring of free pages, in the order of the
 * sequences; the pages of restarted sequences go to the ring's end, in the same
 * order, and are handed out from the next call on.  A sequence is served where it
 * needs no page, or where the needs up to and including its own do not exceed the
 * ring's count; otherwise it gets nothing and its length stays (0 if restarted).
 *   into       receives the table and the lengths; NULL: seqs itself.  It may
 *              share either array with seqs.  Its max_pages and max_len are at
 *              least seqs', and its max_len bounds the new lengths: a count that
 *              is negative or leads past it is not served, and reported.
 *              Entries past a sequence's pages are left as they were.
 *   page_size, num_pages  of the pool, for the numbers that pages may have.
 *   counts     device, batch int32, or NULL: one token each.
 *   restart    device, batch bytes, or NULL: none.
 *   free_pages the ring: `capacity` page numbers (at least all of the pool's that
 *              are handed out this way) and state = {head, count}, device: the place
 *              of the first one, taken modulo the capacity, and how many there are.
 *   left       device, two int32: the state afterwards; NULL: state itself.
 *   offsets    device, batch + 1 int32, or NULL: the counts' exclusive sums,
 *              served or not (a negative count is 0).
 *   positions  device, `tokens` int32, or NULL: of token offsets[b] + i, lens[b] + i.
 *   slots      device, `tokens` int64, or NULL: page * page_size + slot of that
 *              position, -1 where the sequence is not served.
 *   tokens     the room of positions and slots: tokens behind offsets[batch] get
 *              position 0 and slot -1, so that a fixed size serves every call; more
 *              counts than room are reported.
 * Lengths, counts and page numbers are checked on the device, as for the other
 * calls.  batch <= 8192, batch * max_pages < 2^31, and all counts' sum is below
 * 2^31 (reported otherwise).  What it reports lies in the stream's workspace: make one
 * call before capturing a stream into a graph.
 */
typedef struct ss_kv_free {
    int32_t *pages;
    int64_t capacity;
    int32_t *state;
} ss_kv_free;
ss_status ss_kv_assign(const ss_kv_table *seqs, const ss_kv_table *into, int32_t page_size, int64_t num_pages,
                       const int32_t *counts, const uint8_t *restart, const ss_kv_free *free_pages, int32_t *left,
                       int32_t *offsets, int32_t *positions, int64_t *slots, size_t tokens, ss_stream_t stream);

/*
 * Norms of query and key rows with the rotation by their positions, in one
 * pass: for every token's and head's row x
 *   y = R(p) (x / sqrt(mean(x^2) + eps) * w),
 * where R(p) turns the pairs (x_i, x_{i + r/2}), or (x_2i, x_2i+1) where
 * interleaved, i < r/2, by the angle of position p, and leaves elements from r =
 * rotary_dim on as they are:  (a, b) -> (a cos - b sin, b cos + a sin).  Angles
 * are p * turns[i] / 2^64 turns modulo 1, exact for every p; sums and products
 * are fp32, and y is rounded once.  Sines and cosines of SS_ELEM_F32 rows, and of
 * k's on their way into an SS_E4M3 or SS_E2M1 cache, are good to 2^-22 of their own
 * value, and the reciprocal root to half a unit in the last place; those of other
 * rows to 2^-20 (absolute, of pairs whose lengths are 1) and to two units, so that
 * where a cos and b sin nearly cancel an SS_F16 output may be off by more than its
 * rounding.
 *   type       of q, k and the outputs: SS_BF16, SS_F16 or SS_ELEM_F32.
 *   q, k       rows (token, head) of head_dim consecutive elements; strides in
 *              elements, multiples of 16 bytes, at most 2^33, 16-byte aligned.
 *              Either may have no heads (then it is not read).
 *   q_weight, k_weight  device, head_dim numbers of weight_type (SS_BF16, SS_F16
 *              or SS_ELEM_F32), or NULL: ones.
 *   positions  device, a token each; may be negative.
 *   q_out, k_out  each is its own input's rows, or shares no memory with either
 *              (rows may lie between each other's; tensors of two token strides whose
 *              ranges meet are taken for overlapping).
 *   head_dim a multiple of 8, at most 256; rotary_dim a positive multiple of 16,
 *   at most head_dim.  tokens == 0 is a no-op.  The call takes no scratch and may be
 *   the first one on a stream that is being captured.
 *
 * ss_qk_norm_rope_backward: from the gradients of the outputs, dq_out and dk_out,
 * those of the inputs (dq and dk: the rows of an input or of a gradient of their
 * own, or apart from all) and of the weights, summed over all tokens and heads
 * in a fixed order (fp32, head_dim numbers each, or NULL).  The partial sums lie
 * in the stream's workspace: make one call before capturing a stream into a graph,
 * and replay graphs that were captured from one stream one after the other.
 *
 * ss_kv_append_rope: the same with k's and v's rows written into a cache, v's as
 * they are: token t's to slot slots[t] (page * page_size + slot in the page, as
 * ss_kv_assign gives them; a negative one: nowhere).  What the cache holds is as
 * after ss_kv_append of y, which is not rounded to `type` before; the slots'
 * weights become 0.  Slots behind the pool are reported with the token.  No two
 * tokens share a slot, and q_out no memory with the cache.  type: SS_BF16 or SS_F16;
 * rotary_dim a multiple of 32 for an SS_E2M1 cache.  Make one call before capturing a
 * stream into a graph, as for ss_kv_assign.
 */
typedef struct ss_rows {
    void *data;
    int64_t token_stride;
    int64_t head_stride;
} ss_rows;
typedef struct ss_rope {
    const uint64_t *turns; /* device, rotary_dim / 2: the angle of one position in units of 2^-64 turns */
    int32_t rotary_dim;
    int32_t interleaved;
} ss_rope;
typedef struct ss_qk {
    ss_elem type;
    ss_elem weight_type;
    int32_t head_dim;
    int32_t q_heads;
    int32_t kv_heads;
    float eps;
    int64_t tokens;
    ss_rows q;
    ss_rows k;
    const void *q_weight;
    const void *k_weight;
    const int32_t *positions;
    ss_rope rope;
} ss_qk;
ss_status ss_qk_norm_rope(const ss_qk *x, const ss_rows *q_out, const ss_rows *k_out, ss_stream_t stream);
ss_status ss_qk_norm_rope_backward(const ss_qk *x, const ss_rows *dq_out, const ss_rows *dk_out, const ss_rows *dq,
                                   const ss_rows *dk, float *dq_weight, float *dk_weight, ss_stream_t stream);
ss_status ss_kv_append_rope(const ss_kv_pages *cache, const int64_t *slots, const ss_qk *x, const ss_rows *v,
                            const ss_rows *q_out, ss_stream_t stream);

/*
 * Attention of one token per sequence over its cached positions.  Query head
 * j of q_heads = group * kv_heads reads key-value head j / group.  With s(p)
 * = scale * (q . k(p)) over the visible positions {p < len : window <= 0 or p
 * < sinks or p >= len - window}:
 *   out = sum_p exp(s(p) - lse) v(p),   lse = log sum_p exp(s(p)),
 *   weight_out(h, p) = weight_in(h, p) + sum over h's query heads of
 *                      exp(s(p) - lse), for every position p < len.
 * A row with no visible position, or all of whose scores are -inf, gives
 * out = 0 and lse = -inf and adds no weight.  NaN and infinities in a visible
 * row spread as in the formula, whatever the other sequences are: the weight
 * of a finite score is positive, so that an infinite v stays infinite, however
 * small the weight; that of a score of -inf is 0, and 0 times an infinite v is
 * NaN.  Rows that are not visible are not read.
 *   type        of q and out, SS_BF16 or SS_F16: the cache's, or either with
 *               an SS_E4M3 or SS_E2M1 cache.
 *   q, out      row (b, j) at b * seq_stride + j * head_stride (each its own
 *               strides); must not overlap each other or the cache.
 *   lse         device, batch * q_heads floats (natural logarithm), or NULL.
 *   weight_out  device, the layout of ss_kv_pages.weight, or NULL: no weights.
 *               Sequences may share pages (a common prefix) only without
 *               weights: a page's weights are one sequence's.
 *   weight_in   the same layout, or NULL (zeros).  weight_in == weight_out
 *               accumulates in place; a partial overlap is not allowed.
 * Scores, softmax statistics and sums are fp32 (sums of products 128 at a
 * time, each cut below 2^-24 of its sum), exponentials are good to 2^-22, and
 * out is rounded once.  In the sum over v a weight has 16 bits (bf16 caches) or
 * 22 (fp16, e4m3 and e2m1 caches), and up to 2^-38 of the row's largest weight
 * more (fp16); it has 11 bits where q is bf16 and the cache e4m3 with head_dim at
 * most 64 or q_heads more than 8 per key-value head.  lse and the gathered
 * weights are of the fp32 scores.  bf16 queries of an e4m3 or e2m1 cache are held
 * to 2^-32 of their row's largest element.
 * q_heads <= 65536, at most 128 per key-value head, and (max_len / 16 + 1) *
 * q_heads < 2^31.
 */
typedef struct ss_kv_attention {
    ss_elem type;
    int32_t q_heads;
    const void *q;
    int64_t q_seq_stride;
    int64_t q_head_stride;
    void *out;
    int64_t out_seq_stride;
    int64_t out_head_stride;
    float scale;
    int32_t window;
    int32_t sinks;
    float *lse;
    const float *weight_in;
    float *weight_out;
} ss_kv_attention;
ss_status ss_kv_attend(const ss_kv_pages *cache, const ss_kv_table *seqs, const ss_kv_attention *args,
                       ss_stream_t stream);

/*
 * Evicts the least attended tokens: an order-preserving compaction of every
 * (sequence, head) of `src` into the pages of `dst`.  Of a sequence of n
 * positions m = min(n, keep) stay: the first `sinks`, the last `recent`, and
 * of the others those of the largest src weight; equal weights go to the
 * lower position first (-0 equals +0; NaN ranks below -inf).  Kept row i, in
 * the order of positions, goes to position i of the destination: k, v (bit
 * for bit) and, where dst->weight is not NULL, the weight.  Heads choose
 * independently.  A token's weight is 0 from its append to the first attention
 * that keeps weights, and rows of equal weights keep their first positions.
 * dst_seqs->lens receives m; its tables have room for the
 * smaller of keep and src_seqs' max_len.  `dst` has src's type, heads,
 * head_dim and scales (not moved); its page_size and strides are its own,
 * and it may be the same pool.  The destination pages must not be pages that
 * any sequence of src reads; source pages may be shared.
 *   kept  device, batch x kv_heads x keep int32, or NULL: the source position
 *         of each kept row, -1 from m on.
 *   0 <= sinks, 0 <= recent, sinks + recent <= keep, 1 <= keep; max_len <=
 *   2^21, batch * kv_heads <= 2^20.
 */
ss_status ss_kv_evict(const ss_kv_pages *src, const ss_kv_table *src_seqs, const ss_kv_pages *dst,
                      const ss_kv_table *dst_seqs, int32_t keep, int32_t sinks, int32_t recent, int32_t *kept,
                      ss_stream_t stream);

/*
 * Generic scan entry: dtype, inclusive (0/1) and algorithm chosen at run
 * time.  Same argument rules as the named scans.  The reduce-then-scan
 * algorithms ("Prefix sum and other parallel patterns", three passes with
 * scan_block_sums' carry loop; "The CUDA scan algorithm: the tree and the
 * three kernels", Two sweeps over one tree, bank padding of "The stride
 * doubles, and so does the conflict") also take out == in.
 */
ss_status ss_scan(ss_dtype dtype, int inclusive, ss_algo algo, const void *in, void *out,
                  size_t n, ss_stream_t stream);

/*
 * Sum of all n elements of `in`, written to *d_total (device, one element of
 * dtype's type, 4-byte aligned) -- the first step of a scan split over
 * several devices ("Prefix sum and other parallel patterns", A device-level
 * scan: scan then propagate -- the part totals are scanned and each part is
 * offset by the sum of the parts before it).  int32 and uint32 wrap modulo
 * 2^32; fp32 adds in an order that is fixed for a fixed n and device (so the
 * same input gives the same bits on every run).  n == 0 writes 0.  in is
 * 4-byte aligned (16-byte aligned takes the vector path); *d_total must not
 * overlap in.  One launch; uses the stream's workspace.
 */
ss_status ss_reduce_sum(ss_dtype dtype, const void *in, void *d_total, size_t n, ss_stream_t stream);

/*
 * Single-pass scan seeded with a carry: the prefix before in[0] is
 * *d_carry_in (device, one element of the scan's type; NULL means 0), and
 * the inclusive total including the seed is written to *d_carry_out (device,
 * NULL to skip).  Scanning an array in consecutive chunks with the carry
 * passed along gives the scan of the whole array; this is the offset step of
 * a scan split over several calls or several devices (scan each part, scan
 * the parts' totals, seed each part with its offset).  d_carry_out may
 * equal d_carry_in.
 */
ss_status ss_scan_seeded(ss_dtype dtype, int inclusive, const void *in, void *out, size_t n,
                         const void *d_carry_in, void *d_carry_out, ss_stream_t stream);

/*
 * Host-memory scan: h_in and h_out are HOST pointers.  Returns when h_out
 * holds the result (device errors are reported directly).  h_out == h_in is
 * allowed.  Two paths:
 *   - both buffers pinned and mapped into the device address space (for
 *     example from cudaHostAlloc): the scan kernel reads h_in and writes
 *     h_out directly, over NVLink-C2C on a Grace host, with no staging
 *     copies.  It uses the one-CTA-per-tile kernel, whose accesses are plain
 *     16-byte loads and stores;
 *   - otherwise (pageable memory, or ss_set_host_mode(1)): the input is
 *     copied to the device in chunks, each chunk is scanned seeded with the
 *     running carry, and the results are copied back, the copies of one chunk
 *     overlapping the scan of another.
 */
ss_status ss_scan_host(ss_dtype dtype, int inclusive, const void *h_in, void *h_out, size_t n,
                       ss_stream_t stream);

/* Path of ss_scan_host: 0 (default) = direct access when both buffers are
 * mapped pinned memory, else staged; 1 = always staged.  Process-wide. */
ss_status ss_set_host_mode(int mode);

/*
 * Bandwidth probe: copies n uint32 from in to out with the scan's loader and
 * storer and no arithmetic ("The CUDA scan algorithm: the tree and the three
 * kernels", Results: "copy, no scan" as the speed-of-light row).
 */
ss_status ss_copy_u32(const uint32_t *in, uint32_t *out, size_t n, ss_stream_t stream);

/*
 * Diagnostic: the exclusive uint32 (= int32 bits) single-pass scan under
 * tile configuration `config`, recording a timing trace of every tile's
 * look-back ("Prefix sum and other parallel patterns", A device-level scan:
 * how long a tile waits on what earlier tiles published).  d_trace (device,
 * 8-byte aligned) receives 8 uint64 per tile of that configuration
 * (ss_scan_tile_elems() after ss_set_scan_config(config)):
 *   [0] %globaltimer (ns) when the CTA began the tile  [1] aggregate known
 *   [2] aggregate published   [3] look-back resolved   [4] outputs issued
 *   [5] descriptor windows read   [6] polls that found an unpublished tile
 *   [7] SM id (low 32 bits) | CTA index << 32
 * Every row has a traced build (rows 10-12, with the two-level look-back,
 * record [5] = 1).  A persistent row needs 16-byte aligned in/out and n
 * above one tile.  The scan result is the same as scan_exclusive_u32's.
 */
ss_status ss_scan_trace(int config, const uint32_t *in, uint32_t *out, size_t n, uint64_t *d_trace,
                        ss_stream_t stream);

/*
 * Waits for `stream`, then returns and clears the device-side status of
 * that stream's workspace: SS_OK, SS_ERR_LOOKBACK_TIMEOUT, or SS_ERR_CUDA if
 * the stream itself failed.  *failing_tile (may be NULL) receives the first
 * tile that gave up, or -1.
 */
ss_status ss_stream_status(ss_stream_t stream, int64_t *failing_tile);

/* Static description of a status code. */
const char *ss_status_string(ss_status status);

/* Detail of the last error returned on the calling thread ("" if none). */
const char *ss_last_error_detail(void);

/* Elements per tile of the single-pass scan under the current tile
 * configuration (under the automatic choice, of the row used for large n),
 * and the number of configurations that can be selected. */
size_t ss_scan_tile_elems(void);
int ss_scan_config_count(void);

/* Selects the single-pass scan's tile configuration for later calls in this
 * process (ss_scan_config_count() rows: one CTA per tile, or a persistent
 * grid streaming tiles through a shared-memory ring).  -1 (the initial
 * setting) chooses per call by size: row 7 (16384-element tiles) from 2e6
 * to 5e7 elements, row 8 (18432-element tiles, each claimed from the tile
 * counter as its copy starts, so that faster SMs take more tiles) below and
 * above.
 * Results do not depend on it, except for the rounding of fp32 sums.
 * SS_ERR_INVALID_ARG below -1 or from ss_scan_config_count() on. */
ss_status ss_set_scan_config(int config);

/* Selects the persistent compaction kernel used for 16-byte aligned inputs
 * above 16384 elements (flag form), for later calls in this process:
 *   0  streams keys and flags through shared memory with bulk copies;
 *   1  bulk-copies only the flags and loads a 16-byte key vector only where
 *      one of its four flags is set, which reads far fewer key bytes when
 *      few elements are kept; one look-back per 16384 elements;
 *   2  (the default) as 1, with one look-back per tile of four chunks: two
 *      256-thread CTAs per SM and 32768-element tiles, which pays a tile's
 *      fixed costs once per 32768 elements (inputs of 32768 elements or
 *      fewer take 1).  A tile keeping fewer than 1728 keys is written in a
 *      sparse form: each thread loads only its kept keys, one by one, before
 *      the tile's look-back; other tiles gather each warp's kept keys in
 *      shared memory and write 16-byte vectors;
 *   3  as 2 with every tile in the dense form, 4 with every tile in the
 *      sparse form;
 *   5, 6, 7  as 2, 3, 4 with one 512-thread CTA per SM and 65536-element
 *      tiles (sparse below 3456 keys).
 * Results are identical. */
ss_status ss_set_compact_config(int config);

/* Selects the form of later ss_scan_segments calls in this process:
 *   0  (the default) blocked, by mean segment length n / num_segments: 64
 *      threads a CTA below 2048, 128 from there and for num_segments = 0;
 *   1  row-striped: lane l of a warp holds 16-byte vectors l, l + 32, ... of
 *      the warp's span, one 512-thread CTA per SM, 16384-element tiles;
 *   2, 3, 4, 5  blocked: each thread owns 32 consecutive elements (one
 *      tile row), with 256, 128, 512 or 64 threads a CTA, 512 / threads CTAs
 *      per SM and tiles of 32 x threads elements.
 * Integer results are identical; fp32 sums are added in another order and
 * agree within the bound of the flat scans.  SS_ERR_INVALID_ARG for any
 * other value. */
ss_status ss_set_segments_config(int config);

/* Frees every workspace the library allocated (all devices and streams).
 * No call may be in flight. */
void ss_shutdown(void);

/*
 * Test hook for the failure path of the look-back wait.  With tile >= 0,
 * later single-pass calls in this process skip publishing that tile's
 * descriptor, so its successors' waits run out after timeout_ns (their
 * status then reads SS_ERR_LOOKBACK_TIMEOUT).  tile = -1 restores normal
 * operation and timeout_ns = 0 restores the default limit (2 s).  No wait is
 * ever unbounded: every wait also stops after a fixed number of polls.
 */
ss_status ss_debug_set_lookback_fault(int64_t tile, uint64_t timeout_ns);

/*
 * Single-pass scan that allocates nothing.  The pages have no counterpart:
 * it exists for callers that cannot call cudaMalloc -- an application that
 * serves all device memory from its own pool and forbids other allocations
 * to keep its accounting exact, or a latency-critical loop that may never
 * pay for an allocation.  The regular entry points allocate a per-stream
 * workspace on first use; this one keeps its scratch (tile counter, status
 * words, tile descriptors) in a fixed device array of 2 MiB + 256 bytes that
 * every GPU loading the library holds until the process exits.
 *   dtype, inclusive, in, out, stream: as for ss_scan (SS_ALGO_LOOKBACK);
 *        out == in is allowed.  The caller passes inputs and outputs.
 *        `stream` must belong to the current device (the array used is the
 *        current device's); a stream of another device returns
 *        SS_ERR_INVALID_ARG.
 *   n    0 <= n <= 2^30; larger n returns SS_ERR_INVALID_ARG.
 * The first call on a device sets up that device: it looks up the array's
 * device address and zeroes it, which synchronises the device; make that
 * first call before any stream capture.  Every call on a device shares the
 * array and keeps the previous call's contents; no per-call clearing is
 * needed (descriptors carry a launch epoch and the tile counter returns to
 * zero at the end of each launch).  Calls that overlap on the GPU race on
 * the shared array: serialise them (one stream, or events).  The returned
 * status is the only error report: device-side look-back timeouts are not
 * read back by this entry point, nor reported by ss_stream_status().
 */
ss_status ss_scan_noalloc(ss_dtype dtype, int inclusive, const void *in, void *out, size_t n,
                          ss_stream_t stream);

/*
 * Explicit-workspace form, in CUB's two-call shape ("Prefix sum and other
 * parallel patterns", Stream compaction: the library call that first asks
 * for its temporary storage size, then runs with the caller's buffer).
 *
 * ss_scan_temp_bytes: *bytes receives the device scratch, in bytes, that a
 *   scan of n elements needs: a 256-byte header (the tile counter and the
 *   status words) and 8 bytes per 4096 elements and per 32 tiles of them
 *   (the tile descriptors); 0 for n = 0.  Host only; enqueues nothing.
 *
 * ss_scan_ws: the scan of scan_{inclusive,exclusive}_* (dtype SS_I32,
 *   SS_U32 or SS_F32; the same kernels and the same automatic choice by n)
 *   with `temp` as its scratch instead of the library's per-stream
 *   workspace, so the call allocates nothing.
 *   temp        device memory of the stream's device, 256-byte aligned, at
 *               least ss_scan_temp_bytes(n) bytes (temp_bytes), owned by the
 *               caller and not overlapping in or out.  Its contents on entry
 *               do not matter: the call clears the part it uses with one
 *               memset on `stream` before its launch.
 *   in, out, n, stream: as for the scans above; out == in is allowed.
 *   Calls sharing one temp must not overlap on the GPU.  Device-side
 *   timeouts are recorded in temp's header: ss_temp_status reads them.
 *
 * ss_temp_status: waits for `stream`, then returns and clears the device
 *   status held in `temp` (the values of ss_stream_status); *failing_tile
 *   (may be NULL) receives the first tile that gave up, or -1.
 */
ss_status ss_scan_temp_bytes(size_t n, size_t *bytes);
ss_status ss_scan_ws(ss_dtype dtype, int inclusive, const void *in, void *out, size_t n, void *temp,
                     size_t temp_bytes, ss_stream_t stream);
ss_status ss_temp_status(void *temp, ss_stream_t stream, int64_t *failing_tile);

/*
 * Test hooks for ss_scan_noalloc's periodic descriptor clear: the clear runs
 * on the current device's call that makes the count of calls a multiple of
 * ss_debug_noalloc_clear_period() (2^29), before its launch.
 * ss_debug_set_noalloc_calls sets the count of calls made so far on the
 * current device, so that a test reaches a clear in a few calls.
 */
ss_status ss_debug_set_noalloc_calls(uint64_t calls);
uint64_t ss_debug_noalloc_clear_period(void);

#ifdef __cplusplus
}
#endif

#endif /* STREAMSCAN_H */
