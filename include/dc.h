/*
 * dc.h -- C ABI of libdc: the data-parallel core of a deterministic
 * collective on one GPU, with the world's P ranks held as P buffers in the
 * GPU's own memory.
 *
 * Pages cited by title:
 *   [PR491] "perf(cuda): vectorize the deterministic all-gather copy and
 *           right-size its single-block path" (RL-Kernel pull request 491).
 *
 * Conventions for every entry point:
 *   - Pointers named *_ptrs / outs / bytes_per_rank are HOST arrays that the
 *     call reads before it returns; the pointers stored in them are DEVICE
 *     addresses of the current device (cudaMalloc, torch CUDA tensors, or
 *     managed memory).  The caller owns all memory.
 *   - The work is enqueued on `stream` (NULL = the legacy default stream) and
 *     runs asynchronously.  A call allocates no memory, never synchronises,
 *     launches at most one kernel (or as many as its description says), and copies every pointer and size into the
 *     kernel's parameters, so it may be captured into a CUDA graph and the
 *     host arrays may be freed as soon as it returns.
 *   - Arguments are checked before any CUDA call; a rejected call launches
 *     nothing and returns a status with a message in dc_last_error().  A
 *     launch failure returns DC_ERR_CUDA.  Faults inside the kernel surface at
 *     the caller's next synchronisation, as for any CUDA kernel.
 *   - A call whose size is zero succeeds without launching anything (after P
 *     has been checked).
 *   - Results never depend on the path, grid size or stream timing: the
 *     gathers are exact byte copies and the reductions use one fixed
 *     per-element order.
 *   - Calls are thread-safe; options (dc_set_option) are process-wide.
 */
#ifndef DC_H
#define DC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st *dc_stream_t;

typedef enum {
    DC_OK = 0,
    DC_ERR_INVALID = 1,  /* bad count, null pointer, size overflow */
    DC_ERR_ALIGN = 2,    /* a BF16 pointer that is not 2-byte aligned */
    DC_ERR_OVERLAP = 3,  /* an output range overlaps an input or another output */
    DC_ERR_TOO_MANY = 4, /* all_gather_many table larger than the limits below */
    DC_ERR_CUDA = 5,     /* the CUDA runtime refused the launch */
    DC_ERR_TIMEOUT = 6,  /* a bounded device wait ran out (reported by dc_check_device) */
    DC_ERR_BOUNDS = 7    /* bounds-checked build only: a kernel skipped an access outside its
                            job's range (reported by dc_check_device) */
} dc_status_t;

/* Element types and summation orders of the reductions. */
typedef enum { DC_BF16 = 0, DC_F16 = 1, DC_F32 = 2 } dc_dtype_t;
typedef enum { DC_ORDER_LINEAR = 0, DC_ORDER_TREE = 1 } dc_order_t;

#define DC_MAX_RANKS 64          /* P <= 64 */
#define DC_MANY_MAX_TENSORS 256  /* all_gather_many: T <= 256 */
#define DC_MANY_MAX_SEGMENTS 1024 /* all_gather_many: T * P <= 1024 */
#define DC_MANY_MAX_REDUCE_JOBS 256  /* reductions: T (all_reduce) or T * P (reduce_scatter) <= 256 */
#define DC_MANY_MAX_REDUCE_PTRS 1024 /* reductions: 2 * T * P <= 1024 */

/*
 * dc_all_gather -- rank-ordered all-gather ([PR491] section "What",
 * copy_rank_ordered bullet; the Python API there is all_gather(input, out=)).
 *
 *   out[r*bytes_per_rank + j] = peer_ptrs[r][j]   for r < P, j < bytes_per_rank.
 *
 * peer_ptrs: host array of P device pointers, each to bytes_per_rank bytes
 *            (any alignment; peers may overlap or repeat each other).
 * P:         1..DC_MAX_RANKS.
 * out:       device pointer to P*bytes_per_rank bytes, any alignment; it must
 *            not overlap any peer range (DC_ERR_OVERLAP).
 * Bytes outside [out, out + P*bytes_per_rank) are never written.
 * Path: the 16-byte flat vector copy when out, bytes_per_rank and every peer
 * are 16-byte aligned (staged through shared memory with cp.async, or, with
 * the gather_bulk option, bulk copies on the TMA engine); the realigning copy
 * otherwise (across the lanes of a warp, or through a shared-memory ring);
 * one CTA below the measured single-block threshold (output bytes), a grid
 * sized from the 16-byte vector count and the SM count above it.
 */
dc_status_t dc_all_gather(const void *const *peer_ptrs, int P, size_t bytes_per_rank,
                          void *out, dc_stream_t stream);

/*
 * dc_all_gather_many -- T independent all-gathers in one launch, each into
 * its own output, with no packing ([PR491] results paragraph and the
 * author's reply on all_gather_many: several gathers, one handshake, no
 * packing).
 *
 * peer_ptrs:      host array of T*P device pointers, tensor-major:
 *                 peer_ptrs[t*P + r] is rank r's payload of tensor t.
 * bytes_per_rank: host array of T sizes (zero allowed).
 * outs:           host array of T device pointers; outs[t] receives
 *                 P*bytes_per_rank[t] bytes in rank order.  Outputs must not
 *                 overlap each other or any payload.
 * T:              0..DC_MANY_MAX_TENSORS, and T*P <= DC_MANY_MAX_SEGMENTS
 *                 (DC_ERR_TOO_MANY otherwise).
 */
dc_status_t dc_all_gather_many(const void *const *peer_ptrs, const size_t *bytes_per_rank,
                               void *const *outs, int T, int P, dc_stream_t stream);

/*
 * dc_all_reduce_bf16 -- deterministic all_reduce of P BF16 buffers
 * ([PR491] sections "What" and "Not in this PR"; the page does not print the
 * arithmetic, and this is the reading used): for every i < count,
 *
 *   acc = f32(in_ptrs[0][i]);  acc = acc + f32(in_ptrs[q][i]) for q = 1..P-1
 *   (binary32, round to nearest even, in that order);
 *   out_ptrs[r][i] = bf16_round_nearest_even(acc) for every r < P.
 *
 * in_ptrs, out_ptrs: host arrays of P device pointers to `count` BF16
 *            elements each, 2-byte aligned (DC_ERR_ALIGN).  out_ptrs[r] may
 *            be exactly equal to an input pointer (in place); any other
 *            overlap between outputs and inputs, or between outputs, is
 *            DC_ERR_OVERLAP.  Inputs may overlap each other.
 * Subnormals are kept; NaN inputs give a NaN (payload unspecified).
 */
dc_status_t dc_all_reduce_bf16(const void *const *in_ptrs, void *const *out_ptrs, int P,
                               size_t count, dc_stream_t stream);

/*
 * dc_reduce_scatter_bf16 -- deterministic reduce_scatter: input = world x
 * output, as the author's reply on [PR491] describes it.  Each input holds
 * P*count_per_shard BF16 elements; rank r receives shard r:
 *
 *   out_ptrs[r][j] = fold over q = 0..P-1 of in_ptrs[q][r*count_per_shard + j]
 *
 * with the fold of dc_all_reduce_bf16.  out_ptrs[r] may be exactly
 * in_ptrs[q] + r*count_per_shard for some q (in place); other overlaps are
 * DC_ERR_OVERLAP.  Pointers must be 2-byte aligned.
 */
dc_status_t dc_reduce_scatter_bf16(const void *const *in_ptrs, void *const *out_ptrs, int P,
                                   size_t count_per_shard, dc_stream_t stream);

/*
 * dc_all_reduce / dc_reduce_scatter -- the same operations for any element
 * type and either summation order.  Every element is widened exactly to
 * binary32, the P values of an element are added one binary32 add (round to
 * nearest even) at a time in `order`, and the total is rounded once to
 * `dtype` (round to nearest even; DC_F32 totals are stored as they are):
 *   DC_ORDER_LINEAR: ((x0 + x1) + x2) + ... + x_{P-1};
 *   DC_ORDER_TREE:   fold(x[lo..hi)) = fold(x[lo..lo+m)) + fold(x[lo+m..hi)),
 *                    m the largest power of two below hi - lo.
 * [PR491] names a fixed-tree backend ("cuda_ipc_fixed_tree", author's
 * replies) without its shape; DC_ORDER_TREE is the plainest reading, and
 * DC_ORDER_LINEAR the default of the BF16 entry points above.  Pointers must
 * be aligned to the element size (2 or 4 bytes); aliasing rules as above.
 * Speed, not results, depends on alignment: the work runs in 16-byte units
 * anchored at the outputs when all outputs sit at the same address mod 16
 * (inputs at another offset are realigned, at about half the bandwidth), and
 * element by element otherwise.
 */
dc_status_t dc_all_reduce(const void *const *in_ptrs, void *const *out_ptrs, int P, size_t count,
                          dc_dtype_t dtype, dc_order_t order, dc_stream_t stream);
dc_status_t dc_reduce_scatter(const void *const *in_ptrs, void *const *out_ptrs, int P,
                              size_t count_per_shard, dc_dtype_t dtype, dc_order_t order,
                              dc_stream_t stream);

/*
 * dc_reduce -- one rank's share of a reduction: the P inputs folded into ONE
 * output, as dc_all_reduce / dc_reduce_scatter fold them:
 *
 *   out[i] = round(fold over q = 0..P-1 of in_ptrs[q][in_offset + i]),  i < count
 *
 * When every rank is its own process ([PR491] author's replies: the
 * collective's ranks exchange payloads through buffers their peers map),
 * rank r computes only its own output: its all_reduce output (in_offset 0,
 * count = elements per rank) or its reduce_scatter shard (in_offset =
 * r * count_per_shard, count = count_per_shard), from the P mapped buffers.
 * The result is bit-identical to the same rank's output of dc_all_reduce /
 * dc_reduce_scatter.
 *
 * in_ptrs: host array of P device pointers (read during the call), each to
 *          at least in_offset + count elements; aligned to the element size
 *          (DC_ERR_ALIGN).  Inputs may overlap each other.
 * out:     device pointer to count elements, aligned to the element size.
 *          It may be exactly the range of one input that is read (in_ptrs[q]
 *          + in_offset elements: in place); any other overlap with the
 *          elements read is DC_ERR_OVERLAP.
 * count:   0 is a successful no-op.  in_offset + count must not overflow
 *          (DC_ERR_INVALID).
 * One kernel on `stream`; nothing allocated, no synchronisation.
 */
dc_status_t dc_reduce(const void *const *in_ptrs, int P, size_t in_offset, size_t count, void *out,
                      dc_dtype_t dtype, dc_order_t order, dc_stream_t stream);

/*
 * dc_all_reduce_many / dc_reduce_scatter_many -- T independent reductions of
 * the same P, type and order in one launch ([PR491] "Tests":
 * reduce_scatter_many(..., outs=) with caller-given outputs).
 * in_ptrs, out_ptrs: host arrays of T*P device pointers, tensor-major
 *                    (tensor t, rank r at index t*P + r).
 * counts / counts_per_shard: host array of T element counts (zero allowed).
 * Limits: DC_MANY_MAX_REDUCE_JOBS jobs (T for all_reduce, T*P for
 * reduce_scatter) and 2*T*P <= DC_MANY_MAX_REDUCE_PTRS (DC_ERR_TOO_MANY).
 * Outputs may alias only their own tensor's inputs, as in the single forms.
 */
dc_status_t dc_all_reduce_many(const void *const *in_ptrs, void *const *out_ptrs,
                               const size_t *counts, int T, int P, dc_dtype_t dtype,
                               dc_order_t order, dc_stream_t stream);
dc_status_t dc_reduce_scatter_many(const void *const *in_ptrs, void *const *out_ptrs,
                                   const size_t *counts_per_shard, int T, int P, dc_dtype_t dtype,
                                   dc_order_t order, dc_stream_t stream);

/*
 * dc_inject_delay_ns -- keeps one GPU thread busy for `ns` nanoseconds of
 * the GPU's global timer, in stream order.  The rank-skew calibration
 * ("[Benchmark] Add all-reduce rank-skew calibration", vLLM pull request
 * 57037, section "Purpose") puts it on one simulated rank's stream before
 * that rank arrives at the collective.
 *
 * ns:     0..DC_MAX_DELAY_NS (DC_ERR_INVALID above); 0 launches a kernel
 *         that returns at once.
 * stream: the stream to delay.
 * The kernel reads no memory and writes none.  It stops when the timer has
 * advanced by ns, or, should the timer stall, after 4*ns + 2^20 SM cycles.
 * The requested delay is a lower bound on the kernel's duration; time it
 * with events to get the measured delay.
 */
#define DC_MAX_DELAY_NS 1000000000ull
dc_status_t dc_inject_delay_ns(unsigned long long ns, dc_stream_t stream);

/*
 * dc_fused_all_gather -- the staged all-gather protocol of the collective's
 * multi-rank deployment ([PR491] author's replies: the cuda_ipc_fixed_tree
 * backend's CUDA-graph-safe fused protocol, stage -> gather -> complete;
 * section "Not in this PR" and the review threads: a failed launch leaves the
 * protocol pending with no abort path, and peers of a dead rank wait for the
 * process-group timeout), run with the P ranks as CTA groups of one
 * cooperative launch on one GPU, every wait bounded.
 *
 * Rank r stages in_ptrs[r] into staging[r], publishes it, gathers every
 * rank's staging buffer into outs[r] in rank order, and completes once every
 * rank has read its staging buffer.  Afterwards, for every r:
 *
 *   outs[r][q*bytes_per_rank + j] = in_ptrs[q][j]   (q < P, j < bytes_per_rank)
 *
 * and staging[r] holds a copy of in_ptrs[r].
 *
 * in_ptrs, staging, outs: host arrays of P device pointers (16-byte aligned);
 *            each input and staging buffer holds bytes_per_rank bytes, each
 *            output P*bytes_per_rank.  Staging buffers, outputs and the
 *            workspace may overlap nothing; inputs may overlap inputs.
 * bytes_per_rank: a multiple of 16 (DC_ERR_ALIGN otherwise); 0 is a no-op.
 * workspace: device memory of dc_fused_workspace_bytes(P) bytes, 16-byte
 *            aligned, owned by the caller and zero before its first use
 *            (cudaMemset, or dc_fused_reset).  It holds the ranks' epoch flags.
 * epoch:     1 for the first call after the workspace was cleared, then one
 *            more for each call (never 0).  Calls on one workspace must not
 *            overlap on the GPU: issue them on one stream.
 * Every wait for a peer's flag is bounded by the "wait_limit_ns" option.  If
 * one runs out (a rank that never arrives), the waiting CTAs record the fault
 * and return, the outputs are incomplete, and dc_check_device returns
 * DC_ERR_TIMEOUT naming the waiting and the awaited rank; clear the workspace
 * with dc_fused_reset and start again at epoch 1.  P ranks need P*G CTAs
 * resident at once (G chunks per rank, at least one): DC_ERR_INVALID if the
 * GPU cannot hold P of them.
 */
size_t dc_fused_workspace_bytes(int P); /* 0 if P is outside 1..DC_MAX_RANKS */
dc_status_t dc_fused_all_gather(const void *const *in_ptrs, void *const *staging, void *const *outs, int P,
                                size_t bytes_per_rank, void *workspace, unsigned int epoch,
                                dc_stream_t stream);
/* Clears a fused workspace of P ranks on `stream` (cudaMemsetAsync); the next
 * call on it uses epoch 1. */
dc_status_t dc_fused_reset(void *workspace, int P, dc_stream_t stream);

/*
 * dc_fused_all_gather_static -- dc_fused_all_gather for callers that cannot
 * allocate device memory.  The pages describe no such entry point: it is this
 * library's own addition.  Some callers are given only their input and output
 * buffers and may not call cudaMalloc themselves: a plug-in run by a host
 * framework that owns every device allocation, code whose device memory was
 * planned once up front, or code that must not call cudaMalloc/cudaFree
 * because those can synchronise the device.  This form needs no workspace and
 * no staging buffers from them.
 *
 * It computes what dc_fused_all_gather computes (outs[r] = in_ptrs[0] ||
 * in_ptrs[1] || ... for every r; same argument rules for in_ptrs, outs, P and
 * bytes_per_rank), with the epoch flags and the P staging buffers in one
 * static device array of the library: 16 MiB of staging after 64 KiB of
 * flags, held by every GPU that loads the library until the process exits.
 * Limit: P * (bytes_per_rank rounded up to 256) <= 16 MiB; a larger call is
 * rejected with DC_ERR_INVALID before anything is launched.
 *
 * It allocates nothing: no cudaMalloc, no cudaFree, no allocating library
 * routine.  Each call enqueues on `stream` a clear of the flags
 * (cudaMemsetAsync, 64 KiB at most) and one kernel.  The first call made with
 * a device current looks up the array's device address on that device
 * (cudaGetSymbolAddress); make that first call before any stream capture.
 * Every call in the process uses the same array on a given GPU, which keeps
 * the last call's contents: calls whose work overlaps on the GPU (issued on
 * different streams, or from different host threads) race and corrupt each
 * other's results; issue them on one stream.  Waits are bounded as in
 * dc_fused_all_gather and reported by dc_check_device.
 */
dc_status_t dc_fused_all_gather_static(const void *const *in_ptrs, void *const *outs, int P,
                                       size_t bytes_per_rank, dc_stream_t stream);

/*
 * Operators of language models beside the collectives, for reproducible
 * rollouts and training on them: log probabilities over the vocabulary shards
 * of a tensor-parallel head (with their gradient), and the paged key-value
 * cache with the attention of single new tokens over it.  They follow the
 * conventions above (one kernel a call where nothing else is said, no
 * allocation, checks first), and
 * their results depend on no other row or sequence of the call, on no grid
 * and, for the log probabilities, on no sharding: a token has the same bits
 * in a batch of one and in a batch of a thousand.
 *
 * Each takes a block of arguments by address, read before the call returns.
 * Strides count elements.  Sums, maxima and statistics are binary32.
 */

/*
 * dc_token_logprobs -- for each row of logits x and its token y, with
 * z = x / temperature over columns [0, vocab) of the concatenated shards:
 *
 *   lse = log(sum_i exp(z_i));  logprobs = z_y - lse;
 *   entropy = lse - sum_i p_i z_i,  p = exp(z - lse);
 *   top_tokens, top_logprobs = the `top` largest columns by x (equal logits:
 *   lowest index first) and their log probabilities.
 *
 * shards, widths, row_strides: host arrays of `ranks` entries: rank r holds
 *   `widths[r]` columns, row i at shards[r] + i * row_strides[r].  Shards may
 *   be uneven, empty, or column ranges of one tensor; any alignment of the
 *   element type.  Columns past `vocab` (padding) are not read.
 * temperature: 4.24e-39 (so that log2(e) / temperature fits binary32) to 1e30.
 * tokens: int32 or int64 (tokens_64).  A negative token asks for nothing:
 *   its log probability is 0.  A token of vocab or more gives NaN.
 * logprobs [rows]; entropy, lse [rows] and top_logprobs, top_tokens
 *   [rows, top], all contiguous, NULL where not wanted.  top: 0..DC_MAX_TOP.
 * Masked logits (-inf) have probability 0.  A row of nothing else has
 * lse = -inf, log probabilities -inf and entropy 0.  A row with NaN or +inf
 * gives NaN; NaN logits are never among the alternatives, and places that no
 * number fills hold token -1 and NaN.
 */
#define DC_MAX_TOP 32
#define DC_MAX_VOCAB (1 << 22)
typedef struct {
    const void *const *shards;
    const uint64_t *widths;
    const uint64_t *row_strides;
    const void *tokens;
    float *logprobs;
    float *entropy;
    float *lse;
    float *top_logprobs;
    void *top_tokens;
    int64_t rows;
    int64_t vocab;
    double temperature;
    int32_t ranks;
    int32_t dtype;          /* dc_dtype_t of the logits */
    int32_t tokens_64;
    int32_t top_tokens_64;
    int32_t top;
    int32_t reserved;       /* 0 */
} dc_token_logprobs_t;
dc_status_t dc_token_logprobs(const dc_token_logprobs_t *args, dc_stream_t stream);

/*
 * dc_token_logprobs_backward -- the gradient of sum(g * logprobs + h *
 * entropy) with respect to the logits, from the lse and entropy that
 * dc_token_logprobs returned:
 *
 *   grads_i = (1/temperature) (g ([i = y] - p_i) - h p_i (log p_i + entropy))
 *
 * g = grad_logprobs and h = grad_entropy [rows], either NULL (zero); h needs
 * `entropy`.  A negative token's g counts as 0.  grads[r] has widths[r]
 * columns; padding columns receive 0, as do rows whose lse is -1e30 or less:
 * rows of nothing but -inf, or but the lowest value of DC_BF16 or DC_F32, whose
 * lse cannot hold the log of how many they are.  A row of nothing but DC_F16's
 * lowest value (-65504) is a row like others, with the gradient of its uniform
 * probabilities.  log p_i = z_i - lse is good to 2^-24 |lse|, the rounding of
 * lse, and p_i with it.
 * grads[r] may be exactly shards[r] (in place); any other overlap is refused.
 */
typedef struct {
    const void *const *shards;
    const uint64_t *widths;
    const uint64_t *row_strides;
    void *const *grads;
    const uint64_t *grad_row_strides;
    const void *tokens;
    const float *lse;
    const float *entropy;
    const float *grad_logprobs;
    const float *grad_entropy;
    int64_t rows;
    int64_t vocab;
    double temperature;
    int32_t ranks;
    int32_t dtype;
    int32_t tokens_64;
    int32_t reserved;       /* 0 */
} dc_token_logprobs_backward_t;
dc_status_t dc_token_logprobs_backward(const dc_token_logprobs_backward_t *args, dc_stream_t stream);

/*
 * dc_linear_logprobs -- dc_token_logprobs from the rows that a linear head
 * takes, without keeping the logits: with x = hidden W^T, W the concatenated
 * shards (one row per column of the vocabulary), and z = x / temperature,
 *
 *   lse = log(sum_i exp(z_i));  logprobs = z_y - lse;
 *   entropy = lse - sum_i p_i z_i,  p = exp(z - lse).
 *
 * hidden [rows, hidden_size]; weights[r] [widths[r], hidden_size]; DC_BF16 or
 *   DC_F16, rows 16-byte aligned, hidden_size a multiple of 8 up to 2^20.
 *   The products are exact and their sums binary32, as are all statistics.
 * ranks, widths, vocab, temperature, tokens: as for dc_token_logprobs (rows of
 *   the weights past `vocab` are not read), and so are rows of nothing but -inf
 *   and rows with NaN or +inf.  Up to 2^24 rows.
 * logprobs [rows]; entropy, lse [rows] or NULL.
 * A row's bits do not depend on the other rows, and not on the shards where
 * every shard but the last is a multiple of 256 wide.
 *
 * workspace: device memory of at least dc_linear_logprobs_workspace_bytes(rows,
 * hidden_size, columns, 0) bytes (columns: all shards' rows), 256-byte aligned,
 * whose contents do not matter; calls that overlap on the GPU need one each.
 * Two kernels.  The waits inside are bounded ("wait_limit_ns"): one that ran
 * out leaves wrong results, which dc_check_device reports.
 */
typedef struct {
    const void *hidden;
    const void *const *weights;
    const uint64_t *widths;
    const uint64_t *weight_row_strides;
    const void *tokens;
    float *logprobs;
    float *entropy;
    float *lse;
    void *workspace;
    uint64_t workspace_bytes;
    uint64_t hidden_row_stride;
    int64_t rows;
    int64_t hidden_size;
    int64_t vocab;
    double temperature;
    int32_t ranks;
    int32_t dtype;
    int32_t tokens_64;
    int32_t reserved;       /* 0 */
} dc_linear_logprobs_t;
dc_status_t dc_linear_logprobs(const dc_linear_logprobs_t *args, dc_stream_t stream);
/* 0 if the arguments are not supported. */
size_t dc_linear_logprobs_workspace_bytes(int64_t rows, int64_t hidden_size, int64_t columns, int backward);

/*
 * dc_linear_logprobs_backward -- the gradient of sum(g * logprobs + h *
 * entropy) with respect to hidden and the weights, from the lse and entropy
 * that dc_linear_logprobs returned.  With d the logits' gradient (that of
 * dc_token_logprobs_backward, where g, h and `entropy` are described),
 *
 *   grad_hidden = d W;   grad_weights[r] = (d^T hidden) of the shard's columns.
 *
 * The logits are computed again, up to 24576 columns of a shard at a time; d is
 * rounded to 16 bits before its products (for DC_F16 times one power of two for
 * all rows, so that the largest d that these g and h allow fits: rows whose g
 * and h are 2^20 times smaller than the largest lose precision); what that takes
 * from d at the row's token is kept in binary32 and added to both products.  The
 * sums are binary32 and rounded once.
 *
 * grad_hidden [rows, hidden_size] or NULL; grad_weights: host array of
 *   `ranks` pointers, shaped as the weights, or NULL; either is needed.  They
 *   replace what was there.  Rows of the weights' gradient past `vocab` are 0,
 *   as are all of them if there are no rows.  No output may meet an input.
 * A row whose token is vocab or more has NaN for one, as there; one whose lse is
 * -1e30 or less, or whose g and h are 0, has no gradient (its
 * hidden row still has to be finite where grad_weights are wanted: 0 times NaN is
 * NaN there).  A row of grad_hidden does not depend on the other rows (for DC_F16:
 * beyond the power of two).  The order of every sum is fixed; that of
 * grad_hidden's follows from the shards, so that one shard and eight give other
 * bits, within the roundings above.
 * workspace: dc_linear_logprobs_workspace_bytes(rows, hidden_size, columns, 1)
 * bytes, as above.  Several kernels.
 */
typedef struct {
    const void *hidden;
    const void *const *weights;
    const uint64_t *widths;
    const uint64_t *weight_row_strides;
    const void *tokens;
    const float *lse;
    const float *entropy;
    const float *grad_logprobs;
    const float *grad_entropy;
    void *grad_hidden;
    void *const *grad_weights;
    const uint64_t *grad_weight_row_strides;
    void *workspace;
    uint64_t workspace_bytes;
    uint64_t hidden_row_stride;
    uint64_t grad_hidden_row_stride;
    int64_t rows;
    int64_t hidden_size;
    int64_t vocab;
    double temperature;
    int32_t ranks;
    int32_t dtype;
    int32_t tokens_64;
    int32_t reserved;       /* 0 */
} dc_linear_logprobs_backward_t;
dc_status_t dc_linear_logprobs_backward(const dc_linear_logprobs_backward_t *args, dc_stream_t stream);

/* One of the two tensors of a paged cache: element d of head h of token o of
 * page g is data[g*page_stride + o*token_stride + h*head_stride + d], every
 * head 16-byte aligned. */
typedef struct {
    void *data;
    uint64_t page_stride;
    uint64_t token_stride;
    uint64_t head_stride;
} dc_paged_cache_t;

/*
 * dc_kv_append -- puts the keys and values of `tokens` new tokens into a paged
 * cache and rotates keys (and queries, q -> q_out) to their positions.  Token
 * i of sequence s = seqs[i] at position t = positions[i] goes to slot
 * t % page_size of page page_table[s * table_stride + t / page_size].
 *
 * Rotation: of the first rotary_dim elements of a head, pair (j, j +
 * rotary_dim/2), or (2j, 2j + 1) if interleaved, (a, b) becomes (a c - b s,
 * b c + a s) with c = cos_sin[t][j], s = cos_sin[t][rotary_dim/2 + j]; in
 * binary32, rounded once.  rotary_dim 0: none.
 *
 * q, k, v, q_out: [tokens, heads, dim], 16-byte aligned heads, the last
 * dimension contiguous.  q_heads 0: no queries.  q_out may be exactly q.
 * dim: a multiple of 8 (of 4 for DC_F32) up to 1024; rotary_dim a multiple of
 * 16 (half as much for DC_F32, and for pairs that are interleaved).
 * A negative position marks padding: nothing is written for it.  A token
 * whose sequence, position or page does not exist leaves the cache alone and
 * its q_out row is NaN.  Two tokens for one slot: each 16 bytes of its heads
 * hold either's numbers, not all of them the same one's.
 * The caches may be interleaved in one tensor (pages of keys beside pages of
 * values); what a call writes must not fold onto itself (a broadcast q_out or
 * cache), share bytes with what else it writes (a cache that is the other, a
 * slot or a head on) or overlap what it reads (DC_ERR_OVERLAP).  Queries
 * rotated in place may lie beside k and v in one tensor; layouts that cannot be
 * shown to share no byte are refused too.
 */
typedef struct {
    const void *q;
    const void *k;
    const void *v;
    void *q_out;
    const int32_t *positions;
    const int32_t *seqs;
    const int32_t *page_table;
    const float *cos_sin;   /* [cos_sin_rows, rotary_dim] */
    dc_paged_cache_t k_cache;
    dc_paged_cache_t v_cache;
    uint64_t q_token_stride, q_head_stride;
    uint64_t k_token_stride, k_head_stride;
    uint64_t v_token_stride, v_head_stride;
    uint64_t q_out_token_stride, q_out_head_stride;
    int64_t tokens;
    int64_t table_rows, table_width, table_stride;
    int64_t cos_sin_rows;
    int64_t num_pages;
    int32_t page_size;
    int32_t q_heads;
    int32_t kv_heads;
    int32_t dim;
    int32_t rotary_dim;
    int32_t interleaved;
    int32_t dtype;
    int32_t reserved;       /* 0 */
} dc_kv_append_t;
dc_status_t dc_kv_append(const dc_kv_append_t *args, dc_stream_t stream);

/*
 * dc_kv_append_norm -- dc_kv_append of keys and queries that are normed first:
 * a head x of `dim` elements becomes x w / sqrt(mean x^2 + eps), with weights
 * w = q_norm or k_norm [dim] (of the heads' type, or binary32 if norm_32), and
 * is rotated then; in binary32, rounded once.  Values are copied.  q_norm may be
 * NULL without queries.  dim up to 512; everything else as for dc_kv_append.
 */
typedef struct {
    dc_kv_append_t append;
    const void *q_norm;
    const void *k_norm;
    float eps;
    int32_t norm_32;
} dc_kv_append_norm_t;
dc_status_t dc_kv_append_norm(const dc_kv_append_norm_t *args, dc_stream_t stream);

/* A [tokens, heads, dim] tensor: element d of head h of token t is
 * data[t*token_stride + h*head_stride + d], every head 16-byte aligned. */
typedef struct {
    void *data;
    uint64_t token_stride;
    uint64_t head_stride;
} dc_heads_t;

/*
 * dc_qk_norm_rotate -- the queries and keys of a training step: q -> q_out and
 * k -> k_out, each head normed and rotated as dc_kv_append_norm does it (the
 * same bits), to positions[i].
 *
 * A negative position marks padding: its rows are 0, and so is its gradient.  A
 * position past cos_sin gives NaN in its rows.  cos_sin NULL with rotary_dim 0:
 * no rotation.  dim: a multiple of 8 (of 4 for DC_F32) up to 512; rotary_dim as
 * for dc_kv_append.  q_out may be exactly q, and k_out exactly k; outputs lie
 * apart otherwise (heads of one tensor beside one another are fine).
 */
typedef struct {
    dc_heads_t q, k, q_out, k_out;
    const int32_t *positions;
    const float *cos_sin;   /* [cos_sin_rows, rotary_dim] */
    const void *q_norm;
    const void *k_norm;
    int64_t tokens;
    int64_t cos_sin_rows;
    int32_t q_heads;
    int32_t kv_heads;
    int32_t dim;
    int32_t rotary_dim;
    int32_t interleaved;
    int32_t dtype;
    int32_t norm_32;
    float eps;
} dc_qk_norm_rotate_t;
dc_status_t dc_qk_norm_rotate(const dc_qk_norm_rotate_t *args, dc_stream_t stream);

/*
 * dc_qk_norm_rotate_backward -- its gradient: from that of q_out and k_out
 * (grad_q_out, grad_k_out) those of q, k and the weights.  With g the gradient
 * rotated back, r = 1 / sqrt(mean x^2 + eps) and n = x r:
 *
 *   grad_x = r (g w - n mean(g w n));   grad_w = sum over tokens and heads of g n.
 *
 * grad_q and grad_k may be exactly grad_q_out and grad_k_out.  grad_q_norm and
 * grad_k_norm [dim] (typed as the weights) replace what was there; NULL: not
 * wanted.  Their sums are binary32 in one fixed order, which follows from the
 * number of tokens and heads; without tokens they are 0.  A token whose position
 * is past cos_sin makes them NaN.
 * workspace (for them): dc_qk_norm_workspace_bytes bytes, 16-byte aligned, whose
 * contents do not matter; calls that overlap on the GPU need one each.  One or
 * two kernels.
 */
typedef struct {
    dc_heads_t q, k, grad_q_out, grad_k_out, grad_q, grad_k;
    const int32_t *positions;
    const float *cos_sin;
    const void *q_norm;
    const void *k_norm;
    void *grad_q_norm;
    void *grad_k_norm;
    void *workspace;
    uint64_t workspace_bytes;
    int64_t tokens;
    int64_t cos_sin_rows;
    int32_t q_heads;
    int32_t kv_heads;
    int32_t dim;
    int32_t rotary_dim;
    int32_t interleaved;
    int32_t dtype;
    int32_t norm_32;
    float eps;
} dc_qk_norm_rotate_backward_t;
dc_status_t dc_qk_norm_rotate_backward(const dc_qk_norm_rotate_backward_t *args, dc_stream_t stream);
/* 0 if the arguments are not supported. */
size_t dc_qk_norm_workspace_bytes(int64_t tokens, int q_heads, int kv_heads, int dim);

/*
 * dc_paged_attention -- attention of one new token per sequence over a paged
 * cache.  Query head h of sequence b attends, through key head
 * h / (q_heads / kv_heads), to tokens t of [max(0, lengths[b] - window),
 * lengths[b]) (window 0: all):
 *
 *   out = sum_t softmax_t(scale * q . k_t) v_t;
 *   lse = log(sum_t exp(scale * q . k_t))           (NULL if not wanted)
 *
 * q, out: [seqs, q_heads, dim], 16-byte aligned heads; DC_BF16 or DC_F16;
 * dim 64, 96, 128, 192 or 256.  lse [seqs, q_heads], contiguous.
 * A sequence of length 0 gives zeros and lse = -inf.  A page number outside
 * the cache among the attended ones, or a length past the table, gives NaN;
 * entries of the table past a sequence's length are not read.
 *
 * workspace: device memory of at least dc_attention_workspace_bytes(seqs,
 * q_heads, kv_heads, dim, max_tokens) bytes, 16-byte aligned, owned by the
 * caller, zero before its first use (each call leaves it ready for the next,
 * of any shape it is large enough for, and with any workspace_bytes that is
 * enough for that call).  Memory that starts elsewhere, inside a workspace too,
 * is another workspace.  max_tokens: table_width * page_size, or the window if
 * that is shorter.  Calls on one workspace must not overlap on the GPU: one per
 * stream.
 */
typedef struct {
    const void *q;
    void *out;
    float *lse;
    const int32_t *page_table;
    const int32_t *lengths;
    void *workspace;
    uint64_t workspace_bytes;
    dc_paged_cache_t k_cache;
    dc_paged_cache_t v_cache;
    uint64_t q_seq_stride, q_head_stride;
    uint64_t out_seq_stride, out_head_stride;
    int64_t seqs;
    int64_t table_width, table_stride;
    int64_t num_pages;
    int32_t page_size;
    int32_t q_heads;
    int32_t kv_heads;
    int32_t dim;
    int32_t window;
    int32_t dtype;
    float scale;
    int32_t reserved;       /* 0 */
} dc_paged_attention_t;
dc_status_t dc_paged_attention(const dc_paged_attention_t *args, dc_stream_t stream);
/* 0 if the arguments are not supported. */
size_t dc_attention_workspace_bytes(int64_t seqs, int q_heads, int kv_heads, int dim, int64_t max_tokens);

/*
 * dc_prefix_attention -- dc_paged_attention of sequences that share prefixes:
 * the `seqs` sequences are `prefixes` groups of seqs / prefixes neighbours, and
 * sequence b attends to the first prefix_lengths[g] tokens of its group's row g
 * of prefix_table, then to its own lengths[b] tokens of page_table, under one
 * softmax.  A prefix's keys and values are read once for its whole group.
 *
 * own: the arguments of dc_paged_attention (no window); prefix_table int32
 * [prefixes, prefix_table_width], pages of the same caches.  Either part may be
 * empty, or both (zeros and lse = -inf).  A page outside the cache, or a length
 * past its table, gives NaN in the sequences that it belongs to.
 * The prefix's weights are rounded to 16 bits before they meet the values (half
 * a step each, of either sign; for DC_F16 down to 2^-30 of the row's largest),
 * everything else as in dc_paged_attention; an infinite value gives infinities
 * or NaN.
 * A sequence's bits depend on its own tokens and its prefix's, not on the other
 * sequences or prefixes.
 * own.workspace: dc_prefix_attention_workspace_bytes(seqs, prefixes, q_heads,
 * kv_heads, dim, max_prefix_tokens, max_tokens) bytes (widths of the tables
 * times the page size), 16-byte aligned, zero before its first use; each call
 * leaves it ready for the next of these sizes (one that returned DC_ERR_CUDA may
 * not: zero it again).  One per stream.  Three kernels.
 */
typedef struct {
    dc_paged_attention_t own;
    const int32_t *prefix_table;
    const int32_t *prefix_lengths;
    int64_t prefixes;
    int64_t prefix_table_width, prefix_table_stride;
} dc_prefix_attention_t;
dc_status_t dc_prefix_attention(const dc_prefix_attention_t *args, dc_stream_t stream);
/* 0 if the arguments are not supported. */
size_t dc_prefix_attention_workspace_bytes(int64_t seqs, int64_t prefixes, int q_heads, int kv_heads, int dim,
                                           int64_t max_prefix_tokens, int64_t max_tokens);

/*
 * dc_check_device -- reports the faults that this library's kernels recorded
 * on the current device since the last check, and clears them.
 *
 * The bulk-copy gather (the "gather_bulk" path of dc_all_gather) waits for
 * its loads, and dc_fused_all_gather for its peers' flags, with a bound
 * (option "wait_limit_ns", default one second of the GPU's global timer).  A
 * wait that runs out does not hang the stream: the kernel records the fault
 * in a device word, waits with the same bound for its own copies in flight
 * and returns, leaving that call's output incomplete.  No correct bulk launch
 * on a working GPU ever runs out; a fused launch runs out when a rank never
 * arrives.  The tensor-core kernels of dc_linear_logprobs, its gradient and
 * dc_prefix_attention bound their waits for operands, products and results the
 * same way; what they still have in flight then is waited for with a limit of its own (ten
 * seconds).  None of them runs out on a working GPU at the default.
 *
 * Synchronous: it first waits for all work on the current device
 * (cudaDeviceSynchronize), then reads and clears the fault words.
 * Returns DC_OK if no wait ran out, DC_ERR_TIMEOUT if one did, DC_ERR_BOUNDS
 * (bounds-checked build only, see dc_bounds_checked) if a kernel skipped an
 * access outside its range, DC_ERR_CUDA if the synchronisation or the read
 * failed (the CUDA error in dc_last_error()).
 */
dc_status_t dc_check_device(void);

/* Message describing the last failed call on this thread ("" if none). */
const char *dc_last_error(void);

/* Name of a status code, e.g. "DC_ERR_OVERLAP". */
const char *dc_status_name(int status);

/*
 * Process-wide tuning and test options.  Keys:
 *   "force_path"              0 = automatic, 1 = single CTA, 2 = multi CTA
 *   "force_generic"           1 = never use the flat aligned gather path
 *   "gather_single_max_bytes" dc_all_gather on one CTA up to this many output
 *                             bytes (default 0: the grid was never slower on
 *                             GB300; an unaligned gather of fewer than 128
 *                             bytes per rank always runs on one CTA)
 *   "gather_many_single_max_bytes"
 *                             dc_all_gather_many on one CTA up to this many
 *                             output bytes in all (default 16384, measured)
 *   "reduce_single_max_bytes" single-CTA reductions up to this many input
 *                             bytes per rank (default 0: the grid was never
 *                             slower on GB300)
 *   "grid_ctas"               0 = automatic, else the multi-CTA grid size
 *   "pdl"                     1 (default) = launch with programmatic stream
 *                             serialization, so a kernel's launch overlaps the
 *                             end of the previous kernel in the stream (it still
 *                             waits for that kernel before touching memory)
 *   "gather_staged"           1 (default) = aligned gathers stage their loads
 *                             through shared memory with cp.async
 *   "gather_split_cost_pct"   all_gather_many with aligned and unaligned
 *                             tensors: cost of a realigned 16-byte vector in
 *                             percent of a staged aligned one, for splitting
 *                             the grid between the two (default 250, measured)
 *   "gather_split_cost_warp_pct" the same when the unaligned part (more than
 *                             16 tensors) realigns across warps (default 100,
 *                             measured)
 *   "prefetch"                tiles per CTA whose inputs are prefetched into
 *                             L2 before the kernel waits for the previous
 *                             kernel in the stream (dc_all_gather on its
 *                             aligned and staged realigning paths, and the
 *                             reductions; 0 = off; default 1)
 *   "gather_tile_min"         staged aligned gathers: the smallest tile (in
 *                             16-byte vectors) that an output too small for a
 *                             full tile per CTA is cut into, so that it is
 *                             spread evenly over the SMs (default 512, measured)
 *   "reduce_tile_min"         one-tensor all_reduce: the smallest tile (in
 *                             16-byte units) that a reduction too small for a
 *                             full tile per CTA is cut into (default 64,
 *                             measured)
 *   "reduce_staged"           1 (default) = an all_reduce of one tensor whose
 *                             inputs sit at other offsets (mod 16 bytes) than
 *                             its outputs, P = 2, 4 or 8, stages its input
 *                             blocks through shared memory; 0 = realign in
 *                             registers
 *   "gather_bulk"             1 (default) = a 16-byte aligned dc_all_gather
 *                             (out, bytes_per_rank and every peer) of at least
 *                             gather_bulk_min_bytes output bytes runs on the
 *                             TMA engine: 1-D bulk copies global -> shared ->
 *                             global through a ring of shared-memory stages
 *   "gather_bulk_min_bytes"   see gather_bulk (default 0)
 *   "bulk_chunk_bytes"        largest chunk one bulk stage moves (default 16384)
 *   "bulk_chunk_min"          smallest chunk an output too small for one
 *                             full chunk per CTA is cut into (default 2048)
 *   "bulk_stages"             ring stages per CTA (default 6, at most 32)
 *   "bulk_ctas_per_sm"        bulk CTAs per SM (default 2)
 *   "bulk_prefetch"           bulk CTAs prefetch their sources into L2 this
 *                             many chunks ahead of their loads (default 1; at
 *                             most 64 MB ahead over the grid; 0 when
 *                             "prefetch" is 0)
 *   "wait_limit_ns"           bound of one device wait (default 1000000000;
 *                             at least 1000)
 *   "test_bulk_short_tx"      1 = every bulk CTA's first wait runs out (tests
 *                             of dc_check_device)
 *   "test_tensor_late"        tests of the tensor-core kernels' bounded waits:
 *                             1 or 2 = results of the even or odd CTAs are
 *                             late, 3 or 4 = their copies; attention to shared
 *                             prefixes: 1 = a tile's weights, 2 = its values
 *   "gather_realign_warp"     1 (default) = a dc_all_gather whose payloads or
 *                             output are not 16-byte aligned (at least 128
 *                             bytes per rank, output under 4 GiB), and the
 *                             unaligned tensors of a dc_all_gather_many with
 *                             more than 16 of them, realign their vectors
 *                             across the lanes of a warp, in registers;
 *                             0 = through a shared-memory ring
 *   "fused_chunk_min"         dc_fused_all_gather: smallest chunk per CTA
 *                             (default 32768 bytes; measured, 8 ranks x 4 MiB:
 *                             75.8 us at 32 KiB, 81.9 us at 64 KiB)
 *   "fused_tma"               1 (default) = the protocol's gather step streams
 *                             the staged chunks through the TMA engine (one
 *                             thread per CTA, bulk loads and stores through a
 *                             shared-memory ring); 0 = every thread copies
 *                             16-byte vectors
 *   "fused_stages", "fused_sub_bytes"  that ring: stages (1..32, default 3) of
 *                             bytes each (a multiple of 16, default 32768)
 *   "test_fused_absent_ranks" bit r set: rank r of dc_fused_all_gather never
 *                             arrives (tests of its bounded waits)
 *   "test_fail_launch"        1 = report DC_ERR_CUDA instead of launching
 * Environment variables DC_FORCE_PATH, DC_FORCE_GENERIC,
 * DC_GATHER_SINGLE_MAX_BYTES, DC_GATHER_MANY_SINGLE_MAX_BYTES,
 * DC_REDUCE_SINGLE_MAX_BYTES, DC_GRID_CTAS, DC_PDL,
 * DC_GATHER_STAGED, DC_GATHER_SPLIT_COST_PCT, DC_GATHER_SPLIT_COST_WARP_PCT, DC_PREFETCH, DC_GATHER_TILE_MIN,
 * DC_REDUCE_TILE_MIN, DC_REDUCE_STAGED, DC_GATHER_BULK, DC_GATHER_BULK_MIN_BYTES,
 * DC_BULK_CHUNK_BYTES, DC_BULK_CHUNK_MIN, DC_BULK_STAGES, DC_BULK_CTAS_PER_SM,
 * DC_BULK_PREFETCH, DC_GATHER_REALIGN_WARP, DC_FUSED_CHUNK_MIN, DC_FUSED_TMA, DC_FUSED_STAGES,
 * DC_FUSED_SUB_BYTES and DC_WAIT_LIMIT_NS set the initial values (read once,
 * at the first call).
 * dc_set_option returns 0, or -1 for an unknown key or a negative value.
 * dc_get_option returns the value, or -1 for an unknown key.
 */
int dc_set_option(const char *key, long long value);
long long dc_get_option(const char *key);

/* Kernels launched by this library since it was loaded (all threads). */
unsigned long long dc_launch_count(void);

/* CTAs in the grid of the calling thread's last successful launch (0 before
 * the first): a diagnostic of the planner's grid choice. */
int dc_last_grid(void);

/* ABI version: 1. */
int dc_version(void);

/*
 * 1 in the bounds-checked build of the library (libdc_bounds.so, compiled
 * with DC_DEBUG_BOUNDS), 0 in the normal one.  In the checked build every
 * global load, store and L2 prefetch of every kernel is first checked against
 * the range its job allows -- for a load, the 16-byte-block hull of the
 * source bytes the job reads (realigning copies read whole aligned blocks
 * around an unaligned span); for a store, the exact output range.  An access
 * outside is skipped (never made) and the first one is recorded;
 * dc_check_device then returns DC_ERR_BOUNDS with the file, site, address and
 * allowed range.  The kernels never trap.  It is a test build: slower, and
 * otherwise the same results.
 */
int dc_bounds_checked(void);

#ifdef __cplusplus
}
#endif
#endif /* DC_H */
