/*
 * rsx -- ring reduce-scatter / all-gather / all-reduce on one MI355X (gfx950).
 *
 * C ABI of librsx.so.  One process drives W "virtual ranks": rank r is a
 * buffer in the one GPU's HBM, and each call takes a host array of W device
 * pointers where a communicator-based library would take one buffer and a
 * communicator.  Every entry point enqueues its kernels on `stream` and
 * returns without synchronising the host.
 *
 * Sources of the semantics (web pages):
 *   [NC] NCCL 1.x src/reduce_scatter.cu (pytorch mirror, "Git at Google"):
 *        ncclReduceScatter, the ring kernel and GetBlock, its host launcher
 *        (count 0 -> success; one device -> plain copy) and its op/type
 *        dispatch (unknown op / type -> an error code).
 *   [DP] "Distributed primitives": reduce-scatter, all-gather, all-reduce,
 *        Ring AllReduce = ReduceScatter + AllGather, bucketed ring all-reduce.
 *   [SG] Apache SINGA src/io/communicator.cc, fusedSynch / synch: tensors
 *        packed back to back into a fusion buffer, all-reduced, unpacked;
 *        in-place all-reduce of a tensor.
 *   [HV] Horovod horovod/common/operations.cc, PerformOperation: memcpy into
 *        the fusion buffer at running offsets, in-place all-reduce, memcpy out.
 *   [MX] "Add scatter reduce for JACCL#3901": naive all-reduce for messages
 *        of at most 32 KB.
 *
 * Common conventions
 *   - Pointer arrays (`sendbufs`, `recvbufs`, `tensors`, `counts`) are HOST
 *     arrays, read during the call only.  The device buffers they point to
 *     are owned by the caller and must stay valid until the stream work ends.
 *   - The library allocates no device or pinned memory and does not
 *     synchronise; it launches kernels on `stream` (0 = the null stream) on
 *     the calling thread's current HIP device, which must hold every buffer.
 *   - Validation (null pointers, rank count, enum ranges, size overflow,
 *     illegal buffer overlap) happens before any HIP call; a rejected call
 *     has no effect.  A failed launch returns RSX_ERR_HIP, and
 *     rsx_status_string(RSX_ERR_HIP) then names the HIP error (per thread).
 *   - Counts are elements, not bytes.  A count of 0 returns RSX_SUCCESS
 *     without launching anything [NC host launcher].
 *   - Every buffer must start at a multiple of its element size (4 for
 *     fp32, 2 for bf16, ...); any other address returns
 *     RSX_ERR_INVALID_ARGUMENT.  Buffers of 16-byte-aligned address take the
 *     dwordx4 kernels (for reduce-scatter blocks and all-gather pieces whose
 *     byte length is a multiple of 4, with dword-aligned loads where they are
 *     not whole 16-byte vectors); other element-aligned addresses are correct
 *     but slower.
 *   - Bit-exact means equal bit patterns, except that NaN payloads are not
 *     specified: where the result is a NaN, any NaN is correct (the pages fix
 *     no NaN propagation rule; bf16 rounding quiets a NaN as sign|0x7FC0).
 *   - The dwordx4 reduction and gather kernels reserve LDS they do not use
 *     (up to 96 KiB per workgroup) to limit how many of their workgroups
 *     share a CU, unless the calling thread turned that off with
 *     rsx_set_occupancy_caps (for launches that overlap other kernels).
 */
#ifndef RSX_H
#define RSX_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RSX_VERSION 130          /* 1.3.0 */
#define RSX_MAX_RANKS 16         /* largest W a call accepts */
#define RSX_NAIVE_MAX_BYTES 32768 /* RSX_ALGO_AUTO picks naive at or below this, per rank [MX] */
#define RSX_FUSE_BATCH 248       /* tensors per pack/unpack launch */
#define RSX_TOP_MAX 64           /* most alternatives of rsx_token_logprobs */
#define RSX_SPARSE_SCRATCH_BYTES 134217728 /* 128 MiB: scratch array of rsx_sparse_all_reduce_noalloc, per GPU */

typedef enum {
  RSX_FLOAT32 = 0,   /* fp32 in, fp32 fold, fp32 out */
  RSX_BFLOAT16 = 1,  /* bf16 in, widened exactly to fp32, fp32 fold, one RNE rounding to bf16 out */
  RSX_INT32 = 2,     /* int32, two's-complement wrapping sum and product */
  RSX_FLOAT64 = 3,   /* fp64 in, fp64 fold, fp64 out */
  RSX_FLOAT16 = 4,   /* IEEE half in and out, folded in half: the ring partial is rounded (RNE)
                        to half after every step, as the page's T-typed ring buffers hold it
                        [NC ReduceScatterKernelArgs<T>, ThisBuffer / NextBuffer]; avg divides
                        the half fold by W, the quotient rounded to half */
  RSX_INT64 = 5,     /* int64, wrapping */
  RSX_UINT64 = 6,    /* uint64, wrapping */
  RSX_INT8 = 7,      /* int8 (the page's char), wrapping */
  RSX_FLOAT32_HALF_WIRE = 8 /* fp32 in and out with IEEE half as the wire format
                               [Apache SINGA communicator.cc, synchHalf / fusedSynchHalf]:
                               each input is rounded (RNE) to half, the halves are folded
                               as RSX_FLOAT16 is (half partial at every ring step), and the
                               half result is widened to fp32.  Reductions only:
                               rsx_all_gather rejects it with RSX_ERR_INVALID_TYPE; pack and
                               unpack treat it as fp32.  W = 1 still rounds through half. */
} rsx_dtype_t;

typedef enum {
  RSX_SUM = 0,
  RSX_MAX = 1,       /* compare-select fold: a later value replaces the partial only if greater */
  RSX_MIN = 2,       /* compare-select fold: a later value replaces the partial only if smaller */
  RSX_AVG = 3,       /* sum fold, then one division by W in the fold type (signed: toward zero) */
  RSX_PROD = 4       /* product fold (integers wrap) [NC FuncProd] */
} rsx_op_t;

typedef enum {
  RSX_ALGO_RING = 0,       /* segment k folded in ring order (k+1)%W, ..., k; then gathered, in
                              one pass or two (the faster form for the shape; same bits) */
  RSX_ALGO_NAIVE = 1,      /* every element folded in rank order 0..W-1 [MX] */
  RSX_ALGO_AUTO = 2,       /* NAIVE when count * element size <= RSX_NAIVE_MAX_BYTES, else RING */
  RSX_ALGO_RING_FUSED = 3, /* RING, always as one pass (fold, then store to every rank) */
  RSX_ALGO_RING_SPLIT = 4  /* RING, always as a reduce-scatter, then an all-gather [DP] */
} rsx_algo_t;

typedef enum {
  RSX_SUCCESS = 0,
  RSX_ERR_INVALID_ARGUMENT = 1, /* null or misaligned pointer, rank count out of [1, RSX_MAX_RANKS], bad algo */
  RSX_ERR_INVALID_TYPE = 2,     /* dtype outside rsx_dtype_t [NC: invalid type] */
  RSX_ERR_INVALID_OP = 3,       /* op outside rsx_op_t [NC: invalid operation] */
  RSX_ERR_UNSUPPORTED = 4,      /* sizes whose byte count or launch grid overflows */
  RSX_ERR_ALIASING = 5,         /* buffers overlap in a way other than the in-place forms */
  RSX_ERR_HIP = 6               /* a HIP launch failed; see rsx_status_string */
} rsx_status_t;

/*
 * Reduce-scatter [NC ncclReduceScatter; DP "Reduce-Scatter"].
 *
 * sendbufs[r]  device array of W*recvcount elements, rank r's input.
 * recvbufs[k]  device array of recvcount elements, receives block k:
 *              recvbufs[k][i] = fold of sendbufs[r][k*recvcount + i] over
 *              r = (k+1)%W, (k+2)%W, ..., k, in that order (the ring's order:
 *              block k leaves the position after k at step 0 and ends on
 *              position k at step W-1, per GetBlock with the identity ring).
 * nranks       W, 1..RSX_MAX_RANKS.  W = 1 is a copy (nothing if in place).
 * In place: recvbufs[k] == (char*)sendbufs[k] + k*recvcount*size is allowed.
 * Any other overlap of a recv buffer with a send buffer or another recv
 * buffer returns RSX_ERR_ALIASING.  Send buffers may alias each other only
 * when identical.
 */
rsx_status_t rsx_reduce_scatter(const void* const* sendbufs, void* const* recvbufs,
                                int nranks, size_t recvcount, rsx_dtype_t dtype,
                                rsx_op_t op, hipStream_t stream);

/*
 * All-gather [DP "All-Gather"; the gather half of Ring AllReduce].
 *
 * sendbufs[k]  device array of sendcount elements, rank k's piece.
 * recvbufs[r]  device array of W*sendcount elements; on return
 *              recvbufs[r][k*sendcount + i] = sendbufs[k][i] for every r, k.
 * In place: sendbufs[k] == (char*)recvbufs[k] + k*sendcount*size is allowed.
 * Other overlaps return RSX_ERR_ALIASING.
 */
rsx_status_t rsx_all_gather(const void* const* sendbufs, void* const* recvbufs,
                            int nranks, size_t sendcount, rsx_dtype_t dtype,
                            hipStream_t stream);

/*
 * All-reduce [DP Ring AllReduce = ReduceScatter + AllGather; SG synch; HV
 * PerformOperation].
 *
 * sendbufs[r], recvbufs[r]  device arrays of `count` elements.
 * RSX_ALGO_RING: the `count` elements are split into W segments of
 *   S = ceil(count/W): segment k = [min(kS,count), min((k+1)S,count)), see
 *   rsx_segment_begin.  Segment k is folded in ring order (k+1)%W, ..., k and
 *   written to every rank: the result equals rsx_all_gather applied to the
 *   reduce-scatter output whenever W divides count.  Two forms give the
 *   same bits (the same folds in the same order):
 *   - one pass (RSX_ALGO_RING_FUSED): each lane folds its element of all W
 *     inputs in registers and stores the result to all W outputs;
 *   - two passes (RSX_ALGO_RING_SPLIT): a reduce-scatter writes segment k
 *     into recvbufs[k] at its own offset, then an all-gather copies it from
 *     there to the other W-1 outputs, (2W+1)/(2W) of the one-pass bytes.
 *     W must divide count (else RSX_ERR_UNSUPPORTED); any element-aligned address.
 *   RSX_ALGO_RING takes two passes when W >= 7, W divides count, every
 *   buffer and segment is 16-byte aligned and a rank holds at least 4 MiB
 *   (measured faster there), one pass otherwise.
 * RSX_ALGO_NAIVE: every element folded in rank order 0..W-1 [MX].
 * In place: recvbufs[r] == sendbufs[r] for every r (or a permutation of the
 * send buffers) is allowed; other overlaps return RSX_ERR_ALIASING.
 */
rsx_status_t rsx_all_reduce(const void* const* sendbufs, void* const* recvbufs,
                            int nranks, size_t count, rsx_dtype_t dtype, rsx_op_t op,
                            rsx_algo_t algo, hipStream_t stream);

/*
 * Bucketed all-reduce ["Distributed primitives", In practice: the gradient
 * is all-reduced in buckets, one after another].
 *
 * The `count` elements of every rank are cut into consecutive buckets of
 * bucket_elems elements, the last one shorter: bucket b = [b*bucket_elems,
 * min((b+1)*bucket_elems, count)).  Each bucket is an rsx_all_reduce of its
 * own, with its own segments (S = ceil(len/W), ring order per segment) and
 * its own RSX_ALGO_AUTO choice, launched in bucket order on `stream`.  The
 * result equals rsx_all_reduce on each bucket in turn.  When W divides
 * bucket_elems, the full buckets share one launch per pass (each bucket
 * still folded over its own segments in its own ring order) and the shorter
 * last bucket follows.
 * Arguments, ownership, in-place and aliasing rules: as rsx_all_reduce, on
 * the whole buffers.  bucket_elems = 0: RSX_ERR_INVALID_ARGUMENT.
 * RSX_ALGO_RING_SPLIT needs W to divide every bucket (RSX_ERR_UNSUPPORTED).
 * The whole call is validated before the first launch.
 */
rsx_status_t rsx_all_reduce_bucketed(const void* const* sendbufs, void* const* recvbufs,
                                     int nranks, size_t count, size_t bucket_elems,
                                     rsx_dtype_t dtype, rsx_op_t op, rsx_algo_t algo,
                                     hipStream_t stream);

/*
 * One bucket of a bucketed all-reduce ["Distributed primitives", In
 * practice: each bucket is all-reduced as soon as the backward pass has
 * produced it, on a stream of its own].
 *
 * The all-reduce of bucket `bucket` alone, [bucket*bucket_elems,
 * min((bucket+1)*bucket_elems, count)), with that bucket's own segments and
 * RSX_ALGO_AUTO choice: the result equals what rsx_all_reduce_bucketed
 * stores for it.  For callers that enqueue each bucket when its inputs are
 * ready.  Arguments and validation as rsx_all_reduce_bucketed, on the whole
 * buffers; bucket >= rsx_bucket_count(count, bucket_elems):
 * RSX_ERR_INVALID_ARGUMENT (count = 0: nothing to do, RSX_SUCCESS).
 */
rsx_status_t rsx_all_reduce_bucket(const void* const* sendbufs, void* const* recvbufs,
                                   int nranks, size_t count, size_t bucket_elems, size_t bucket,
                                   rsx_dtype_t dtype, rsx_op_t op, rsx_algo_t algo,
                                   hipStream_t stream);

/* Buckets of a bucketed all-reduce: ceil(count / bucket_elems); 0 when
 * bucket_elems is 0. */
size_t rsx_bucket_count(size_t count, size_t bucket_elems);

/*
 * Tensor-fusion pack [SG fusedSynch(send=false); HV PerformOperation memcpy in].
 *
 * Copies tensors[i] (device, counts[i] elements) to
 * fused + (counts[0] + ... + counts[i-1]) elements: back to back, in list
 * order, with no padding.  `fused` must hold the sum of counts and must not
 * overlap any tensor (RSX_ERR_ALIASING).  ntensors >= 0; zero-count tensors
 * are skipped and may be null.  Launches one kernel per RSX_FUSE_BATCH
 * non-empty tensors (a tensor above 16 GiB counts once per 16 GiB).  The sum
 * of counts times the element size must stay below 2^40 bytes
 * (RSX_ERR_UNSUPPORTED otherwise).
 */
rsx_status_t rsx_fuse_pack(const void* const* tensors, const size_t* counts, int ntensors,
                           void* fused, rsx_dtype_t dtype, hipStream_t stream);

/*
 * Tensor-fusion unpack [SG fusedSynch(send=true) copy-out; HV memcpy out]:
 * the inverse of rsx_fuse_pack, same offsets and rules.
 */
rsx_status_t rsx_fuse_unpack(const void* fused, void* const* tensors, const size_t* counts,
                             int ntensors, rsx_dtype_t dtype, hipStream_t stream);

/*
 * Tensor-fusion all-reduce without a fusion buffer [SG fusedSynch; HV
 * PerformOperation; DP Ring AllReduce].
 *
 * sendtensors[r*ntensors + i], recvtensors[r*ntensors + i]: device arrays of
 * rank r's tensor i, counts[i] elements each (the same count on every rank).
 * The result is, bit for bit, that of rsx_fuse_pack of each rank's list into
 * a buffer of F = counts[0] + ... + counts[n-1] elements, rsx_all_reduce of
 * the W buffers with `algo`, then rsx_fuse_unpack into recvtensors: element
 * j of tensor i sits at fused offset counts[0] + ... + counts[i-1] + j and is
 * folded in the order of the fused segment holding that offset.  No fusion
 * buffer is read or written, so HBM traffic is one all-reduce of the tensors.
 * RSX_ALGO_AUTO picks naive when F * element size <= RSX_NAIVE_MAX_BYTES.
 * Ring order is always one pass here (RSX_ALGO_RING_FUSED and RSX_ALGO_RING
 * alike); RSX_ALGO_RING_SPLIT returns RSX_ERR_UNSUPPORTED.
 * In place: recvtensors[r*n + i] == sendtensors[r2*n + i] (same tensor index)
 * is allowed; any other overlap of a destination returns RSX_ERR_ALIASING.
 * Zero-count tensors are skipped and may be null.  Launches about one kernel
 * per 256 / (2W) tensors (256 / W when every destination is its own source).
 */
rsx_status_t rsx_fused_all_reduce(const void* const* sendtensors, void* const* recvtensors,
                                  const size_t* counts, int ntensors, int nranks,
                                  rsx_dtype_t dtype, rsx_op_t op, rsx_algo_t algo,
                                  hipStream_t stream);

/* Sparsification of rsx_sparse_all_reduce [SG valSparsAllReduce / topKSparsAllReduce]. */
typedef enum {
  RSX_SPARSE_THRESHOLD = 0, /* send the entries with |x| >= threshold (never a zero) */
  RSX_SPARSE_TOPK = 1       /* send the k largest values (not magnitudes); ties by lower index */
} rsx_sparse_mode_t;

/*
 * K of the top-K mode as the page computes it: ceil(fraction * count) with
 * `fraction` a float and `count` converted to float, the product rounded to
 * float [SG topKSparsAllReduce].  Returns 0 when the product is not positive
 * (or NaN).  Host arithmetic only.
 */
size_t rsx_sparse_topk_count(size_t count, float fraction);

/*
 * Bytes of device workspace rsx_sparse_all_reduce needs for these sizes:
 * per-tile counts and offsets, radix histograms and 8 bytes per element per
 * rank (rounded up to whole 4096-element tiles) of per-tile entry slots.
 * The same for both modes and with or without an accumulation.  0 for
 * invalid arguments.
 */
size_t rsx_sparse_workspace_size(int nranks, size_t count, rsx_sparse_mode_t mode, int has_accum);

/*
 * Sparsified all-reduce with error feedback [SG valSparsAllReduce,
 * topKSparsAllReduce, via sparsification / fusedSparsification].
 *
 * For each rank r, with g = grads[r] + accums[r] (one fp32 add; g = grads[r]
 * when accums is NULL):
 *   RSX_SPARSE_THRESHOLD: entry i is sent when |g[i]| >= threshold and
 *     g[i] != 0 (any threshold: a NaN threshold sends nothing, one <= 0
 *     every nonzero entry);
 *   RSX_SPARSE_TOPK: the k largest g[i] are sent (a NaN ranks below every
 *     number, -0 equals +0, equal values are taken by increasing index);
 *   with accums: accums[r][i] = g[i] - (0 + g[i]) where sent, g[i] - 0 where
 *     not (what was not sent; a sent inf leaves NaN);
 *   msg_idx[r][0..nnz[r]), msg_val[r][0..nnz[r]): the sent (zero-based
 *     index, g value) pairs in increasing index order (the page's wire
 *     message; its top-K message holds the same pairs sorted by value).
 * Then every outs[r][i] = the fp32 sum, starting from +0 and taking ranks
 * 0, 1, ..., W-1 in order, of the values sent for index i (+0 if none).
 *
 * grads[r], outs[r], accums[r]: device arrays of `count` fp32, 16-byte
 *   aligned.  accums may be NULL (no error feedback); if not, every entry
 *   must be set.  outs[r] == grads[r] is allowed (in place, as the page
 *   writes the result into the gradient).
 * msg_idx[r], msg_val[r]: device arrays of msg_capacity entries, 4-byte
 *   aligned; msg_capacity >= count (threshold) or >= k (top-K).
 * nnz: device array of nranks uint32, the message lengths (k for top-K).
 * workspace: device memory, 256-byte aligned, of at least
 *   rsx_sparse_workspace_size(...) bytes; its contents are scratch.
 * count <= UINT32_MAX (indices are uint32); k <= count.
 * count 0: nnz is zeroed and nothing else is touched.
 * The outputs may overlap the gradients (they are written after every read
 * of the gradients; e.g. outs[r] == grads[r]) and gradients may overlap each
 * other; any other overlap among grads, accums, outs, messages, nnz and the
 * workspace is RSX_ERR_ALIASING.  Invalid sizes, pointers, alignment, mode or
 * capacity: RSX_ERR_INVALID_ARGUMENT; count > UINT32_MAX: RSX_ERR_UNSUPPORTED.
 * With an accumulation, top-K writes accums[r] twice (a guess of the
 * residual, then its corrections), so accums[r] must not be read by other
 * work meanwhile.  Validation precedes every HIP call.  Enqueues 4 kernels
 * (threshold) or up to 16 (top-K) on `stream`; allocates nothing and does
 * not synchronise.
 */
rsx_status_t rsx_sparse_all_reduce(const float* const* grads, float* const* accums,
                                   float* const* outs, int nranks, size_t count,
                                   rsx_sparse_mode_t mode, float threshold, size_t k,
                                   uint32_t* const* msg_idx, float* const* msg_val,
                                   size_t msg_capacity, uint32_t* nnz, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream);

/*
 * The sparsified all-reduce above without a workspace argument, for callers
 * that cannot allocate device memory (code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc).  Same arguments, results,
 * validation and errors as rsx_sparse_all_reduce; it calls no hipMalloc or
 * hipFree and allocates nothing.
 *
 * Its workspace is a library-owned array of RSX_SPARSE_SCRATCH_BYTES in each
 * GPU's memory, held from the first call on that GPU until the process ends.
 * Sizes whose rsx_sparse_workspace_size(...) exceeds RSX_SPARSE_SCRATCH_BYTES
 * return RSX_ERR_UNSUPPORTED (8 bytes per element of every rank plus a little:
 * e.g. W * count up to about 16 M elements).  The kernels initialise what they
 * read of it, so contents left by an earlier call do not matter.  Every call
 * on one GPU uses the same array: calls that overlap in time on one GPU (on
 * different streams, or from different threads) race and give wrong results;
 * serialise them.  Enqueues on `stream` and does not synchronise.
 */
rsx_status_t rsx_sparse_all_reduce_noalloc(const float* const* grads, float* const* accums,
                                           float* const* outs, int nranks, size_t count,
                                           rsx_sparse_mode_t mode, float threshold, size_t k,
                                           uint32_t* const* msg_idx, float* const* msg_val,
                                           size_t msg_capacity, uint32_t* nnz, hipStream_t stream);

/*
 * Tensor-fusion planner [HV BackgroundThreadLoop, fusion of consecutive
 * all-reduce requests; HorovodGlobalState tensor_fusion_threshold, default
 * 64 MiB, overridden by an environment variable].
 *
 * Groups tensors 0..ntensors-1 in order: a group starts at the first tensor
 * not yet grouped and takes each next tensor while that tensor has the
 * group's dtype and the group's bytes plus its bytes stay <= threshold_bytes.
 * A tensor that does not fit ends the group; none is skipped.  A tensor
 * larger than the threshold is a group of its own.
 * counts[i], dtypes[i]: tensor i's element count and type (host arrays).
 * group_end: host array of at least ntensors ints; group g is tensors
 *   [group_end[g-1], group_end[g]) (group_end[-1] taken as 0).
 * Returns the number of groups (0 for no tensors), or -1 for a null array, a
 * negative ntensors or an invalid dtype.  Host logic only: no HIP call.
 */
int rsx_fusion_plan(const size_t* counts, const rsx_dtype_t* dtypes, int ntensors,
                    size_t threshold_bytes, int* group_end);

/*
 * Training-step operators: what makes the gradients that the collectives
 * above reduce.
 *
 * Rows.  A matrix argument is rows of `dim` elements that lie side by side,
 * `stride` elements from one row's first to the next row's (stride >= dim; a
 * matrix that is only read may have stride 0, one row standing for all).
 * Any element-aligned address, stride and length is correct.
 * Element types are RSX_FLOAT32, RSX_BFLOAT16 and RSX_FLOAT16; sums, norms
 * and softmax statistics are held in fp32 and rounded once, to nearest even,
 * at the store.  Token types are RSX_INT32 and RSX_INT64.  Other types:
 * RSX_ERR_INVALID_TYPE.  Results are the same bits on every run.
 * Overlap of an output with anything else is RSX_ERR_ALIASING, except for the
 * in-place forms named; rows of two matrices of one stride in bytes may
 * interleave.  Sizes: dim, vocab, rows and token counts below 2^31, buffers
 * below 2^45 bytes, else RSX_ERR_UNSUPPORTED.  A workspace is device memory,
 * 256-byte aligned, of at least the bytes that its _workspace_size gives
 * (null is right for 0); its contents are scratch, and two calls that may run
 * at the same time need two.
 * Launched, like everything here, on `stream`, with nothing allocated and no
 * synchronisation; they may be captured into a graph.
 */

/*
 * Embedding lookup with scaling: with t = tokens[i] - first,
 * out[i] = scale * table[t] for 0 <= t < vocab, else a row of zeros.
 * `first` is the token id of the table's first row: a table cut by rows over
 * the ranks is looked up part by part, and the sum all-reduce of the outputs
 * is the whole table's lookup.  first + vocab is at most 2^63.
 */
rsx_status_t rsx_embedding(const void* table, size_t table_stride, size_t vocab, size_t dim,
                           rsx_dtype_t table_type, const void* tokens, size_t ntokens,
                           rsx_dtype_t token_type, int64_t first, float scale, void* out,
                           size_t out_stride, rsx_dtype_t out_type, hipStream_t stream);

/*
 * Gradient of rsx_embedding in its table:
 * grad[v] = (accumulate ? grad[v] : 0) + scale * sum of dout[i] over the i
 * with tokens[i] - first = v.  A row's sum is taken in the order of its
 * positions, in parts: many tokens are sorted for it.  Without `accumulate` every
 * row is written, with it only the rows that occur.
 */
size_t rsx_embedding_grad_workspace_size(size_t ntokens, size_t vocab, size_t dim);
rsx_status_t rsx_embedding_grad(const void* dout, size_t dout_stride, rsx_dtype_t dout_type,
                                const void* tokens, size_t ntokens, rsx_dtype_t token_type,
                                int64_t first, float scale, void* grad, size_t grad_stride,
                                size_t vocab, size_t dim, rsx_dtype_t grad_type, int accumulate,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Layer norm: y = (x - mean) * rstd * weight + bias, with each row's
 * mean = sum x / dim and rstd = (sum (x - mean)^2 / dim + eps)^(-1/2).
 * weight, bias: `dim` elements of weight_type (x's type or RSX_FLOAT32), or
 * null (1 and 0).  mean, rstd: `rows` fp32, or null.
 * codes, scales: null, or an 8-bit checkpoint of x written on the way, as
 * rsx_checkpoint_pack does.  y == x with one stride is allowed.
 * dim = 0 writes nothing, mean and rstd neither.
 */
rsx_status_t rsx_layer_norm(const void* x, size_t x_stride, const void* weight, const void* bias,
                            void* y, size_t y_stride, float* mean, float* rstd, int8_t* codes,
                            uint8_t* scales, size_t rows, size_t dim, float eps, rsx_dtype_t type,
                            rsx_dtype_t weight_type, hipStream_t stream);

/*
 * Gradients of rsx_layer_norm: with xhat = (x - mean) * rstd and g = dy * weight,
 * dx = rstd * (g - mean(g) - xhat * mean(g * xhat)), dweight = sum over rows of
 * dy * xhat, dbias = sum over rows of dy (either may be null).
 * The input is x, or with x null the checkpoint (codes, scales) of it; mean and
 * rstd are the forward pass's.  dx == dy or dx == x with one stride is allowed.
 * rows = 0 sets dweight and dbias to 0.
 */
size_t rsx_layer_norm_grad_workspace_size(size_t rows, size_t dim);
rsx_status_t rsx_layer_norm_grad(const void* dy, size_t dy_stride, const void* x, size_t x_stride,
                                 const int8_t* codes, const uint8_t* scales, const float* mean,
                                 const float* rstd, const void* weight, void* dx, size_t dx_stride,
                                 void* dweight, void* dbias, size_t rows, size_t dim,
                                 rsx_dtype_t type, rsx_dtype_t weight_type, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream);

/*
 * Activation checkpoints in 8 bits.  Each row is cut into blocks of
 * RSX_CHECKPOINT_BLOCK elements (the last may be shorter).  With 2^E <= m <
 * 2^(E+1) the block's largest magnitude, x is kept as the int8 code
 * q = rint(x / 2^(E-6)), clamped to [-127, 127], and comes back as
 * q * 2^(E-6), rounded to the output's type.  scales holds E - 6 + 127 (0 for
 * blocks below 2^-120); a block with an infinity or a NaN has 255 and comes
 * back as NaN throughout.
 * codes: [rows][dim]; scales: [rows][ceil(dim / RSX_CHECKPOINT_BLOCK)].
 */
#define RSX_CHECKPOINT_BLOCK 32
rsx_status_t rsx_checkpoint_pack(const void* x, size_t x_stride, int8_t* codes, uint8_t* scales,
                                 size_t rows, size_t dim, rsx_dtype_t type, hipStream_t stream);
rsx_status_t rsx_checkpoint_unpack(const int8_t* codes, const uint8_t* scales, void* out,
                                   size_t out_stride, size_t rows, size_t dim, rsx_dtype_t type,
                                   hipStream_t stream);

/*
 * Log probabilities of given tokens.  For each row of logits:
 * lse = log sum exp z; logprob = z[token] - lse (0 for a token outside
 * [0, vocab)); entropy = -sum p log p (may be null); and the `top` largest
 * logits, in order, of equal ones the lower index first (a NaN ranks below
 * every number): top_token[row][k] and top_logprob[row][k], its log probability,
 * the same bits as logprob has for that token.
 * top: 0..min(vocab, RSX_TOP_MAX); with 0 the two arrays may be null.
 * A logit of -inf is masked.  A row with nothing else has lse = -inf, log
 * probabilities of -inf and entropy 0; a row with a NaN or +inf has NaN.
 * The _rest form also keeps lse_rest (`rows` fp32, or null): what the rounding of
 * lse took, so that lse + lse_rest has the digits of log sum exp z whatever its
 * size.  0 where lse is no number.
 */
size_t rsx_token_logprobs_workspace_size(size_t rows, size_t vocab, int top);
rsx_status_t rsx_token_logprobs(const void* logits, size_t stride, rsx_dtype_t type,
                                const void* tokens, rsx_dtype_t token_type, size_t rows,
                                size_t vocab, int top, float* logprob, float* entropy, float* lse,
                                float* top_logprob, int32_t* top_token, void* workspace,
                                size_t workspace_bytes, hipStream_t stream);
rsx_status_t rsx_token_logprobs_rest(const void* logits, size_t stride, rsx_dtype_t type,
                                     const void* tokens, rsx_dtype_t token_type, size_t rows,
                                     size_t vocab, int top, float* logprob, float* entropy,
                                     float* lse, float* lse_rest, float* top_logprob,
                                     int32_t* top_token, void* workspace, size_t workspace_bytes,
                                     hipStream_t stream);

/*
 * Gradient of the log probability and of the entropy in the logits:
 * dlogits[j] = dlogprob * (delta(j, token) - p_j) - dentropy * p_j * (log p_j + entropy),
 * rounded to the logits' type.  lse and entropy are the forward pass's;
 * dentropy may be null (then entropy may be too).  A token outside [0, vocab)
 * has no gradient through its log probability; a row of masked logits alone
 * has a gradient of 0.  dlogits == logits with one stride is allowed.
 * log p_j = z_j - lse, in the _rest form (z_j - lse) - lse_rest.  Without the
 * rest each p is off by lse's rounding, 2^-24 |lse| of itself: little for logits
 * of ordinary size, 1e-3 at 16384, and past 2^24 a row of equal logits has p = 1
 * for each.  lse_rest: as rsx_token_logprobs_rest keeps it, or null.
 */
rsx_status_t rsx_token_logprobs_grad(const void* logits, size_t stride, rsx_dtype_t type,
                                     const void* tokens, rsx_dtype_t token_type, const float* lse,
                                     const float* entropy, const float* dlogprob,
                                     const float* dentropy, void* dlogits, size_t dlogits_stride,
                                     size_t rows, size_t vocab, hipStream_t stream);
rsx_status_t rsx_token_logprobs_grad_rest(const void* logits, size_t stride, rsx_dtype_t type,
                                          const void* tokens, rsx_dtype_t token_type,
                                          const float* lse, const float* lse_rest,
                                          const float* entropy, const float* dlogprob,
                                          const float* dentropy, void* dlogits,
                                          size_t dlogits_stride, size_t rows, size_t vocab,
                                          hipStream_t stream);

/*
 * The step's matrix products: the feed-forward block, the output matrix with
 * its loss, and the orthogonalised update.  Rows, types, aliasing, workspaces
 * and streams as above, with these differences.
 * Sums are held in fp32.  fp32 matrices are multiplied as sums of three bf16
 * values, which hold every bit of values from 2^-100 on; of smaller ones what is
 * below 2^-126 is lost (products of few rows: in fp32).  An infinity gives what
 * it gives in fp32.  Widths (elements of a row but the vocabulary) are below 2^22.
 * Where a 16-bit matrix lies so that its rows are whole 16-byte chunks (address,
 * stride and width multiples of 16 bytes, no stride of 0) it is read in place;
 * from any other a copy is made in the workspace, in every call.  The
 * _workspace_size functions have `copies` for that: 0 if every matrix that the
 * call reads lies so, else 1.  A workspace for 1 is right for 0 too.
 */

/* Activations, in fp32: x / (1 + exp(-x)); x * Phi(x), Phi the normal
 * distribution's; the same by x / (1 + exp(-2 sqrt(2 / pi) (x + 0.044715 x^3)));
 * max(x, 0), with a slope of 0 at 0. */
typedef enum {
  RSX_ACT_SILU = 0,
  RSX_ACT_GELU = 1,
  RSX_ACT_GELU_TANH = 2,
  RSX_ACT_RELU = 3
} rsx_activation_t;

/*
 * Gated feed-forward block: with g = x w_gate^T and u = x w_up^T,
 * out = (act(g) * u) w_down^T.
 * x, out: [rows][dim]; w_gate, w_up: [hidden][dim]; w_down: [dim][hidden].
 * gate, up: [rows][hidden] fp32, dense: g and u for the gradient; or both null.
 * Between the products act(g) * u is rounded to `type` (fp16: infinite beyond 65504),
 * or, where w_down has fewer than 2^18 elements, to the sum of two values of it, with
 * which an infinity in w_down may give a NaN; fp32: kept whole.
 * out overlaps nothing that is read.
 */
size_t rsx_feed_forward_workspace_size(size_t rows, size_t dim, size_t hidden, rsx_dtype_t type,
                                       int copies);
rsx_status_t rsx_feed_forward(const void* x, size_t x_stride, const void* w_gate,
                              size_t gate_stride, const void* w_up, size_t up_stride,
                              const void* w_down, size_t down_stride, void* out, size_t out_stride,
                              float* gate, float* up, size_t rows, size_t dim, size_t hidden,
                              rsx_activation_t activation, rsx_dtype_t type, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);

/*
 * Gradients of rsx_feed_forward for dout, from the gate and up that it kept:
 * ds = dout w_down, dg = ds * up * act'(gate), du = ds * act(gate);
 * dx = dg w_gate + du w_up, dw_gate = dg^T x, dw_up = du^T x and
 * dw_down = dout^T (act(gate) * up), the three added to what is there with
 * `accumulate`.  dx may be null, and so may the three dw together.
 * dg, du and act(gate) * up are rounded to `type` (fp32: kept whole; fp16 keeps
 * nothing below 2^-25 or beyond 65504, so dout is to be scaled to its range).  The
 * dw are of weight_grad_type: `type` or RSX_FLOAT32.
 */
size_t rsx_feed_forward_grad_workspace_size(size_t rows, size_t dim, size_t hidden,
                                            rsx_dtype_t type, int copies);
rsx_status_t rsx_feed_forward_grad(const void* dout, size_t dout_stride, const void* x,
                                   size_t x_stride, const void* w_gate, size_t gate_stride,
                                   const void* w_up, size_t up_stride, const void* w_down,
                                   size_t down_stride, const float* gate, const float* up, void* dx,
                                   size_t dx_stride, void* dw_gate, size_t dw_gate_stride,
                                   void* dw_up, size_t dw_up_stride, void* dw_down,
                                   size_t dw_down_stride, size_t rows, size_t dim, size_t hidden,
                                   rsx_activation_t activation, rsx_dtype_t type,
                                   rsx_dtype_t weight_grad_type, int accumulate, void* workspace,
                                   size_t workspace_bytes, hipStream_t stream);

/*
 * rsx_token_logprobs_rest of the logits scale * hidden weight^T, which are not
 * stored: hidden [rows][dim], weight [vocab][dim] of one type.  The logits are
 * fp32 here.  entropy and lse_rest may be null.  dim = 0: logits of 0.
 */
size_t rsx_linear_logprobs_workspace_size(size_t rows, size_t vocab, size_t dim, rsx_dtype_t type,
                                          int copies);
rsx_status_t rsx_linear_logprobs(const void* hidden, size_t hidden_stride, const void* weight,
                                 size_t weight_stride, rsx_dtype_t type, const void* tokens,
                                 rsx_dtype_t token_type, size_t rows, size_t vocab, size_t dim,
                                 float scale, float* logprob, float* entropy, float* lse,
                                 float* lse_rest, void* workspace, size_t workspace_bytes,
                                 hipStream_t stream);

/*
 * Gradients of rsx_linear_logprobs: with dz as rsx_token_logprobs_grad_rest
 * gives it (lse_rest may be null), times scale, dhidden = dz weight and
 * dweight = dz^T hidden (with `accumulate` added to what is there).  Either may
 * be null.  dweight is of dweight_type: `type` or RSX_FLOAT32.
 * A row whose token is outside [0, vocab) or whose dlogprob is 0, and whose
 * dentropy is 0 or null, has a gradient of 0 and adds nothing to dweight, whatever
 * its values are: NaN and infinities of a batch's padding stay there.
 * dhidden is a product like any other: an infinity that masks a token in the
 * forward pass makes it NaN, being multiplied with a dz of 0.
 * The vocabulary is taken in pieces of 4096 to 2^20 columns, of which the logits
 * are multiplied again; the workspace has dz of all rows for one of them, 2, 4
 * (fp16) or 6 (fp32) bytes each.
 * dz is rounded to bf16, each row by itself divided by its token's dz, and the
 * rows of hidden times that to bf16 too (fp16 matrices: either to 16 bits, with the
 * range of fp32; fp32: kept whole).
 */
size_t rsx_linear_logprobs_grad_workspace_size(size_t rows, size_t vocab, size_t dim,
                                               rsx_dtype_t type, int copies);
rsx_status_t rsx_linear_logprobs_grad(const void* hidden, size_t hidden_stride, const void* weight,
                                      size_t weight_stride, rsx_dtype_t type, const void* tokens,
                                      rsx_dtype_t token_type, const float* lse,
                                      const float* lse_rest, const float* entropy,
                                      const float* dlogprob, const float* dentropy, void* dhidden,
                                      size_t dhidden_stride, void* dweight, size_t dweight_stride,
                                      rsx_dtype_t dweight_type, int accumulate, size_t rows,
                                      size_t vocab, size_t dim, float scale, void* workspace,
                                      size_t workspace_bytes, hipStream_t stream);

/*
 * Orthogonalised updates by Newton-Schulz products, of a stack of `batch`
 * matrices [rows][cols], x_matrix (out_matrix) elements from one to the next (one
 * behind the other, or side by side within a row stride):
 * X = x / (|x| + eps) with the Frobenius norm |x|, then `steps` (at least 1) times
 * A = X X^T, X = a X + (b A + c A A) X; for rows > cols the same of the transpose.
 * out = X, of `type`; out == x with the same strides is allowed.
 * X, A and b A + c A A are held to 22 bits (of an fp32 update whose smaller side
 * is below 128 to 24), with a least step of 2^-36, and products summed in fp32.  Of
 * a bf16 update whose smaller side is 256 or more the last of several steps
 * multiplies 11 bits.  Their values may not pass 16 (the singular values of X begin
 * at 1 or less, and stay below 1.3 with the usual coefficients 3.4445, -4.775, 2.0315).
 * A matrix of zeros gives zeros if eps > 0.  batch is below 2^16.
 */
size_t rsx_newton_schulz_workspace_size(size_t batch, size_t rows, size_t cols);
rsx_status_t rsx_newton_schulz(const void* x, size_t x_stride, size_t x_matrix, void* out,
                               size_t out_stride, size_t out_matrix, size_t batch, size_t rows,
                               size_t cols, int steps, float a, float b, float c, float eps,
                               rsx_dtype_t type, void* workspace, size_t workspace_bytes,
                               hipStream_t stream);

/*
 * First element of segment k in RSX_ALGO_RING all-reduce of `count`
 * elements over `nranks` ranks: min(k * ceil(count/nranks), count).
 * k may be 0..nranks (k = nranks gives count).  Returns 0 for nranks < 1.
 */
size_t rsx_segment_begin(size_t count, int nranks, int k);

/* Size in bytes of one element of `dtype`, 0 if it is not a valid dtype. */
size_t rsx_dtype_size(rsx_dtype_t dtype);

/* Static description of a status; for RSX_ERR_HIP the calling thread's last
 * HIP error text.  Never NULL. */
const char* rsx_status_string(rsx_status_t status);

/* RSX_VERSION of the built library. */
int rsx_version(void);

/*
 * Occupancy caps of the calling thread's launches; returns the previous
 * setting (1 on, 0 off).  On by default: the dwordx4 reduction and gather
 * kernels then reserve LDS they do not use, so that fewer of their
 * workgroups share a CU, which keeps HBM busiest when a collective runs by
 * itself (W = 8 reduce-scatter 378 -> 361 us, one-pass all-reduce
 * 769 -> 735 us).  Reserved LDS also keeps other kernels off those CUs:
 * turn the caps off for launches meant to overlap compute on another stream
 * (bucketed all-reduce beside a matmul per bucket: 1,371 us with the caps,
 * 1,185 us without).  Results are the same either way.  Host state only.
 */
int rsx_set_occupancy_caps(int enable);

#ifdef __cplusplus
}
#endif

#endif /* RSX_H */
