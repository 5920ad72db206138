/*
 * grz.h -- C ABI of libgrz, the data-parallel / ZeRO-1 gradient pipeline on
 * one AMD Instinct MI355X (gfx950).
 *
 * One step of the pipeline, for N ranks whose gradients sit in N flat arenas:
 *
 *   dp_reduce_scatter_mean   ring-order average of the ranks' gradients
 *   dp_grad_sqnorm           global squared norm and clip factor
 *   dp_grad_sqnorm_of        the same, straight from an fp32 gradient array
 *   zero1_adamw_step         clipped AdamW on the owned shard (+ bf16 copy,
 *                            optionally written straight into the replicas)
 *   zero1_all_gather         owned bf16 shards into every replica arena
 *   dp_all_gather            the same for fp32 / fp64 / bf16 shards (the
 *                            second half of a plain all-reduce)
 *   zero1_fused_step         the four above for one shard in one launch
 *
 * and the operators addressed by token ids, at the two ends of that arena (the
 * embedding table and the loss over the vocabulary):
 *
 *   dp_embed_lookup          scaled rows of the table in a weight arena
 *   dp_embed_grad            its gradient, into a gradient arena
 *   dp_token_logprobs        log probability of given tokens, entropy, top list
 *   dp_token_logprobs_grad   its gradient
 *   dp_distill_loss          loss against a teacher's top logits
 *   dp_distill_grad          its gradient
 *
 * the operators of a mixture of experts between them:
 *
 *   dp_expert_route          a token's experts and their weights
 *   dp_expert_route_grad     the gradient of the weights, to the router's logits
 *   dp_expert_sort           the tokens' slots sorted by expert
 *   dp_expert_dispatch       the tokens' rows in that order
 *   dp_expert_combine        rows back to their tokens, summed with the weights
 *   dp_expert_combine_grad   gradient of that sum
 *
 * and the norm and the clip for gradients that are tensors of their own, beside
 * the arena (a rank's experts) or in its place:
 *
 *   dp_grad_sqnorm_tensors   squared norm and clip factor over many tensors
 *   dp_grad_clip_tensors     the tensors scaled by the factor
 *
 * Sources: "Lab 09 -- Parallelism, simulated" s.1 "Ring all-reduce" (the
 * N = 3 schedule table; "Tips": in reduce-scatter step t rank r sends chunk
 * (r - t) mod N and ends owning chunk (r + 1) mod N) and s.2 (sum, then
 * divide by N); "A4 -- Multi-GPU with NCCL and ZeRO-1", "Part 2 -- Tensor
 * Sharding", "Part 3 -- Gradient Reduction" (reduce-scatter with ncclAvg),
 * "Part 4 -- Multi-GPU Backward and Update" (AdamW only on the shard, then
 * all-gather); "Distributed training" (noeira), "Four strategies, one
 * interface" (clip_grads_device, step; one flat arena per replica) and "The
 * process group" (every rank simulated on one device).
 *
 * Conventions shared by every entry point:
 *
 *  - Memory.  Every pointer named "device" is HIP device memory owned by the
 *    caller; the library allocates nothing and keeps no state between calls
 *    (apart from the per-thread grid cap of grz_set_max_blocks, which never
 *    changes a result, and the static per-device scratch of
 *    dp_grad_sqnorm_noalloc), so concurrent calls on different streams are
 *    safe when they touch disjoint buffers.  Buffers must stay alive until
 *    the stream has run the enqueued work.  Host arrays (pointer tables, bucket lists, argument
 *    structs) are read during the call only.
 *  - Streams.  Work is enqueued on `stream` (0 = the null stream).  No entry
 *    point synchronises the host: results are ready when the stream is.
 *  - Errors.  Arguments are checked before anything is enqueued; on a bad
 *    argument nothing is launched and a GRZ_E* code is returned (see
 *    grz_strerror).  A launch failure reported by HIP returns GRZ_EHIP.
 *  - Buckets.  A bucket is a contiguous element range [offset, offset +
 *    length) of the arena; buckets are listed in processing order (reverse
 *    layer order: "Distributed training", "Overlap and graphs", plan_buckets;
 *    "A4", "Part 4": the backward pass produces the last layer first).
 *    Chunk c of a bucket is its c-th piece under the numpy.array_split rule
 *    (the first length % N chunks are one element longer).
 *  - Shards.  The ZeRO-1 shard of chunk c is chunk c of every bucket,
 *    concatenated in processing order ("shard-compact" layout).  Rank r owns
 *    chunk (r + 1) mod N.  Unless GRZ_UNEVEN is given, every bucket length
 *    must be divisible by N (an uneven count is an error in "Part 2 --
 *    Tensor Sharding"), else GRZ_EINDIVISIBLE.
 *  - Pieces.  The norm is summed over pieces of GRZ_PIECE consecutive
 *    elements of one chunk (the last piece of a chunk may be shorter).  The
 *    pieces of a plan are numbered bucket by bucket, chunk 0..N-1 within a
 *    bucket, piece by piece within a chunk; dp_piece_count gives their
 *    number and dp_piece_offset where a (bucket, chunk) starts.  The same
 *    pieces, hence the same norm bits, come out of a ZeRO-1 and a plain
 *    data-parallel run of the same plan.
 *  - Arithmetic.  bf16 and fp32 gradients are summed in fp32, fp64 ones in
 *    fp64, one rounding per addition, in ring order; the mean is one IEEE
 *    division by N.  AdamW runs in fp32 with every operation rounded on its
 *    own (no fused multiply-add) and correctly rounded division and square
 *    root.  bf16 outputs are round-to-nearest-even of the fp32 master.
 */
#ifndef GRZ_H
#define GRZ_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
enum {
  GRZ_OK = 0,
  GRZ_EINVAL = 1,        /* null pointer, bad count, bad dtype, bad flag, ... */
  GRZ_EINDIVISIBLE = 2,  /* a bucket length is not divisible by N            */
  GRZ_EALIGN = 3,        /* a device pointer is not aligned to its element   */
  GRZ_EHIP = 4,          /* HIP reported an error when launching             */
  GRZ_ERANGE = 5         /* a bucket leaves the arena or a size is too large */
};

/* Gradient element types. */
enum { GRZ_F32 = 0, GRZ_BF16 = 1, GRZ_F64 = 2 };

/* Flags.  An entry point returns GRZ_EINVAL for a flag it does not take:
 * the reduce (dp_reduce_scatter_mean and its _range form) takes all but
 * GRZ_ARGS_DEVICE and GRZ_COOPERATIVE, the _weighted form all but those and
 * GRZ_SUM; zero1_adamw_gather takes GRZ_UNEVEN, GRZ_ARGS_DEVICE and
 * GRZ_MEAN_BF16; the
 * all-gathers take GRZ_UNEVEN; zero1_fused_step GRZ_UNEVEN, GRZ_IN_COMPACT,
 * GRZ_ARGS_DEVICE and GRZ_COOPERATIVE; dp_embed_grad and dp_expert_combine
 * GRZ_ACCUMULATE; dp_expert_route and its gradient GRZ_NORMALIZE.  Their
 * meaning is in each entry point's comment. */
enum {
  GRZ_SUM = 1,        /* keep the sum: skip the division by N            */
  GRZ_UNEVEN = 2,     /* allow bucket lengths not divisible by N         */
  GRZ_IN_COMPACT = 4, /* rank inputs hold only the reduced chunk, compact */
  GRZ_BF16_WIRE = 8,  /* bf16 gradients: round every partial sum to bf16  */
  GRZ_IN_RANGE = 16,  /* rank inputs hold only the reduced bucket range     */
  GRZ_ARGS_DEVICE = 32, /* zero1_adamw_gather: `args` is a device pointer   */
  GRZ_OUT_GLOBAL = 64,  /* reduce, chunk >= 0: mean_out indexed like the arena */
  GRZ_IN_TILED = 128,   /* with GRZ_IN_COMPACT: one receive buffer, the N ranks'
                           values of each piece side by side               */
  GRZ_MEAN_BF16 = 256,  /* the mean (gradient shard) is held in bf16         */
  GRZ_COOPERATIVE = 512, /* zero1_fused_step: a cooperative launch           */
  GRZ_ACCUMULATE = 1024, /* dp_embed_grad, dp_expert_combine: add to what the
                            output holds                                    */
  GRZ_NORMALIZE = 2048  /* dp_expert_route: the listed weights sum to 1       */
};

#define GRZ_MAX_RANKS 16    /* N and the number of replicas per call       */
#define GRZ_PIECE 4096      /* elements per norm piece                      */
#define GRZ_MAX_TOP 128     /* longest top list of a row                    */
#define GRZ_MAX_EXPERTS 1024 /* experts of a mixture                         */
#define GRZ_MAX_SLOTS 32    /* experts a token goes to                      */

typedef struct {
  int64_t offset; /* first element of the bucket in the arena */
  int64_t length; /* elements in the bucket                   */
} grz_bucket;

/* Per-step AdamW scalars, all fp32.  bias_corr1/2 are 1 - beta1^t and
 * 1 - beta2^t for the step t (starting at 1), evaluated by the caller. */
typedef struct {
  float lr;
  float beta1;
  float beta2;
  float eps;
  float weight_decay;
  float bias_corr1;
  float bias_corr2;
} grz_adamw_args;

/* A tensor of a list: `numel` consecutive elements (GRZ_F32 or GRZ_BF16) in
 * device memory, at any element's address. */
typedef struct {
  void* data;
  int64_t numel;
  int dtype;
} grz_tensor;

/* Version of the ABI (major * 100 + minor). */
int grz_version(void);

/* Launch-width knob: the largest grid (workgroups) the grid-stride kernels
 * use; the default, 2^30, means one workgroup per tile (4096 elements and
 * 256 threads for the reduce, 512 and 64 for the all-gather, 256 and 64 for
 * the optimizer).
 * It changes speed only; the piece layout, the fold order and the norm tree,
 * hence every result bit, do not depend on it.  It applies to the calls the
 * calling host thread makes afterwards (each thread has its own value,
 * starting at 2^30), so callers on other threads never see it.  GRZ_EINVAL
 * outside 1..2^30. */
int grz_set_max_blocks(int blocks);

/* Static description of a status code; never NULL. */
const char* grz_strerror(int status);

/* Chunk rank `rank` owns after the ring reduce-scatter: (rank + 1) mod N
 * ("Lab 09", s.1, the "owns" row; "Tips").  -1 on a bad argument. */
int dp_ring_owned_chunk(int rank, int nranks);

/* Rank that owns chunk `chunk`: (chunk - 1) mod N.  -1 on a bad argument. */
int dp_ring_chunk_owner(int chunk, int nranks);

/* Range of chunk `chunk` of a bucket of `length` elements split over N
 * (array_split rule): *offset within the bucket and *count elements. */
int dp_chunk_range(int64_t length, int nranks, int chunk, int64_t* offset, int64_t* count);

/* Number of norm pieces of a plan over all N chunks of every bucket, or a
 * negative GRZ_E* code. */
int64_t dp_piece_count(const grz_bucket* buckets, int nbuckets, int nranks, int flags);

/* Index of the first piece of chunk `chunk` of bucket `bucket`, or a
 * negative GRZ_E* code. */
int64_t dp_piece_offset(const grz_bucket* buckets, int nbuckets, int nranks, int flags,
                        int bucket, int chunk);

/* Elements of the ZeRO-1 shard of chunk `chunk` (sum over buckets of the
 * chunk's length), or a negative GRZ_E* code. */
int64_t dp_shard_numel(const grz_bucket* buckets, int nbuckets, int nranks, int chunk,
                       int flags);

/* Elements of the GRZ_IN_TILED receive buffer of chunk `chunk`: the chunk's
 * pieces (GRZ_PIECE elements each, the last piece of each bucket's chunk
 * possibly shorter) times N times GRZ_PIECE, or a negative GRZ_E* code. */
int64_t dp_tiled_numel(const grz_bucket* buckets, int nbuckets, int nranks, int chunk,
                       int flags);

/*
 * Ring-order reduce-scatter-mean ("Lab 09", s.1 and "Tips"; "A4", "Part 3",
 * ncclReduceScatter / ncclAllReduce with ncclAvg).
 *
 * rank_grads  host array of N device pointers: rank j's flat gradient arena
 *             of `dtype` elements.  With GRZ_IN_COMPACT, rank j's values of
 *             chunk `chunk` only, in shard-compact layout (what arrives over
 *             the wire for one owner).  With GRZ_IN_COMPACT | GRZ_IN_TILED,
 *             the N ranks' values arrive in one receive buffer of
 *             dp_tiled_numel elements: number the chunk's pieces k = 0, 1, ...
 *             in plan order (bucket by bucket, GRZ_PIECE elements each, the
 *             last piece of each bucket's chunk possibly shorter); rank j's
 *             values of piece k start at element (k * N + j) * GRZ_PIECE
 *             (the rest of a short piece's slot is not read).  rank_grads[j]
 *             must then be the buffer + j * GRZ_PIECE elements (GRZ_EINVAL
 *             otherwise).  A tile's loads are then one contiguous run instead
 *             of N runs in N buffers, which MI355X's HBM streams faster (the
 *             7B share's reduce 2.62-2.65 ms against 2.76-2.77 ms); the
 *             results are the same bits.
 * nranks      N, 1..GRZ_MAX_RANKS.
 * dtype       GRZ_F32, GRZ_BF16 (uint16 bit patterns) or GRZ_F64.
 * buckets     host array of `nbuckets` (1..) buckets in processing order.
 * chunk       0..N-1: reduce that chunk of every bucket (ZeRO-1; mean_out is
 *             shard-compact, dp_shard_numel elements).  -1: reduce every
 *             chunk (plain data parallelism; mean_out is indexed like the
 *             arena and only bucket ranges are written).
 * flags       GRZ_SUM, GRZ_UNEVEN, GRZ_IN_COMPACT (needs chunk >= 0),
 *             GRZ_IN_TILED (needs GRZ_IN_COMPACT),
 *             GRZ_OUT_GLOBAL (chunk >= 0: mean_out is indexed like the arena
 *             and only the chunk's ranges are written -- the reduce-scatter
 *             half of a plain all-reduce, whose all-gather half, dp_all_gather,
 *             brings the other chunks; no effect with chunk -1),
 *             GRZ_BF16_WIRE (needs GRZ_BF16): the ring's wire format is bf16,
 *             so every partial sum of the fold -- the last one included -- is
 *             rounded to bf16 (nearest even) before the next rank adds to it
 *             ("13.5 Multi-GPU from First Principles", exercise 8); the mean
 *             is that bf16 sum divided by N in fp32.
 *             GRZ_MEAN_BF16 (F32 or BF16 input): the owner holds its gradient
 *             shard in bf16, as "Lab 09", s.4 counts a ZeRO-2 rank's bytes
 *             (2 per parameter, divided by N): the fp32 mean is rounded once
 *             to bf16 (nearest even) and written as uint16 bit patterns.
 * mean_out    device; fp32 for F32/BF16 input (uint16 bf16 patterns with
 *             GRZ_MEAN_BF16), fp64 for F64 input.
 * piece_sqnorm device fp64 array of dp_piece_count elements, or NULL.  The
 *             slots of the reduced chunks receive the sum of squares of the
 *             piece's output values (with GRZ_MEAN_BF16, of the rounded
 *             values); other slots are left untouched.
 *
 * Element c-th chunk value = (((g_c + g_{c+1}) + g_{c+2}) + ... + g_{c-1}) / N
 * with rank indices mod N: the sum starts at rank c and travels the ring.
 */
int dp_reduce_scatter_mean(const void* const* rank_grads, int nranks, int dtype,
                           const grz_bucket* buckets, int nbuckets, int chunk, int flags,
                           void* mean_out, double* piece_sqnorm, hipStream_t stream);

/*
 * dp_reduce_scatter_mean restricted to buckets [bucket_first, bucket_first +
 * bucket_count) of the plan: the call a bucket-overlapped backward issues as
 * each bucket's gradients become ready ("A4", "Part 3": the reduction runs
 * on its own stream, ordered after the compute stream by an event; "Lab 09",
 * s.2, and "Distributed training", "Overlap and graphs": each bucket is
 * reduced as soon as backward has produced it).  Shard-compact offsets,
 * arena offsets, piece numbers and GRZ_IN_TILED slots are those of the whole
 * plan (only the range's slots are read), so reducing
 * the buckets one call at a time, in any order, leaves exactly the bytes one
 * call over the whole plan leaves.  GRZ_EINVAL if the range leaves the plan.
 *
 * With GRZ_IN_RANGE (not with GRZ_IN_COMPACT), rank_grads[j] holds only the
 * range: arena element i is at index i - lo, lo the lowest offset of the
 * range's buckets.  This is how a ZeRO-2 backward feeds the reduction from a
 * staging buffer the size of one bucket instead of a full gradient arena
 * ("Lab 09", s.4, stage 2 shards the gradients too; "Distributed training",
 * "Four strategies, one interface", ZeroSharded[2]).
 */
int dp_reduce_scatter_mean_range(const void* const* rank_grads, int nranks, int dtype,
                                 const grz_bucket* buckets, int nbuckets, int bucket_first,
                                 int bucket_count, int chunk, int flags, void* mean_out,
                                 double* piece_sqnorm, hipStream_t stream);

/*
 * Token-weighted reduce-scatter for shards of unequal size ("Lab 09", s.2:
 * with variable-length sequences, sum the per-token losses and divide by the
 * global token count; "13.5 Multi-GPU from First Principles", exercise 2:
 * averaging the shards' means weights a token by the size of its shard, and
 * the exact recipe needs the token counts exchanged before the update).
 *
 * rank_grads[j] holds rank j's gradient SUMMED over its own tokens (not
 * divided); token_counts (host, N entries >= 0) are the ranks' token counts.
 * The library adds the counts (the one extra scalar all-reduce) and computes
 * (ring-order sum) / total, one IEEE division, total <= 2^24 (GRZ_ERANGE
 * above, so that it is an exact fp32).  Everything else is
 * dp_reduce_scatter_mean_range; GRZ_SUM is refused.
 */
int dp_reduce_scatter_weighted(const void* const* rank_grads, const int64_t* token_counts,
                               int nranks, int dtype, const grz_bucket* buckets, int nbuckets,
                               int bucket_first, int bucket_count, int chunk, int flags,
                               void* mean_out, double* piece_sqnorm, hipStream_t stream);

/* Bytes of workspace dp_grad_sqnorm needs for `npieces` pieces (may be 0). */
size_t dp_grad_sqnorm_workspace(int64_t npieces);

/*
 * Global squared norm and clip factor ("Distributed training",
 * clip_grads_device(max_norm): clipping stays on the device).
 *
 * piece_sqnorm  device fp64, `npieces` partial sums in piece order.
 * max_norm      clip threshold; <= 0 disables clipping (factor 1).
 * workspace     device, dp_grad_sqnorm_workspace(npieces) bytes (NULL if 0).
 * sqnorm_out    device fp64 scalar: the pieces summed in a fixed tree order
 *               that depends only on npieces.
 * clip_scale_out device fp32 scalar: fp32(max_norm / sqrt(sqnorm)) when
 *               sqrt(sqnorm) > max_norm, else 1.
 */
int dp_grad_sqnorm(const double* piece_sqnorm, int64_t npieces, double max_norm,
                   void* workspace, double* sqnorm_out, float* clip_scale_out,
                   hipStream_t stream);

/*
 * dp_grad_sqnorm without a workspace argument and without allocating, for
 * callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc).  The tree's middle
 * levels go to a static array of GRZ_NOALLOC_SCRATCH_BYTES per device, which
 * the library holds until the process ends; its device address is looked up
 * on the first call on each device (the device current when the call is made,
 * which must be the stream's).  Same arguments, results (bit for bit) and
 * errors as dp_grad_sqnorm, plus GRZ_ERANGE when
 * dp_grad_sqnorm_workspace(npieces) exceeds GRZ_NOALLOC_SCRATCH_BYTES (more
 * than 33,546,240 pieces, about 1.4e11 gradient elements) and GRZ_EINVAL when
 * a non-null stream belongs to another device than the current one.  Nothing
 * needs clearing between calls: each call writes every scratch value it
 * reads.  All calls on one device share the array, so calls that overlap on
 * one device (different streams, or different host threads) race: order them.
 */
#define GRZ_NOALLOC_SCRATCH_BYTES 65536
int dp_grad_sqnorm_noalloc(const double* piece_sqnorm, int64_t npieces, double max_norm,
                           double* sqnorm_out, float* clip_scale_out, hipStream_t stream);

/*
 * dp_grad_sqnorm, and in its last launch the work of grz_step_args_next:
 * *current = table[min(*counter, count - 1)]; *counter += 1 (all device
 * memory).  A captured step ("Distributed training", "Overlap and graphs": one
 * graph per GPU, replayed) needs both before its optimizer runs; done by the
 * norm's single-workgroup launch they cost one launch fewer per replay.
 * Arguments and errors as dp_grad_sqnorm and grz_step_args_next.
 */
int dp_grad_sqnorm_step_args(const double* piece_sqnorm, int64_t npieces, double max_norm,
                             void* workspace, double* sqnorm_out, float* clip_scale_out,
                             const grz_adamw_args* table, int64_t count, int64_t* counter,
                             grz_adamw_args* current, hipStream_t stream);

/* Bytes of workspace dp_grad_sqnorm_of needs for `n` gradient elements. */
size_t dp_grad_sqnorm_of_workspace(int64_t n);

/*
 * dp_grad_sqnorm over a plain fp32 gradient array that is already reduced
 * (one chunk of one bucket): the library forms the piece sums itself, pieces
 * of GRZ_PIECE consecutive elements summed exactly as dp_reduce_scatter_mean
 * sums them, then combines them in the same tree.  So the result equals, bit
 * for bit, dp_reduce_scatter_mean of a single rank (N = 1, one bucket of `n`
 * elements) followed by dp_grad_sqnorm ("Distributed training",
 * clip_grads_device(max_norm) on a flat fp32 arena).
 *
 * grad          device fp32, `n` elements (any 4-byte alignment).
 * workspace     device, dp_grad_sqnorm_of_workspace(n) bytes, 8-byte aligned;
 *               on return it holds the ceil(n / GRZ_PIECE) piece sums first.
 * sqnorm_out, clip_scale_out, max_norm  as for dp_grad_sqnorm (either output
 *               may be NULL, not both).
 * Errors: GRZ_EINVAL for a NULL grad/workspace with n > 0, both outputs NULL
 * or n < 0; GRZ_EALIGN; GRZ_ERANGE beyond 4096^3 pieces.
 */
int dp_grad_sqnorm_of(const float* grad, int64_t n, double max_norm, void* workspace,
                      double* sqnorm_out, float* clip_scale_out, hipStream_t stream);

/*
 * Clipped AdamW on one rank's shard ("A4", "Part 4": adamw_update only for
 * this rank's shard; "Distributed training", step()).
 *
 * master, m, v  device fp32, `n` elements each, updated in place.
 * mean_grad     device fp32, `n` elements (dp_reduce_scatter_mean output).
 * clip_scale    device fp32 scalar (dp_grad_sqnorm output) or NULL for 1.
 * args          host, the step's scalars.
 * bf16_out      device uint16, `n` elements of RNE_bf16(new master), or NULL.
 *
 * Per element: g = mean*scale; m = b1*m + (1-b1)*g; v = b2*v + (1-b2)*(g*g);
 * master -= lr*((m/bc1) / (sqrt(v/bc2) + eps) + wd*master).
 */
int zero1_adamw_step(float* master, float* m, float* v, const float* mean_grad, int64_t n,
                     const float* clip_scale, const grz_adamw_args* args, uint16_t* bf16_out,
                     hipStream_t stream);

/*
 * zero1_adamw_step with the all-gather fused into its epilogue: the new bf16
 * weights of the shard of chunk `chunk` go straight to their arena offsets in
 * every replica (no shard-compact bf16 round trip).  The shard geometry is
 * (buckets, nbuckets, nranks, chunk, flags) as in dp_reduce_scatter_mean;
 * chunk -1 means the whole plan in arena indexing (plain data parallelism:
 * master, m, v and mean_grad are then indexed like the arena).
 *
 * mean_grad  device; fp32 values, or with GRZ_MEAN_BF16 the bf16 patterns
 *            the reduce wrote with that flag (each widened exactly to fp32
 *            before the clip factor multiplies it).
 * replicas   host array of `nreplicas` (0..GRZ_MAX_RANKS) device uint16
 *            arenas.
 * flags      GRZ_UNEVEN; GRZ_MEAN_BF16; GRZ_ARGS_DEVICE: `args` points to
 *            device memory and is read by the kernel when it runs, so that a
 *            captured step (HIP graph) can be replayed with each step's
 *            scalars ("Distributed training", "Overlap and graphs": one graph
 *            per GPU, replayed).
 */
int zero1_adamw_gather(float* master, float* m, float* v, const void* mean_grad,
                       const grz_bucket* buckets, int nbuckets, int nranks, int chunk,
                       int flags, const float* clip_scale, const grz_adamw_args* args,
                       uint16_t* const* replicas, int nreplicas, hipStream_t stream);

/*
 * Enqueue: *current = table[min(*counter, count - 1)]; *counter += 1.  All
 * three are device pointers; `table` holds the per-step scalars of steps
 * 1..count (row t-1 for step t) and `*counter` the next row.  Placed in front
 * of a zero1_adamw_gather(..., GRZ_ARGS_DEVICE, current, ...) inside a
 * captured step, it advances the step scalars on every replay.
 */
int grz_step_args_next(const grz_adamw_args* table, int64_t count, int64_t* counter,
                       grz_adamw_args* current, hipStream_t stream);

/*
 * All-gather of bf16 shards ("Lab 09", s.1, all-gather rows of the N = 3
 * table; "A4", "Part 4", ncclAllGather after the update).
 *
 * shards     host array of N entries: shards[r] is rank r's shard-compact
 *            bf16 shard (chunk (r + 1) mod N of every bucket) on the device,
 *            or NULL for a rank whose shard is already in place.
 * replicas   host array of `nreplicas` device uint16 arenas; every non-NULL
 *            shard is copied into each of them at its arena offsets.
 */
int zero1_all_gather(const uint16_t* const* shards, int nranks, const grz_bucket* buckets,
                     int nbuckets, int flags, uint16_t* const* replicas, int nreplicas,
                     hipStream_t stream);

/*
 * zero1_all_gather for shards of any element type: GRZ_BF16 (2 bytes),
 * GRZ_F32 (4) or GRZ_F64 (8).  With fp32 shards it is the all-gather half of
 * a plain all-reduce of the mean ("Lab 09", s.1: an all-reduce is a
 * reduce-scatter followed by an all-gather; "A4", "Part 3", ncclAllReduce):
 * rank r's mean of chunk (r + 1) mod N, from dp_reduce_scatter_mean, lands at
 * its arena offsets in every replica.  The copy is of bytes: the values
 * arrive unchanged.  shards[r] is shard-compact (dp_shard_numel elements) or
 * NULL; replicas are arenas of `dtype` elements.  Errors as zero1_all_gather,
 * plus GRZ_EINVAL for another dtype and GRZ_EALIGN for a pointer not aligned
 * to its element.
 */
int dp_all_gather(const void* const* shards, int nranks, int dtype, const grz_bucket* buckets,
                  int nbuckets, int flags, void* const* replicas, int nreplicas,
                  hipStream_t stream);

/* Bytes of workspace zero1_fused_step needs for a plan of `npieces` pieces. */
size_t zero1_fused_workspace(int64_t npieces);

/*
 * Pieces (GRZ_PIECE-element tiles of the reduced chunks) that one
 * zero1_fused_step launch can hold for N ranks of `dtype` gradients on the
 * current device: 4 per workgroup that can be resident at once, less one
 * workgroup that folds the norm (1024 resident on a 256-CU MI355X, so 4092
 * pieces, 16.76 M elements).  A plan of more than 4096 pieces in all (the
 * peers' included) takes one more folding workgroup per 4096 pieces, so 4
 * pieces less each.  A negative value is minus a GRZ_E* code.
 */
int64_t zero1_fused_capacity(int nranks, int dtype);

/*
 * The whole step of one shard in one launch: reduce-scatter-mean, global
 * norm, clip, AdamW and the bf16 write ("A4", "Part 4": reduce, update the
 * shard, all-gather; "Distributed training", "Four strategies, one
 * interface": clip_grads_device then step), for a shard small enough that
 * its mean stays in registers.  Every result is bit-identical to
 *   dp_reduce_scatter_mean -> dp_grad_sqnorm -> zero1_adamw_gather
 * on the same inputs; the mean itself is never stored unless `mean_out` is
 * given, which saves 8 bytes of memory traffic per owned element.  The grid
 * synchronises internally (all pieces summed before the norm is read: each
 * piece sum is published in a workspace slot that carries the launch's
 * parity, and the readers poll it), so its workgroups must be resident at
 * once.  The grid is sized to what the occupancy allows resident, so on a
 * device that runs nothing else at the same time they are; with
 * GRZ_COOPERATIVE the launch is cooperative and HIP guarantees it (or
 * refuses the launch), at about 17 us more per call on MI355X.  Without it,
 * kernels of other streams that hold compute units for longer than the
 * poll limit make the waits give up (see `workspace`): the call then
 * reports it and no tile holds anything but its old state or its update.
 *
 * rank_grads, nranks, dtype, buckets, nbuckets, chunk
 *            as for dp_reduce_scatter_mean; dtype GRZ_BF16 or GRZ_F32.
 *            chunk >= 0: one rank's ZeRO-1 shard (master/m/v and mean_out
 *            shard-compact); chunk = -1: every chunk (plain data parallelism,
 *            master/m/v indexed like the arena).
 * flags      GRZ_UNEVEN, GRZ_IN_COMPACT (as for the reduce), GRZ_ARGS_DEVICE
 *            (as for zero1_adamw_gather), GRZ_COOPERATIVE (above).
 *            GRZ_BF16_WIRE, GRZ_SUM, GRZ_IN_TILED and GRZ_MEAN_BF16 are not
 *            taken (GRZ_EINVAL): use the separate entry points.
 * master, m, v  device fp32 state, updated in place.
 * args       the step's scalars (host, or device with GRZ_ARGS_DEVICE).
 * max_norm   clip threshold (<= 0: no clipping).
 * replicas   host array of `nreplicas` device bf16 arenas (0..16); each gets
 *            the new weights of the processed chunks at their arena offsets.
 * piece_sqnorm device fp64, dp_piece_count entries.  The kernel writes the
 *            pieces of the processed chunks; the other entries (the peers'
 *            pieces, when chunk >= 0) must hold their values already.
 * workspace  device, zero1_fused_workspace(npieces) bytes, 8-byte aligned,
 *            ZEROED before its first use.  Its first 256 bytes are control
 *            words: the 32-bit word at byte 8 is the time-out flag, the word
 *            at byte 12 the number of polls a wait makes before it gives up
 *            (0, as zeroed: 2^22, a few seconds; the caller may set it
 *            before the launch), the words at bytes 16 and 20 a launch
 *            counter and the piece count of the last launch.  The rest holds
 *            the published piece sums.  A completed call leaves the workspace
 *            ready for the next call of a plan with the same piece count; a
 *            call with another piece count raises the flag and writes
 *            nothing.  A non-zero flag means a wait gave up (or the piece
 *            count changed): a workgroup whose wait gave up writes nothing
 *            after it (its tiles of master, m, v, the replicas and the mean
 *            keep their previous values, and it stores no norm), so each tile
 *            holds either its previous state or its correct update; the
 *            call's result as a whole is then incomplete, and while the flag
 *            is up every further call on the workspace returns at once
 *            without writing anything.  Zero the workspace (the poll limit
 *            word may be kept) before the next call.  Calls that share a
 *            workspace must not overlap.  The peers' entries of piece_sqnorm
 *            are sums of squares: non-negative (a NaN is carried as NaN).
 * sqnorm_out, clip_scale_out  device scalars as for dp_grad_sqnorm, or NULL.
 * mean_out   device fp32 copy of the mean (as dp_reduce_scatter_mean writes
 *            it), or NULL.
 * Errors: as dp_reduce_scatter_mean and zero1_adamw_gather; GRZ_ERANGE when
 * the plan has more pieces than zero1_fused_capacity (less its folding
 * workgroups), more than 32 (bucket, chunk) segments, or more than 2^20
 * pieces in all; GRZ_EHIP when the launch fails (with GRZ_COOPERATIVE, also
 * when the device cannot launch cooperatively).
 */
int zero1_fused_step(const void* const* rank_grads, int nranks, int dtype,
                     const grz_bucket* buckets, int nbuckets, int chunk, int flags,
                     float* master, float* m, float* v, const grz_adamw_args* args,
                     double max_norm, uint16_t* const* replicas, int nreplicas,
                     double* piece_sqnorm, void* workspace, double* sqnorm_out,
                     float* clip_scale_out, float* mean_out, hipStream_t stream);

/*
 * zero1_fused_step whose step scalars come from a table and advance in the
 * same launch, for a captured step replayed once per step ("Distributed
 * training", "Overlap and graphs": one graph per GPU, replayed): the launch
 * uses row min(*counter, count - 1) of `table` (rows as for
 * grz_step_args_next), copies it to *current and adds one to *counter, as
 * grz_step_args_next followed by zero1_fused_step with GRZ_ARGS_DEVICE would,
 * without the extra launch.  table, counter and current are device pointers;
 * GRZ_ARGS_DEVICE is implied (passing it: GRZ_EINVAL).  A call refused at its
 * start (the workspace's flag up, or another piece count; see
 * zero1_fused_step) leaves the counter as it was; after a wait gave up it
 * may have advanced (workgroup 0 advances it once it has the norm).
 * Everything else is zero1_fused_step.
 */
int zero1_fused_step_args(const void* const* rank_grads, int nranks, int dtype,
                          const grz_bucket* buckets, int nbuckets, int chunk, int flags,
                          float* master, float* m, float* v, const grz_adamw_args* table,
                          int64_t count, int64_t* counter, grz_adamw_args* current,
                          double max_norm, uint16_t* const* replicas, int nreplicas,
                          double* piece_sqnorm, void* workspace, double* sqnorm_out,
                          float* clip_scale_out, float* mean_out, hipStream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Operators addressed by token ids ("Distributed training" (noeira), "Four
 * strategies, one interface": weights and gradients are flat arenas; these
 * read the embedding table in the one and fill its gradient in the other, and
 * form the loss whose per-token weights dp_reduce_scatter_weighted averages).
 *
 * Shared conventions:
 *
 *  - Row matrices.  `rows` x `cols` values of GRZ_F32 or GRZ_BF16, row r at
 *    data + r * stride elements (stride >= cols), aligned to its element: a
 *    tensor at any place of an arena.  Rows on 16-byte borders are fastest.
 *    Elements between cols and stride are neither read nor written.
 *  - Ids.  int32 (id_bits 32) or int64 (id_bits 64) device arrays.  An id
 *    outside [0, vocab) names no row (padding, ignored targets).
 *  - Sizes.  At most 2^31 - 1 rows and columns, further limits at the entry
 *    points; beyond them GRZ_ERANGE.  Calls with n = 0 do nothing (dp_embed_grad
 *    still zeroes its table).
 *  - Arithmetic.  Every sum, maximum and exponential in fp32; each output is
 *    rounded once to its type (bf16: nearest even).  The same call on the same
 *    values gives the same bits; the order of a vocabulary row's sums follows
 *    its place on the 16-byte borders, so another layout may round otherwise.
 *  - Errors, beside each entry point's own: GRZ_EINVAL for a null pointer, a
 *    type or flag that is not taken, or an output (or workspace) that overlaps
 *    an input or another output (two matrices do if their spans, first to last
 *    element, do); GRZ_EALIGN; GRZ_ERANGE.  Two overlaps are taken: dlogits
 *    that are the logits, and a logprob, entropy or loss array that is the same
 *    array as glogprob, gentropy or weights.
 */

/*
 * out[i] = scale * table[ids[i]], a row of zeros where the id names no row.
 *
 * table  device, vocab x dim; out  device, n x dim; any of the two types each.
 */
int dp_embed_lookup(const void* table, int table_dtype, int64_t vocab, int64_t dim,
                    int64_t table_stride, const void* ids, int id_bits, int64_t n, float scale,
                    void* out, int out_dtype, int64_t out_stride, hipStream_t stream);

/* Bytes of workspace dp_embed_grad needs (0 for n = 0, dim = 0 or sizes it refuses). */
size_t dp_embed_grad_workspace(int64_t n, int64_t vocab, int64_t dim);

/*
 * Gradient of dp_embed_lookup with respect to the table:
 * dtable[v] = scale * sum over i with ids[i] = v of dout[i], and zeros in the
 * rows that no id names; with GRZ_ACCUMULATE that sum is added to what the row
 * holds (the head's gradient of a tied table, an earlier micro-batch), rounded
 * once, and rows no id names are not touched.
 *
 * The ids are sorted by a stable sort and each row's sum runs over its
 * positions in ascending order, cut at fixed places, so the same ids and dout
 * give the same bits.  ("A4", "Common Mistakes": stray atomics.)
 *
 * dout       device, n x dim; dtable  device, vocab x dim.
 * workspace  device, dp_embed_grad_workspace(n, vocab, dim) bytes, 16-byte
 *            aligned; needs no initial value.  Calls that may run at the same
 *            time need one each.
 * Errors: GRZ_ERANGE beyond 2^28 ids, 2^26 rows or 2^22 - 64 columns.
 */
int dp_embed_grad(const void* dout, int dout_dtype, int64_t dout_stride, const void* ids,
                  int id_bits, int64_t n, int64_t vocab, int64_t dim, float scale, int flags,
                  void* workspace, void* dtable, int dtable_dtype, int64_t dtable_stride,
                  hipStream_t stream);

/*
 * Log probabilities under q = softmax(logits[i]) over the vocabulary.
 *
 * logits        device, n x vocab.
 * targets       device, n ids, or NULL (then logprob is NULL as well).
 * logprob       device fp32[n]: log q(targets[i]), 0 where the target names no
 *               token; or NULL.
 * entropy       device fp32[n]: -sum q log q (a token of q = 0 adds 0); or NULL.
 * top           0..min(GRZ_MAX_TOP, vocab): length of the top list.
 * top_ids       device int32[n * top]: the tokens of the largest logits, larger
 *               first, equal ones by lower id (NaN counts as largest).
 * top_logprobs  device fp32[n * top]: their log q.
 * A logit of -inf is a token of probability 0.  A row that holds a NaN or
 * +inf, or nothing but -inf, has no softmax: its results are NaN (its top ids
 * are still in order).  The top list of such a row, of one with fewer logits above
 * -inf than top, or with several hundred near the top-th largest, may take a pass
 * over the row per place.
 * Errors: GRZ_EINVAL also when no output is asked for.
 */
int dp_token_logprobs(const void* logits, int dtype, int64_t n, int64_t vocab, int64_t stride,
                      const void* targets, int id_bits, int top, float* logprob, float* entropy,
                      int32_t* top_ids, float* top_logprobs, hipStream_t stream);

/*
 * Gradient of dp_token_logprobs' logprob and entropy:
 * dlogits[i][v] = glogprob[i] (1[v = targets[i]] - q_v)
 *                 - gentropy[i] q_v (log q_v + H_i).
 * (glogprob = -weight: the weighted cross entropy's gradient.)
 *
 * glogprob, gentropy  device fp32[n], the incoming gradients; either may be
 *                     NULL for 0, not both.  glogprob counts as 0 where the
 *                     target names no token; a row with both 0 gets zeros
 *                     whatever its logits hold.
 * logprob, entropy    device fp32[n] or NULL, as from dp_token_logprobs.
 * dlogits             device, n x vocab of the logits' type; may be the logits
 *                     themselves (same pointer and stride).
 */
int dp_token_logprobs_grad(const void* logits, int dtype, int64_t n, int64_t vocab,
                           int64_t stride, const void* targets, int id_bits,
                           const float* glogprob, const float* gentropy, float* logprob,
                           float* entropy, void* dlogits, int64_t dlogits_stride,
                           hipStream_t stream);

/*
 * Distillation from a teacher's top logits.  With p = softmax over the k listed
 * entries of teacher_logits[i] / T and q = softmax over the vocabulary of
 * logits[i] / T:
 *
 *   loss[i] = weights[i] T^2 sum_j p_j (log p_j - log q(teacher_ids[i][j]))
 *
 * (k = 1 with the target's id and T = 1 is the cross entropy.)
 *
 * logits          device, n x vocab.
 * teacher_ids     device, n * k ids, contiguous.  An entry that names no token
 *                 is left out, as is a teacher logit of -inf; a token listed
 *                 twice has the sum of its entries' p.
 * teacher_logits  device, n * k values of teacher_dtype (GRZ_F32 or GRZ_BF16),
 *                 contiguous; log probabilities will do.
 * k               1..GRZ_MAX_TOP.
 * temperature     T, from 1e-18 to 1e18.
 * weights         device fp32[n], or NULL for 1.  A row of weight 0, or with
 *                 nothing listed, has loss 0 and gradient 0 whatever its
 *                 logits hold.
 * loss            device fp32[n].
 * Errors: GRZ_ERANGE also when n * k exceeds 2^31 - 1.
 */
int dp_distill_loss(const void* logits, int dtype, int64_t n, int64_t vocab, int64_t stride,
                    const void* teacher_ids, int id_bits, const void* teacher_logits,
                    int teacher_dtype, int k, float temperature, const float* weights,
                    float* loss, hipStream_t stream);

/*
 * Gradient of grad_scale * sum of dp_distill_loss's losses:
 * dlogits[i][v] = grad_scale weights[i] T (q_v - sum of p_j with id v).
 *
 * loss     as above, from the same pass over the logits; or NULL.
 * dlogits  device, n x vocab of the logits' type; may be the logits themselves
 *          (same pointer and stride).
 */
int dp_distill_grad(const void* logits, int dtype, int64_t n, int64_t vocab, int64_t stride,
                    const void* teacher_ids, int id_bits, const void* teacher_logits,
                    int teacher_dtype, int k, float temperature, const float* weights,
                    float grad_scale, float* loss, void* dlogits, int64_t dlogits_stride,
                    hipStream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Mixture-of-experts operators: the way of n tokens to k experts each and back.
 *
 *   ids, weights     = dp_expert_route(router logits)
 *   offsets, places  = dp_expert_sort(ids)
 *   rows             = dp_expert_dispatch(x, places)
 *   y[r]             = expert e's output for rows[r], offsets[e] <= r < offsets[e + 1]
 *   out              = dp_expert_combine(y, places, weights)
 * and the gradients' way:
 *   dy, dweights     = dp_expert_combine_grad(dout, y, places, weights)
 *   drows            = the experts' gradients for dy
 *   dx               = dp_expert_combine(drows, places, no weights)
 *   dlogits          = dp_expert_route_grad(dweights)
 * (A dispatch with weights: dx = dp_expert_combine(drows, places, weights), and
 * dweights = dp_expert_combine_grad(dout = x, y = drows) without dy.)
 *
 * Shared conventions: row matrices, sizes, arithmetic and errors as for the
 * operators addressed by token ids (rows on 128-byte lines are fastest; others, at
 * any element's address, take 10 to 30 % longer), and
 *
 *  - Slots.  A token has k of them (1..GRZ_MAX_SLOTS), slot j of token i at index
 *    i * k + j of the contiguous n x k arrays.  n * k is at most 2^28, columns at
 *    most 2^22 - 64 (GRZ_ERANGE).
 *  - An id outside [0, experts) names no expert, a place outside [0, rows) no row:
 *    the slot adds nothing, is stored nowhere, and what its weight and dweight
 *    entries hold is not read.
 *  - Places that name a row twice are an error of the caller: what is written there
 *    then holds elements of either token, and the dweights of its slots are
 *    undefined where dy is y.  Nothing else is affected.
 *  - Rows that no place names are left as they were.
 *  - Overlaps are judged by whole spans: what lies between a matrix's rows counts as
 *    the matrix's.
 */

/*
 * The k experts with the largest logits of each token, larger first, equal ones by
 * lower id (NaN counts as largest), and their weights under p = softmax(logits[i]):
 * p itself, or with GRZ_NORMALIZE p divided by the k weights' sum (the softmax
 * over the listed logits).
 *
 * logits   device, n x experts (1..GRZ_MAX_EXPERTS).
 * k        1..min(GRZ_MAX_SLOTS, experts).
 * ids      device int32[n * k]; weights  device fp32[n * k].
 * A logit of -inf closes an expert to the token: it is never listed, and where
 * fewer than k are open the last slots have id -1 and weight 0 (all of them in a
 * row with nothing open, a padded position).  A row that holds a NaN or +inf has
 * no softmax: its listed experts' weights are NaN (the ids are still in order).
 * Errors: GRZ_EINVAL for k > experts; GRZ_ERANGE beyond GRZ_MAX_EXPERTS.
 */
int dp_expert_route(const void* logits, int dtype, int64_t n, int64_t experts, int64_t stride,
                    int k, int flags, int32_t* ids, float* weights, hipStream_t stream);

/*
 * Gradient of dp_expert_route's weights with respect to the logits, the choice of
 * the experts being fixed.  With w_j the weight of the expert e_j in slot j and g_j =
 * dweights[i][j]:
 *
 *   dlogits[i][e] = sum over e_j = e of g_j w_j - p_e sum_j g_j w_j
 *   with GRZ_NORMALIZE:  sum over e_j = e of w_j (g_j - sum_l g_l w_l)
 *
 * ids       device int32[n * k], dp_expert_route's or any others (an expert listed
 *           twice has its slots' sum).  A listed expert that is closed has weight 0.
 * dweights  device fp32[n * k].  A row whose slots name no expert, or only with
 *           dweights of 0, gets zeros whatever its logits hold.
 * dlogits   device, n x experts of the logits' type; may be the logits themselves
 *           (same pointer and stride).
 */
int dp_expert_route_grad(const void* logits, int dtype, int64_t n, int64_t experts,
                         int64_t stride, int k, int flags, const int32_t* ids,
                         const float* dweights, void* dlogits, int64_t dlogits_stride,
                         hipStream_t stream);

/* Bytes of workspace dp_expert_sort needs (0 for few slots or sizes it refuses). */
size_t dp_expert_sort_workspace(int64_t n, int k, int64_t experts);

/*
 * Places of the slots sorted by expert, stable (an expert's rows in the order of
 * its tokens).
 *
 * ids        device, n * k ids (id_bits 32 or 64), contiguous.
 * experts    1..GRZ_MAX_EXPERTS.
 * workspace  device, dp_expert_sort_workspace bytes, 4-byte aligned; needs no
 *            initial value.  Calls that may run at the same time need one each.
 * offsets    device int32[experts + 1]: expert e's rows are offsets[e] ..
 *            offsets[e + 1] - 1; offsets[experts] is the number of rows.
 * places     device int32[n * k]: the slot's row, -1 where the id names no expert.
 * n = 0 still writes the offsets.
 */
int dp_expert_sort(const void* ids, int id_bits, int64_t n, int k, int64_t experts,
                   void* workspace, int32_t* offsets, int32_t* places, hipStream_t stream);

/*
 * out[places[i][j]] = weights[i][j] x[i] (x[i] itself without weights).
 *
 * x  device, n x dim; places  device int32[n * k]; weights  device fp32[n * k] or
 * NULL; out  device, rows x dim; any of the two types each.
 */
int dp_expert_dispatch(const void* x, int x_dtype, int64_t x_stride, const int32_t* places,
                       const float* weights, int64_t n, int k, int64_t dim, int64_t rows,
                       void* out, int out_dtype, int64_t out_stride, hipStream_t stream);

/*
 * out[i] = sum over j of weights[i][j] y[places[i][j]] (of the rows themselves
 * without weights), in the slots' order; with GRZ_ACCUMULATE onto what out[i]
 * holds, rounded once.  A token without places gets zeros (or keeps its row).
 *
 * y  device, rows x dim; out  device, n x dim; any of the two types each; places,
 * weights  as for dp_expert_dispatch.
 */
int dp_expert_combine(const void* y, int y_dtype, int64_t y_stride, int64_t rows,
                      const int32_t* places, const float* weights, int64_t n, int k, int64_t dim,
                      int flags, void* out, int out_dtype, int64_t out_stride,
                      hipStream_t stream);

/*
 * Gradient of dp_expert_combine:
 *   dy[places[i][j]] = weights[i][j] dout[i]         (1 without weights)
 *   dweights[i][j]   = sum over the columns of dout[i] y[places[i][j]]
 *
 * dout      device, n x dim of either type.
 * y         device, rows x dim (not read, and may be NULL, without dweights).
 * dy        device, rows x dim of y's type, or NULL; may be y itself (same pointer
 *           and stride).
 * dweights  device fp32[n * k] or NULL (not both): 0 for a slot without a row.
 */
int dp_expert_combine_grad(const void* dout, int dout_dtype, int64_t dout_stride, const void* y,
                           int y_dtype, int64_t y_stride, int64_t rows, const int32_t* places,
                           const float* weights, int64_t n, int k, int64_t dim, void* dy,
                           int64_t dy_stride, float* dweights, hipStream_t stream);

/*
 * ---------------------------------------------------------------------------
 * Gradients that are tensors of their own ("Distributed training",
 * clip_grads_device(max_norm), for a model whose gradients are not, or not all, in
 * the flat arena: an expert-parallel rank's experts are averaged over no rank).
 *
 * Lists are host arrays of grz_tensor, read during the call only; the tensors may
 * be of both types, of any length (0 too) and at any element's address.  2^37
 * elements in all at most (GRZ_ERANGE).
 */

/* Norm pieces of the list: GRZ_PIECE consecutive elements of one tensor each, the
 * last of a tensor possibly shorter, numbered tensor by tensor; or a negative
 * GRZ_E* code. */
int64_t dp_tensor_pieces(const grz_tensor* tensors, int64_t count);

/* Bytes of workspace dp_grad_sqnorm_tensors needs (0 also for what it refuses). */
size_t dp_grad_sqnorm_tensors_workspace(const grz_tensor* tensors, int64_t count, int64_t lead);

/*
 * Global squared norm and clip factor over `lead` pieces whose sums are there
 * already (the arena's, from dp_reduce_scatter_mean; a peer's experts') and all
 * elements of the list: the list's piece sums, formed as the reduce forms the
 * arena's, then dp_grad_sqnorm over all of them.  One fp32 tensor and lead 0 give
 * the bits of dp_grad_sqnorm_of.
 *
 * workspace  device, dp_grad_sqnorm_tensors_workspace bytes, 8-byte aligned.  Its
 *            first `lead` doubles are the sums that are there; on return the
 *            list's dp_tensor_pieces follow them.  Calls that may run at the same
 *            time need one each.  The pieces' order decides the sum's last bits:
 *            ranks that want the same ones fold all ranks' pieces in one order.
 * max_norm, sqnorm_out, clip_scale_out  as for dp_grad_sqnorm (either output may be
 *            NULL, not both).  A tensor listed twice counts twice.
 */
int dp_grad_sqnorm_tensors(const grz_tensor* tensors, int64_t count, double max_norm,
                           int64_t lead, void* workspace, double* sqnorm_out,
                           float* clip_scale_out, hipStream_t stream);

/*
 * out[t][e] = clip_scale grads[t][e]: one fp32 product, rounded once to the output's
 * type.
 *
 * clip_scale  device fp32 scalar (dp_grad_sqnorm's output) or NULL for 1.
 * out         host list of the same lengths (types may differ: into a flat arena,
 *             say), or NULL to scale the gradients in place.  In place, a factor
 *             of 1 reads and writes nothing.
 * Errors: GRZ_EINVAL also where an output lies over another tensor of either
 * list than its own gradient, or over that one in part.
 */
int dp_grad_clip_tensors(const grz_tensor* grads, int64_t count, const float* clip_scale,
                         const grz_tensor* out, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GRZ_H */
