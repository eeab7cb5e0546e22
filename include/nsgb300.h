/*
 * nsgb300 -- shape-batched quintic Newton-Schulz for GB300 (sm_103a), with the
 * shard -> home pack and home -> shard unpack around it, and operators of the
 * training step whose gradients it orthogonalises.
 *
 * C ABI of libnsgb300.so. Every function returns an int status (NS_OK = 0 or
 * a negative NS_ERR_* code), never throws and never aborts the process.
 * Device buffers are plain device pointers owned by the caller; the library
 * owns only the plan (host metadata plus, for pack/unpack, a small device
 * routing table it allocates on the first pack/unpack call on a device).
 * Asynchronous work is ordered on the `stream` argument (a cudaStream_t passed
 * as void*; NULL = the legacy default stream). Errors found on the device
 * (a bounded wait that ran out, an index a kernel refused) are recorded in a
 * device status word and reported by ns_check_status().
 *
 * Sources (page title, entry):
 *  [LSA]  Megatron-Core API, core.optimizer.layer_sharded_a2a:
 *         params_by_home, route_to_ns_home, route_from_ns_home.
 *  [OP]   Megatron-Core API, core.distributed.fsdp.src.megatron_fsdp.
 *         experimental.owner_planning: select_ge_2d_params, ns_cost_fn,
 *         _OwnerWork, assign_owner_work, GroupOwnerLayout, OwnerGatherPlan,
 *         OwnerScatterPlan.
 *  [ISS]  Megatron-LM issue #6720 "[GTP][Muon] Optimize Muon step
 *         performance": shape-batched NS, SYRK symmetric kernels,
 *         fp32/TF32 Gram + trace ridge.
 */
#ifndef NSGB300_H
#define NSGB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------ status codes */
enum {
  NS_OK = 0,
  NS_ERR_ARG = -1,           /* null pointer, bad count, S/shard_dim mismatch   */
  NS_ERR_SHAPE = -2,         /* ndim < 2 for a participating tensor, bad dims   */
  NS_ERR_NOT_DIVISIBLE = -3, /* shard_dim size (or buffer size) not divisible by S */
  NS_ERR_HOME = -4,          /* home/owner missing, out of range, or not a holder */
  NS_ERR_CUDA = -5,          /* a CUDA runtime/driver call failed               */
  NS_ERR_TIMEOUT = -6,       /* a kernel's bounded wait ran out (device status)  */
  NS_ERR_DEVICE_CHECK = -7,  /* a kernel refused an out-of-range index           */
  NS_ERR_UNSUPPORTED = -8,   /* mode or device not supported by this library    */
  NS_ERR_WORKSPACE = -9      /* workspace missing, too small or misaligned       */
};

/* Precision policy of a plan (gram_mode). */
enum {
  NS_BF16 = 0,      /* bf16 X, A, B operands, fp32 accumulation and epilogues; bf16 in, bf16 out */
  NS_FP32_GRAM = 1, /* fp32 X, A, B as split-TF32 (hi, lo) pairs; bf16 in, fp32 out */
  /* [ISS] Gram-space NS ("gram_once"), same fp32 precision: A = X X^T once, then
   * per step Q = aI + bA + cA^2, A <- Q A Q, P <- Q P on m x m matrices only,
   * and X_k = P X_0 at the end. Exact reformulation of the same iteration;
   * fewer flops when n is well above m. bf16 in, fp32 out. */
  NS_FP32_GRAM_SPACE = 2,
  /* Per shape bucket, Gram-space when n >= 2m and NS_FP32_GRAM otherwise:
   * with k = 5 steps Gram-space does 4m^2n + 8km^3 flops against the
   * standard k(4m^2n + 2m^3), fewer once n > 1.875 m. Same precision and
   * results per matrix as the mode chosen for its bucket. bf16 in, fp32 out. */
  NS_FP32_AUTO = 3
};

/* Data model of a plan. */
enum {
  NS_LAYOUT_ROW_SHARD = 0, /* [LSA] every rank holds a (P/S, Q) slice of every param    */
  NS_LAYOUT_FLAT = 1,      /* [OP]  one flat buffer split evenly into S rank ranges     */
  NS_LAYOUT_TWO_STAGE = 2  /* [LSA] GTP_remat (dim 0) x TP (partition_dim) shards, one fused gather */
};

typedef struct ns_plan ns_plan_t; /* opaque; owned by the library */

/* ------------------------------------------------------------- host only */

/* [OP] ns_cost_fn. View `shape` (ndim >= 2) as (rows, cols) = (shape[0],
 * prod(shape[1:])); cost = rows*cols*(min(rows, cols)*steps + 1), exact in
 * int64. NS_ERR_SHAPE if ndim < 2 or a dim is negative; NS_ERR_ARG on null
 * pointers, steps < 0, or int64 overflow. */
int ns_cost(const int64_t* shape, int ndim, int steps, int64_t* cost_out);

/* [OP] assign_owner_work: greedy LPT. Tensors with one candidate are taken
 * first in index order, then the rest in descending cost (equal costs keep
 * index order); each goes to its least-loaded candidate, equal loads to the
 * candidate listed first. Candidates of tensor i are
 * cand_idx[cand_ptr[i] .. cand_ptr[i+1]) (CSR), ranks in [0, n_ranks), listed
 * in buffer order. owner_out[i] receives the owner. NS_ERR_HOME if a tensor
 * has no candidate or a candidate is out of range; NS_ERR_ARG on bad
 * arguments (costs must be > 0). */
int ns_assign_owner_work(int n_tensors, const int64_t* costs, const int32_t* cand_ptr,
                         const int32_t* cand_idx, int n_ranks, int32_t* owner_out);

/* [LSA] route_to_ns_home / route_from_ns_home plan cache, [OP] ns_cost_fn.
 * Row-shard plan over n_tensors params; tensor i has ndims[i] dims, listed
 * consecutively in shapes_flat. Every param is sharded S ways along
 * shard_dim (its size there must be divisible by S: NS_ERR_NOT_DIVISIBLE).
 * home_of[i] in [0, S) is param i's NS home; NULL asks for LPT homes over all
 * S ranks with cost ns_cost(shape, steps). steps >= 0; (a, b, c) are the
 * quintic coefficients used in every step; eps is added to the Frobenius
 * norm; ridge >= 0 adds ridge*(trace(A)/m)*I to A before B is formed (only
 * in NS_FP32_GRAM mode; must be 0 in NS_BF16 mode). The plan copies every
 * input array; the caller owns its validity only in the sense of [LSA]:
 * reuse it only while shapes, homes and S are unchanged. No CUDA call. */
int ns_plan_create(int n_tensors, const int32_t* ndims, const int64_t* shapes_flat, int steps,
                   float a, float b, float c, float eps, int gram_mode, float ridge, int S,
                   int shard_dim, const int32_t* home_of, ns_plan_t** plan_out);

/* [LSA] two-stage exchange (GTP_remat group along dim 0, then TP group along
 * partition_dim) and [ISS] its fusion into one exchange. S = R * T simulated
 * ranks, rank r*T + t holding remat slice r (along dim 0, of R) of TP slice t
 * (along partition_dims[i], of T) of every param, params in index order.
 * ns_pack_to_home assembles each param on its home in ONE gather, equal bit
 * for bit to running the two stages one after the other; ns_unpack_from_home
 * is its inverse. partition_dims[i] = 0 needs shape[0] % (R*T) == 0; else
 * shape[0] % R == 0 and shape[partition_dim] % T == 0 (NS_ERR_NOT_DIVISIBLE).
 * home_of in [0, R*T) or NULL for LPT homes. Other arguments as in
 * ns_plan_create. No CUDA call. */
int ns_plan_create_two_stage(int n_tensors, const int32_t* ndims, const int64_t* shapes_flat,
                             const int32_t* partition_dims, int R, int T, int steps, float a, float b,
                             float c, float eps, int gram_mode, float ridge, const int32_t* home_of,
                             ns_plan_t** plan_out);

/* [OP] GroupOwnerLayout / OwnerGatherPlan data model. Flat-buffer plan: tensor
 * i occupies elements [offsets[i], offsets[i] + numel_i) of a buffer of
 * buffer_size elements (buffer_size % S == 0, else NS_ERR_NOT_DIVISIBLE);
 * rank r holds [r*size/S, (r+1)*size/S). participating[i] != 0 marks the
 * tensors that take part (NULL = every tensor with ndim >= 2, the
 * select_ge_2d_params default); participating tensors must not overlap and
 * must have ndim >= 2 and numel > 0. owner_of[i] (read for participating i
 * only) must be a rank holding part of tensor i (NS_ERR_HOME otherwise);
 * NULL asks for assign_owner_work's default LPT owners. Other arguments as
 * in ns_plan_create. No CUDA call. */
int ns_plan_create_flat(int n_tensors, const int32_t* ndims, const int64_t* shapes_flat,
                        const int64_t* offsets, int64_t buffer_size, const uint8_t* participating,
                        int steps, float a, float b, float c, float eps, int gram_mode, float ridge,
                        int S, const int32_t* owner_of, ns_plan_t** plan_out);

/* Frees the plan and any device routing tables it uploaded. NULL is a no-op. */
int ns_plan_destroy(ns_plan_t* plan);

/* Plan summary: info[0] = n_tensors, [1] = participating count, [2] = S,
 * [3] = layout, [4] = gram_mode, [5] = steps, [6] = number of shape
 * buckets, [7] = per-rank buffer elements (row-shard) or buffer_size/S (flat),
 * [8] = input element bytes, [9] = output element bytes. info has >= 10 slots. */
int ns_plan_info(const ns_plan_t* plan, int64_t* info);

/* [LSA] params_by_home source: home_out[i] = home (owner) of tensor i, or -1
 * for a tensor that does not participate. home_out has n_tensors slots. */
int ns_plan_homes(const ns_plan_t* plan, int32_t* home_out);

/* Layout of the home buffers: home_offsets[i] = element offset of tensor i in
 * its home buffer (-1 if not participating); home_sizes[h] = elements in home
 * buffer h; rank_sizes[r] = elements in rank buffer r. Any pointer may be
 * NULL. Home h holds its tensors complete, in increasing index order. */
int ns_plan_home_layout(const ns_plan_t* plan, int64_t* home_offsets, int64_t* home_sizes,
                        int64_t* rank_sizes);

/* Bytes of device workspace ns_orthogonalize_batched needs (256-byte
 * aligned base required). Zero when nothing participates. */
int ns_plan_workspace_bytes(const ns_plan_t* plan, uint64_t* bytes);

/* [OP] OwnerGatherPlan metadata seen from rank rho (flat plans only, else
 * NS_ERR_ARG). send_sizes[o] = elements rho sends to owner o (0 = absent,
 * always 0 for o == rho); recv_sizes[s] = elements rho receives from s;
 * recv_offsets[i*S + s] = offset of tensor i's piece inside s's buffer to rho
 * (-1 = absent); own_sizes[i] = elements of rho's own shard of tensor i if
 * rho owns i, else -1. Any output pointer may be NULL. */
int ns_owner_gather_meta(const ns_plan_t* plan, int rho, int64_t* send_sizes, int64_t* recv_sizes,
                         int64_t* recv_offsets, int64_t* own_sizes);

/* [OP] OwnerScatterPlan metadata seen from rank rho (flat plans only):
 * send_sizes[d] = result elements rho (as owner) sends to d; recv_sizes[o]
 * = elements rho receives from owner o; recv_offsets[i*S + o] = offset of
 * tensor i's result piece inside o's buffer to rho (-1 = absent). */
int ns_owner_scatter_meta(const ns_plan_t* plan, int rho, int64_t* send_sizes, int64_t* recv_sizes,
                          int64_t* recv_offsets);

/* [LSA] route_to_ns_home / route_from_ns_home as one all_to_allv of row
 * shards, seen from rank rho (row-shard and two-stage plans; flat plans use
 * ns_owner_gather_meta, NS_ERR_ARG here). Every rank holds a piece of
 * numel/S elements of every participating tensor.
 *   send_counts[h], send_displs[h]: elements rho sends to home h and their
 *     offset in rho's send buffer, which holds, home by home in rank order,
 *     rho's pieces of the tensors homed on h in index order;
 *   recv_counts[s], recv_displs[s]: elements rho receives from rank s and
 *     their offset in rho's receive buffer (source by source in rank order,
 *     each segment the pieces of the tensors homed on rho in index order);
 *   send_pos[i]: offset of rho's piece of tensor i in its send buffer (-1 if
 *     tensor i does not participate);
 *   recv_pos[i*S + s]: offset of rank s's piece of tensor i in rho's receive
 *     buffer (-1 unless rho is tensor i's home).
 * The reverse exchange (route_from_ns_home) swaps the send and receive
 * sides. Arrays of S (counts, displs), n_tensors (send_pos) and n_tensors*S
 * (recv_pos) entries; any pointer may be NULL. Host only. */
int ns_plan_rank_splits(const ns_plan_t* plan, int rho, int64_t* send_counts, int64_t* send_displs,
                        int64_t* recv_counts, int64_t* recv_displs, int64_t* send_pos, int64_t* recv_pos);

const char* ns_status_string(int status);

/* ----------------------------------------------------------------- device */

/* [OP] ns_cost_fn step, [ISS] shape-batched NS. Orthogonalises the n
 * participating tensors of the plan (n must equal the participating count),
 * in index order: in[j] / out[j] are device pointers to the j-th participating
 * tensor, contiguous row-major in its original shape (bf16 in; bf16 out in
 * NS_BF16 mode, fp32 out in NS_FP32_GRAM mode). out[j] == in[j] is allowed;
 * other overlaps are not. Each tensor is viewed as (shape[0], prod(shape[1:])),
 * transposed so rows <= cols, scaled by 1/(||X||_F + eps), run for `steps`
 * steps of A = X X^T; X = a X + (b A + c A A) X, transposed back and stored.
 * workspace must hold ns_plan_workspace_bytes() bytes, 256-byte aligned; it
 * is scratch (no contents kept between calls). Asynchronous on `stream`;
 * calls that share a workspace must not overlap on the GPU. After a first
 * call on a device (it looks up per-device state), the call may be captured
 * into a CUDA graph and replayed: it allocates, synchronises and queries
 * nothing; a replay reads the buffers' current contents. The library's kernels
 * are launched with programmatic stream serialization: each may start its
 * set-up while the previous kernel in the stream runs, and reads or writes no
 * data before that kernel has completed, so ordering with the caller's work
 * on `stream` is as for ordinary launches. */
int ns_orthogonalize_batched(ns_plan_t* plan, const void* const* in, void* const* out, int n,
                             void* workspace, uint64_t workspace_bytes, void* stream);

/* [LSA] route_to_ns_home, [OP] OwnerGatherPlan.pack + reconstruct_full.
 * Device-local gather over S simulated ranks (no collective): rank_bufs[r]
 * (S device pointers, input dtype) hold rank r's data -- row-shard plans: its
 * (P/S, Q) shard of every param, in index order; flat plans: elements
 * [r*size/S, (r+1)*size/S) of the flat buffer. home_bufs[h] (S pointers)
 * receive home h's complete tensors in increasing index order, at the offsets
 * ns_plan_home_layout reports. S and shard_dim must equal the plan's (flat
 * plans: shard_dim 0). Bit-exact copy. The first pack/unpack call on a device
 * uploads the plan's routing table (cudaMalloc + copy): make it before any
 * stream capture. */
int ns_pack_to_home(ns_plan_t* plan, const void* const* rank_bufs, int S, int shard_dim,
                    void* const* home_bufs, void* stream);

/* [LSA] route_from_ns_home, [OP] OwnerScatterPlan.pack + unpack. Inverse of
 * ns_pack_to_home on the output dtype: home_bufs[h] hold complete results,
 * rank_bufs[r] receive rank r's shard of every result (flat plans: only the
 * elements of participating tensors are written). */
int ns_unpack_from_home(ns_plan_t* plan, const void* const* home_bufs, int S, int shard_dim,
                        void* const* rank_bufs, void* stream);

/* [ISS] wave dispatch, single-GPU form. A pipeline splits the plan's
 * participating tensors (bf16 plans only, else NS_ERR_UNSUPPORTED) into at
 * most n_waves waves of consecutive tensors with balanced ns_cost (no wave
 * when no tensor participates; one wave when every shape bucket runs as one
 * CTA per matrix, see ns_set_small_path; n_waves < 1 is NS_ERR_ARG). The plan must
 * outlive the pipeline. ns_pipeline_run then performs pack ->
 * Newton-Schulz -> unpack for the whole plan, with the same results as
 * ns_pack_to_home + ns_orthogonalize_batched + ns_unpack_from_home. Work runs
 * on three streams owned by the pipeline: the pack and prologue of a wave
 * overlap the NS products of the previous wave, and the unpack of a wave
 * overlaps the next one. Buffers as in ns_pack_to_home / ns_unpack_from_home
 * (home_in receives the gathered inputs, home_out the results); for row-shard
 * plans with shard_dim 0, where every row of a tensor is contiguous in one
 * rank buffer, the prologue reads the rank buffers directly and the last B*X
 * launch of each wave writes the results straight into rank_out, so home_in
 * and home_out are left untouched (a wave whose last launch cannot address
 * all its matrices still stages its results in home_out). When every bucket
 * of such a plan runs as one CTA per matrix, the whole call is that one
 * launch, issued on `stream` itself. workspace
 * holds two wave workspaces (ns_pipeline_info), 256-byte aligned. The call
 * is ordered after prior work on `stream`, and later work on `stream` waits
 * for all of it. The first run on a device creates the pipeline's streams
 * and events: make it before any stream capture. Runs that overlap on the
 * GPU must not share a pipeline or a workspace. */
typedef struct ns_pipeline ns_pipeline_t;
int ns_pipeline_create(ns_plan_t* plan, int n_waves, ns_pipeline_t** pipeline_out);
int ns_pipeline_info(const ns_pipeline_t* pipeline, int* n_waves, uint64_t* workspace_bytes);
int ns_pipeline_run(ns_pipeline_t* pipeline, const void* const* rank_in, void* const* home_in,
                    void* const* home_out, void* const* rank_out, void* workspace, uint64_t workspace_bytes,
                    void* stream);
int ns_pipeline_destroy(ns_pipeline_t* pipeline);

/* Synchronises `stream`, then reads and clears the current device's status
 * word: NS_ERR_TIMEOUT or NS_ERR_DEVICE_CHECK if a kernel recorded one, else
 * NS_ERR_CUDA on a pending CUDA error, else NS_OK. plan may be NULL. */
int ns_check_status(ns_plan_t* plan, void* stream);

/* No counterpart on the pages: an addition for callers that cannot allocate
 * device memory when they orthogonalise (e.g. a plugin inside a host program
 * whose caching allocator owns the GPU's memory, or code that must not call
 * cudaMalloc after start-up). Same computation and arguments as
 * ns_orthogonalize_batched, but the scratch memory is a static device array
 * of NS_FIXED_WS_BYTES inside the library instead of a caller workspace.
 * Allocates nothing (no cudaMalloc, no cudaFree). Returns NS_ERR_WORKSPACE if
 * the plan needs more than NS_FIXED_WS_BYTES (see ns_plan_workspace_bytes).
 * The array exists once per GPU that loads the library and is held until the
 * process exits. When it is reserved depends on CUDA's module loading: under
 * lazy loading (the default) the first call on a device, which looks up the
 * array's device address (cudaGetSymbolAddress) with that device current,
 * loads the module holding it and so reserves the NS_FIXED_WS_BYTES then --
 * that first call can fail with NS_ERR_CUDA if the GPU is already full, so
 * make it at start-up (and before any stream capture); under eager loading
 * (CUDA_MODULE_LOADING=EAGER) every process that loads the library holds the
 * array from the start, whether or not it calls this function. Every call
 * shares the array and finds the previous call's contents there (the kernels
 * write every byte they read first), so calls that overlap on the GPU (e.g.
 * on two streams) race. */
#define NS_FIXED_WS_BYTES (64ull << 20)
int ns_orthogonalize_batched_fixed_ws(ns_plan_t* plan, const void* const* in, void* const* out, int n,
                                      void* stream);

/* ------------------------------------------------ training-step operators
 * No counterpart on the pages: what a training step needs next to the
 * optimiser, around the matrices it orthogonalises -- the routing of tokens
 * to the experts of a mixture-of-experts layer, the norms and the rotation of
 * a fused QKV projection's queries and keys, and a distillation loss -- each
 * with its gradient.
 *
 * Common to all: device buffers are the caller's; strides are in elements and
 * the last dimension is contiguous; element types are NS_DT_*; sums, norms and
 * softmax statistics are in fp32 and a result is rounded to its type once; the
 * same call gives the same bits (no atomics on floating values). Buffers
 * of one call must not overlap unless its text says so. A zero count (tokens,
 * heads, rows) is valid and does what the formulas say. Workspaces are scratch
 * (no contents kept between calls), 256-byte aligned. Work is asynchronous on
 * `stream`; after a first call on a device every call may be captured into a
 * CUDA graph. An index that points outside its buffer is refused on the
 * device: the access is skipped and ns_check_status reports
 * NS_ERR_DEVICE_CHECK. Arguments are checked on the host: NS_ERR_ARG for null
 * pointers, addresses that their elements cannot have and values outside their
 * domain, NS_ERR_SHAPE for sizes or strides
 * that do not fit each other, NS_ERR_UNSUPPORTED past a stated limit,
 * NS_ERR_WORKSPACE as elsewhere. */

/* Element types. */
enum {
  NS_DT_BF16 = 0,
  NS_DT_FP16 = 1,
  NS_DT_FP32 = 2
};

/* Rows that hold any routing of tokens x k slots to `experts` experts when
 * every expert's segment is padded to a multiple of `align` rows and keeps at
 * most `capacity` slots (0: all). Host only. */
int ns_moe_rows(int64_t tokens, int k, int experts, int align, int64_t capacity, int64_t* rows_out);

/* Bytes of device workspace of ns_moe_sort (may be 0). Host only. */
int ns_moe_sort_workspace_bytes(int64_t tokens, int k, int experts, uint64_t* bytes);

/* Tokens sorted by expert. expert_ids[t * k + j] (int32 or int64: id_bytes 4
 * or 8) is token t's j-th choice; a negative one goes nowhere, one >= experts
 * is refused and goes nowhere. The sort is stable: within an expert, slots
 * s = t * k + j keep their order, and those past `capacity` (0: no limit) are
 * dropped. counts[e] = slots kept by expert e; offsets[e] = first row of its
 * segment, offsets[experts] = rows in use (segments padded to multiples of
 * align); row_of_slot[s] = row of slot s or -1; slot_of_row[r] = slot of row r
 * or -1, for all `rows` rows (rows >= ns_moe_rows, NS_ERR_SHAPE otherwise).
 * 1 <= k <= 32, 1 <= experts <= 1024; tokens * k and rows at most 2^30, here and
 * below. */
int ns_moe_sort(const void* expert_ids, int id_bytes, int64_t tokens, int k, int experts, int align,
                int64_t capacity, int64_t rows, int32_t* row_of_slot, int32_t* slot_of_row, int32_t* counts,
                int32_t* offsets, void* workspace, uint64_t workspace_bytes, void* stream);

/* out[r] = x[slot_of_row[r] / k], and 0 for every row without a slot, so that
 * a product over padded segments sees no stale values. x is [tokens][dim],
 * out [rows][dim], dim < 2^29; row_of_slot and slot_of_row as ns_moe_sort wrote
 * them. */
int ns_moe_dispatch(const void* x, int64_t x_stride, int dtype, int64_t tokens, int k, int64_t dim,
                    const int32_t* row_of_slot, const int32_t* slot_of_row, int64_t rows, void* out,
                    int64_t out_stride, void* stream);

/* Gradient of ns_moe_dispatch: grad_x[t] = sum over token t's kept slots of
 * grad_rows[row] (0 if it has none). */
int ns_moe_dispatch_grad(const void* grad_rows, int64_t rows_stride, int dtype, int64_t tokens, int k, int64_t dim,
                         const int32_t* row_of_slot, int64_t rows, void* grad_x, int64_t grad_x_stride,
                         void* stream);

/* y[t] = sum over token t's kept slots of weights[t * k + j] * expert_rows[row]
 * (0 if it has none). weights fp32 [tokens][k], NULL = 1; the weight of a
 * dropped slot is not used, whatever it holds. */
int ns_moe_combine(const void* expert_rows, int64_t rows_stride, int dtype, int64_t tokens, int k, int64_t dim,
                   const int32_t* row_of_slot, const float* weights, int64_t rows, void* y, int64_t y_stride,
                   void* stream);

/* Gradient of ns_moe_combine: grad_rows[row] = weight * grad_y[t] (0 for every
 * row without a slot), grad_weights[t * k + j] = <grad_y[t], expert_rows[row]>
 * (0 for a dropped slot). grad_rows may be expert_rows itself, with the same
 * stride. */
int ns_moe_combine_grad(const void* grad_y, int64_t grad_y_stride, const void* expert_rows, int64_t rows_stride,
                        int dtype, int64_t tokens, int k, int64_t dim, const int32_t* row_of_slot,
                        const int32_t* slot_of_row, const float* weights, int64_t rows, void* grad_rows,
                        int64_t grad_rows_stride, float* grad_weights, void* stream);

/* Norms of queries and keys for each head with the position rotation:
 * y = R_pos (x / sqrt(mean(x^2) + eps) * weight) for every head x of head_dim
 * values. q is [tokens][q_heads][head_dim] and k [tokens][k_heads][head_dim]
 * (for instance column ranges of one fused projection); strides[8] holds the
 * (token, head) strides of q, k, q_out, k_out in that order. q_weight and
 * k_weight (NULL = 1) have head_dim values of weight_dtype (dtype or fp32).
 * The rotation acts on the first rot_dim (even, 0 = none) values: pairs
 * (i, i + rot_dim / 2), or (2i, 2i + 1) if interleaved = 1, turned by the
 * angle whose cosine and sine are table[pos][i] and
 * table[pos][rot_dim / 2 + i] (fp32 [table_rows][rot_dim]). positions[t] is
 * int32 or int64 (position_bytes 4 or 8), NULL = t; a token whose position is
 * outside the table is refused (its outputs are not written). head_dim <= 1024,
 * tokens * (q_heads + k_heads) < 2^30. The sum of a head's squares is in fp32:
 * a root mean square above 1e18 (of 128 values) has no norm there.
 * q_out may be q and k_out may be k, with the same strides. */
int ns_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const int64_t* strides, int dtype,
                    int64_t tokens, int q_heads, int k_heads, int head_dim, int rot_dim, int interleaved,
                    const void* q_weight, const void* k_weight, int weight_dtype, float eps, const float* table,
                    int64_t table_rows, const void* positions, int position_bytes, void* stream);

/* Bytes of device workspace of ns_qk_norm_rope_grad (needed only with a
 * weight gradient). Host only. */
int ns_qk_norm_rope_grad_workspace_bytes(int head_dim, uint64_t* bytes);

/* Gradient of ns_qk_norm_rope: from grad_q_out, grad_k_out and the forward's
 * q and k, grad_q and grad_k, and the weights' gradients (fp32 [head_dim], sums
 * over tokens and heads; NULL = not wanted). strides[12] holds the (token,
 * head) strides of q, k, grad_q, grad_k, grad_q_out, grad_k_out. grad_q may be
 * grad_q_out or q, and grad_k likewise, with the same strides. */
int ns_qk_norm_rope_grad(const void* grad_q_out, const void* grad_k_out, const void* q, const void* k, void* grad_q,
                         void* grad_k, const int64_t* strides, int dtype, int64_t tokens, int q_heads, int k_heads,
                         int head_dim, int rot_dim, int interleaved, const void* q_weight, const void* k_weight,
                         int weight_dtype, float* grad_q_weight, float* grad_k_weight, float eps,
                         const float* table, int64_t table_rows, const void* positions, int position_bytes,
                         void* workspace, uint64_t workspace_bytes, void* stream);

/* Distillation from a teacher's top logits. For token t with student logits s
 * (vocab values), the teacher's `top` values z at entries i (teacher_values and
 * teacher_ids, contiguous [tokens][top]; ids int32 or int64):
 *   p_j  = exp(z_j / temperature - Z), Z = teacher_lse[t] (the teacher's
 *          log-sum-exp of z / temperature over its whole vocabulary) or, if
 *          teacher_lse is NULL, the log-sum-exp over the entries given
 *   lse  = log-sum-exp of s / temperature
 *   loss = weights[t] * sum_j p_j (log p_j - s[i_j] / temperature + lse)
 * and, unless grad_logits is NULL,
 *   grad_logits[v] = weights[t] / temperature *
 *                    (sum_j p_j * exp(s[v] / temperature - lse) - sum of the p_j with i_j = v).
 * weights NULL = 1. Entries with a negative id (padding) or a value of -inf
 * are left out; an id >= vocab is refused and left out. A token whose weight is
 * 0 or that has no entry left gets loss 0, lse 0 and a zero gradient, whatever
 * its logits hold. grad_logits may be logits itself, with the same stride.
 * top <= 1024, temperature in [1e-30, 1e30]. Any other row needs a finite logit, of whatever size: one of -inf
 * gives NaN. Where s / temperature leaves fp32's range lse is infinite; loss and grad_logits are not affected. */
int ns_distill_loss(const void* logits, int64_t logits_stride, int dtype, int64_t tokens, int64_t vocab,
                    const void* teacher_values, int teacher_dtype, const void* teacher_ids, int id_bytes, int top,
                    const float* weights, const float* teacher_lse, float temperature, float* loss, float* lse,
                    void* grad_logits, int64_t grad_stride, void* stream);

/* The gradient alone, from the lse that ns_distill_loss wrote for the same
 * logits: for a backward pass that comes later, with other weights. A token
 * that ns_distill_loss left out has no lse (it wrote -0 there): where such a
 * token has a weight and entries now, its gradient is NaN. */
int ns_distill_grad(const void* logits, int64_t logits_stride, int dtype, int64_t tokens, int64_t vocab,
                    const void* teacher_values, int teacher_dtype, const void* teacher_ids, int id_bytes, int top,
                    const float* weights, const float* teacher_lse, float temperature, const float* lse,
                    void* grad_logits, int64_t grad_stride, void* stream);

/* ---- gradient norm and clipping. Tensors are given as arrays of `count`
 * addresses, numbers of values and types (NS_DT_*, which may differ from tensor
 * to tensor): host arrays that are read before the call returns. A tensor's
 * values are contiguous in memory, at any address that they can have; it may
 * be empty. At most 2^20 tensors, 2^43 bytes together. A tensor that ns_grad_clip
 * writes must not overlap the call's others (several blocks would write it at
 * once); the calls on torch tensors refuse one that begins where another does. */

/* Bytes of device workspace of ns_grad_norm. Host only. */
int ns_grad_norm_workspace_bytes(int count, uint64_t* bytes);

/* *norm (device, fp32) = sqrt(sum of squares of all values of all tensors), 0
 * without any. Squares that leave fp32's range are summed in 64 bits, so that
 * finite values have their norm whatever their size; one above fp32's largest
 * value is infinite. An infinite value makes it infinite, a NaN makes it NaN. */
int ns_grad_norm(const void* const* grads, const int64_t* numels, const int* dtypes, int count, float* norm,
                 void* workspace, uint64_t workspace_bytes, void* stream);

/* outs[i] = c * grads[i], c = min(1, max_norm / (*norm + eps)), rounded once.
 * *norm is on the device: what ns_grad_norm wrote, or the norm over several
 * calls or ranks. outs[i] may be grads[i] itself, and is not touched then if
 * c = 1. An infinite norm gives c = 0 (infinite values become NaN), unless
 * max_norm is infinite as well (c = 1); a norm that is NaN makes every value NaN.
 * max_norm >= 0, eps >= 0 and finite. */
int ns_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels, const int* dtypes, int count,
                 const float* norm, float max_norm, float eps, void* stream);

/* The norms after and before a block of a residual network, with the block's
 * gate and the residual's scale. For each token, with the block's output b and
 * the residual x of dim values:
 *   u = b / sqrt(mean(b^2) + eps) * branch_weight (post_norm = 0: b * branch_weight)
 *   h = residual_scale * x + branch_scale * gate * u      -> residual_out
 *   n = h / sqrt(mean(h^2) + eps) * weight                -> out
 * branch, out and the weights' type is dtype, the residual's residual_dtype
 * (dtype or fp32); branch_weight and weight (NULL = 1) have dim values of
 * weight_dtype (dtype or fp32). gate_kind 0: no gate; 1: fp32 [tokens], one for
 * each token; 2: [tokens][dim] of dtype. branch NULL: h = residual_scale * x
 * (the norm before the first block; the gate is not used). residual_out NULL or
 * out NULL: not wanted; n is computed from h before h is rounded. strides[5]:
 * row strides of branch, residual, residual_out, out and gate. residual_out may
 * be residual and out may be branch or gate, with the same stride. dim at most
 * 2^20, tokens * dim at most 2^40. Sums of squares are in fp32: a row whose sum is
 * above 3.4e38 (a root mean square of 1e17 at 32768 columns) has no norm there, nor
 * with eps = 0 one whose root mean square is below 1e-18. Rows beyond 8192 columns
 * are read several times. */
int ns_block_norm(const void* branch, const void* residual, void* residual_out, void* out, const int64_t* strides,
                  int dtype, int residual_dtype, int64_t tokens, int64_t dim, const void* branch_weight,
                  const void* weight, int weight_dtype, const void* gate, int gate_kind, int post_norm,
                  float residual_scale, float branch_scale, float eps, void* stream);

/* Bytes of device workspace of ns_block_norm_grad (needed only with a weight
 * gradient). Host only. */
int ns_block_norm_grad_workspace_bytes(int64_t dim, uint64_t* bytes);

/* Gradient of ns_block_norm, from the gradients of residual_out and of out
 * (either may be NULL: zero) and the forward's branch, gate and residual_out (h
 * as it was stored; with residual_scale 1 and no branch that is residual): the
 * gradients of branch, residual and gate, and the weights' (fp32 [dim], sums over
 * tokens); each may be NULL: not wanted. The gate's gradient has the gate's form
 * and type. strides[8]: row strides of branch, residual_out, grad_branch,
 * grad_residual, grad_residual_out, grad_out, gate and grad_gate. Outputs may be
 * inputs of the same type and shape with the same stride (grad_residual may be
 * grad_residual_out, grad_branch may be grad_out or branch, grad_gate may be
 * gate), each input at most once. The sum of grad_out * weight * residual_out over a
 * row is in fp32 as well. Without tokens the weights' gradients are zero; with dim 0
 * nothing is written. */
int ns_block_norm_grad(const void* grad_residual_out, const void* grad_out, const void* branch, const void* residual_out,
                       void* grad_branch, void* grad_residual, const int64_t* strides, int dtype, int residual_dtype,
                       int64_t tokens, int64_t dim, const void* branch_weight, const void* weight, int weight_dtype,
                       const void* gate, int gate_kind, float* grad_branch_weight, float* grad_weight, void* grad_gate,
                       int post_norm, float residual_scale, float branch_scale, float eps, void* workspace,
                       uint64_t workspace_bytes, void* stream);

/* Bytes of device workspace of ns_moe_few_tokens. Host only. */
int ns_moe_few_tokens_workspace_bytes(int64_t tokens, int k, int64_t dim, int64_t ffn, uint64_t* bytes);

/* A whole mixture-of-experts layer for a few tokens (a decoding step), without
 * sorting them: for every slot s = t * k + j with expert e = expert_ids[s]
 *   h_s = silu(G_e x_t) * (U_e x_t),  silu(a) = a / (1 + exp(-a))
 *   y_t = sum over t's slots of weights[s] * D_e h_s
 * where gate_up is [experts][2 * ffn][dim], G_e its first ffn rows of expert e
 * and U_e the others, and down is [experts][dim][ffn], all contiguous. Ids are
 * int32 or int64; a negative one goes nowhere, one >= experts is refused and goes
 * nowhere; a token may name an expert more than once. weights fp32
 * [tokens][k], NULL = 1; the weight of a slot that goes nowhere is not used,
 * whatever it holds, and the matrices of experts that no token names are not
 * read. Those of the others are read once for every 16 slots that name them.
 * Products of bf16 and fp16 factors are exact; the hidden value and the factors of
 * fp32 layers take part as two tf32 values each (2^-22 off); sums are in fp32. An
 * infinite factor (an fp32 x, a matrix value, a hidden value) may give NaN where
 * infinity is due, in the tokens that meet it. y may be x itself. tokens <= 256,
 * 1 <= k <= 32, 1 <= experts <= 1024, dim and ffn < 2^20, ffn >= 1; for more
 * tokens: ns_moe_sort, ns_moe_dispatch and ns_moe_combine. */
int ns_moe_few_tokens(const void* x, int64_t x_stride, int dtype, int64_t tokens, int k, int64_t dim, int64_t ffn,
                      int experts, const void* expert_ids, int id_bytes, const float* weights, const void* gate_up,
                      const void* down, void* y, int64_t y_stride, void* workspace, uint64_t workspace_bytes,
                      void* stream);

/* ---------------------------------------------------------- test support
 * No counterpart on the pages: hooks with which tests drive the library's
 * device-side error paths without faulting or hanging the GPU. */

/* Arms the next bf16 GEMM launch of this process (any phase, any thread) to
 * stall: its TMA producer issues no copy, so its MMA issuer's first wait for
 * operands cannot complete; every wait of that launch is bounded by
 * wait_limit_ns (1e5 .. 1e10 ns, else NS_ERR_ARG), after which the kernel
 * records a timeout in the device status word and unwinds (nothing is in
 * flight: no copy or MMA was issued). The call that contains the launch
 * returns normally but its results are garbage; ns_check_status then reports
 * NS_ERR_TIMEOUT, and later calls run normally. One-shot. */
int ns_test_stall_next_gemm(uint64_t wait_limit_ns);

/* Sets the home index of tensor `tensor` in the plan's routing table (and in
 * every device copy already uploaded) to `home`, which may be out of range:
 * pack and unpack then refuse that tensor's entry (its data is not moved),
 * record the refusal in the device status word, and ns_check_status reports
 * NS_ERR_DEVICE_CHECK. Restore the plan's own home to undo. NS_ERR_ARG if
 * the tensor has no routing entry. Synchronous (cudaMemcpy). */
int ns_test_set_route_home(ns_plan_t* plan, int tensor, int home);

/* ------------------------------------------------------------ measurement
 * Not part of the pages' interface: support for measuring the kernels above.
 * Kernel kinds: 0 = Gram (X X^T), 1 = A*A with the b*A + c*A^2 epilogue,
 * 2 = B*X with the a*X epilogue, 3 = norm/scale/transpose prologue and
 * output store, 4 = pack/unpack, 5 = the last step's B*X launches, which also
 * store the results (to the caller's tensors or the rank buffers), 6 = the
 * whole iteration of small matrices, one CTA per matrix. Launch
 * counters are always on. When timing
 * is enabled, every launch is bracketed by two CUDA events recorded on the
 * stream it is launched on; ns_profile_read synchronises those events. */

/* Tuning: how the bf16 GEMM phases use the tensor cores. cl = 1: one CTA per
 * 128 x 256 tile (tcgen05 cta_group::1); cl = 3: clusters of two CTAs running
 * the 2-SM MMA (cta_group::2) on 256 x 256 tiles, each SM holding half of
 * each operand; cl = 0 (default) picks 3 for the Gram and A*A phases, and 3
 * for B*X when every bucket has an even number of 128-row tile rows (else 1):
 * the fastest measured per phase. The paired mode applies to launches whose
 * buckets all have at least two 128-row tile rows; others use 1. Any other
 * value is NS_ERR_ARG. Process-wide; all modes give bitwise-identical
 * results. */
int ns_set_gemm_cluster(int cl);

/* Tuning: bf16 shape buckets with m <= 128 and n <= 512 (m, n the short and
 * long side of the 2-D view) run, when enable = 1 (the default), as one CTA per
 * matrix that keeps X, A and B in shared memory and the products in TMEM for
 * the whole iteration: one launch instead of a prologue, 3*steps GEMM
 * launches and a store. enable = 0 sends them through the GEMM launches like
 * every other bucket. Same arithmetic (bf16 operands, fp32 accumulation and
 * epilogues); results agree to rounding, not bit for bit. Other values are
 * NS_ERR_ARG. Process-wide. */
int ns_set_small_path(int enable);

/* Tuning: how the bf16 path stores the symmetric matrices A = X X^T and
 * B = b A + c A^2 (SYRK: only the tiles that touch the upper triangle are
 * computed; [ISS], SYRK symmetric kernels).
 * Both tilings compute exactly the upper 256 x 256 pair blocks of each
 * m_pad x m_pad result, in full. mode = 0 (the default): only those blocks
 * are stored, and the products that read A or B (A*A, B*X) load the K-blocks
 * left of their rows' diagonal pair block from the stored transposed block
 * (MN-major). mode = 1: the symmetric products also write the transpose of
 * every block above the diagonal pair blocks (the mirror), and the readers
 * take rows only. Other values are NS_ERR_ARG. Process-wide; both modes give
 * bitwise-identical results (the same products in the same K order). */
int ns_set_symmetric_store(int mode);

/* enable != 0 turns per-launch event timing on, 0 off. Process-wide. */
int ns_profile_enable(int enable);

/* launches[7] (may be NULL) receives the launch count per kind and gpu_ms[7]
 * (may be NULL) the summed event time per kind since the last reset; reset
 * != 0 clears both afterwards. */
int ns_profile_read(int reset, int64_t* launches, double* gpu_ms);

/* The same for the training-step operators, launches[3] and gpu_ms[3]:
 * 0 = sort, dispatch, combine and the layer for a few tokens, 1 = head norms and
 * rotation, 2 = distillation. */
int ns_profile_read_training(int reset, int64_t* launches, double* gpu_ms);

/* The same, launches[2] and gpu_ms[2]: 0 = gradient norm and clipping, 1 = block
 * norms. */
int ns_profile_read_blocks(int reset, int64_t* launches, double* gpu_ms);

#ifdef __cplusplus
}
#endif

#endif /* NSGB300_H */
