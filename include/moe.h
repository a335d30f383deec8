/*
 * moe.h -- C ABI of the GB300 (sm_103a) gated Mixture-of-Experts FFN layer, forward pass.
 *
 * One layer, one GPU, every expert resident in device memory:
 *
 *   gate      logits[t,e] = sum_i x[t,i] Wg[i,e] (fp32), softmax over experts, top-1 or
 *             top-2 by logit.  Each token is sent to experts by a gating function
 *             (DeepSpeed-MoE review, "MoE based NLG Model Architecture").
 *   dispatch  capacity C = ceil(cf T / E) per expert; assignments taken in token order,
 *             those past an expert's capacity are dropped; compact slots per expert.
 *   experts   FFN_e(x) = GeLU_tanh(x W1[e]) W2[e], fp16 operands, fp32 accumulation.
 *   combine   out[t] = sum_j w[t,j] FFN_{e_j}(x_t) over kept assignments: Top2-MoE sums the
 *             outputs of two experts (same review, "Phenomenon2").
 *   residual  mlp_type 'residual' (DeepSpeed-MoE Inference wiki, "PR-MoE 최적화로 더 낮은 비용";
 *             PR-MoE in the review) adds a fixed dense MLP GeLU(x Wr1) Wr2 to the routed
 *             expert's output (review, "Phenomenon2": Residual-MoE).
 *
 * The pages fix none of the exact formulas; the readings used are stated beside each call
 * (no biases; fp32 fused-multiply-add chain for the logits; ties go to the lower expert
 * index; top-1 weight = softmax probability of the chosen expert; top-2 weights are the two
 * probabilities renormalised to sum 1 before drops and not after; capacity independent of
 * k; dropped assignments contribute zero; GeLU in its tanh form).
 *
 * Conventions for every call:
 *   - Matrices are dense row-major.  Shapes are given as [rows, cols].
 *   - Every pointer argument is a DEVICE pointer owned by the caller, unless stated.  The
 *     library never allocates or frees device memory, keeps no pointer after a call
 *     returns, and never synchronises `stream` (moe_status_read excepted).
 *   - All work is enqueued on `stream` (a cudaStream_t; 0 is the legacy default stream);
 *     calls return once the work is enqueued.
 *   - Return value: a moe_status.  Argument errors are detected on the host before anything
 *     is enqueued, and nothing is written then.  MOE_ERR_CUDA reports a failed launch.
 *     Errors found on the device while a call runs (a bounded wait that gave up) are
 *     recorded in the workspace's status word and read with moe_status_read.
 *   - No call throws across this boundary; all are safe to call from any host thread as
 *     long as concurrent calls use different workspaces and outputs.
 *   - T = 0 (an empty batch) is valid: the call enqueues nothing and returns MOE_OK (the
 *     training calls clear what is summed over the batch, and their status word).
 *
 * Supported shapes: E <= 1024, k in {1, 2}, k <= E.  MOE_F16 (tensor-core path): d, f and
 * f_res multiples of 128.  MOE_F32 (SIMT path): d and f multiples of 4.  Every pointer
 * 16-byte aligned.  Otherwise MOE_ERR_UNSUPPORTED.
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define MOE_API __attribute__((visibility("default")))
#else
#define MOE_API
#endif

typedef struct CUstream_st* moe_stream_t; /* same type as cudaStream_t */

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,    /* a size, pointer, k, capacity factor or enum is invalid */
  MOE_ERR_UNSUPPORTED = 2,    /* valid, but a shape / alignment this build does not run */
  MOE_ERR_WORKSPACE = 3,      /* workspace missing or smaller than moe_workspace_size */
  MOE_ERR_CUDA = 4,           /* a CUDA launch or API call failed */
  MOE_ERR_TIMEOUT = 5,        /* device side: a bounded wait gave up (status word) */
  MOE_ERR_DEVICE_BOUNDS = 6   /* device side: an index failed its bounds check (status word):
                                 the expert FFN's offsets left [0, S_max] or decreased, or a
                                 perm entry left [0, T).  The offending index is clamped (no
                                 access leaves its buffer) and the outputs are unspecified.
                                 moe_combine's slot_of is not checked (the call has no bound
                                 for it): pass it as moe_dispatch writes it */
} moe_status;

typedef enum { MOE_F32 = 0, MOE_F16 = 1 } moe_dtype;           /* activations and expert weights */
typedef enum { MOE_MLP_STANDARD = 0, MOE_MLP_RESIDUAL = 1 } moe_mlp_type;

/*
 * Capacity per expert: C = ceil(cf * T / E), with cf*T and the division evaluated in
 * double.  The pages define no per-expert token capacity: the "expert capacity" of the
 * DeepSpeed-MoE review ("Phenomenon2") is the number of experts each token passes through
 * (k here; Top2-MoE doubles it).  The token capacity of an expert is therefore a reading:
 * the capacity-factor rule above, with overflow dropped in token order.  Host only.
 * cf = +INFINITY selects the dropless mode: C = T, so no assignment is dropped and a hot
 * expert's rows are spread over as many tiles as it needs (the single-GPU counterpart of the
 * physical expert replicas of "Fast MoE Inference via Predictive Prefetching and Expert
 * Replication", methodology).  Every entry taking a capacity factor accepts it.
 * Returns C (0 when T = 0), or -1 when T < 0, E < 1, cf <= 0 or NaN, or C > 2^31-1.
 */
MOE_API int moe_capacity(int T, int E, float capacity_factor);

/*
 * Bytes of workspace that moe_layer_forward needs for this shape (and enough for
 * moe_expert_ffn of the same shape).  Host only; writes *bytes.  f_res is ignored for
 * MOE_MLP_STANDARD.  Returns MOE_ERR_INVALID_ARG / MOE_ERR_UNSUPPORTED as the calls would.
 */
MOE_API moe_status moe_workspace_size(int T, int d, int f, int E, int k, float capacity_factor,
                              moe_mlp_type mlp_type, int f_res, moe_dtype dtype, size_t* bytes);

/*
 * Gate: logits, softmax and top-k (DeepSpeed-MoE review, "MoE based NLG Model
 * Architecture": tokens reach experts through a gating function; "Phenomenon2": Top2).
 *   tokens     [T, d] in `dtype` (f16 values are widened exactly to f32).
 *   Wg         [d, E] float32.
 *   logits_in  nullable [T, E] float32: when given, the logits are taken from here and
 *              tokens / Wg are not read (may be NULL then).
 *   logits_out [T, E] float32: the logits used; required when logits_in is NULL (it holds
 *              them), otherwise nullable (a copy of logits_in).
 *   probs_out  nullable [T, E] float32: softmax over E.
 *   topk_idx   [T, k] int32: experts by descending logit, ties to the lower index.
 *   topk_w     [T, k] float32: k = 1: p[e1]; k = 2: p[e_j] / (p[e1] + p[e2]).
 * The logits are the fp32 chain acc = fmaf(x[t,i], Wg[i,e], acc), i ascending from +0, so
 * they (and hence routing) are reproducible bit for bit by any IEEE implementation.
 */
MOE_API moe_status moe_gate_topk(const void* tokens, moe_dtype dtype, const float* Wg,
                                 const float* logits_in, int T, int d, int E, int k, float* logits_out,
                         float* probs_out, int32_t* topk_idx, float* topk_w, moe_stream_t stream);

/*
 * Capacity-limited dispatch (reading: token-major order, capacity ceil(cf T / E)).
 *   topk_idx   [T, k] int32 experts; an index outside [0, E) is not counted and its
 *              assignment is dropped (slot_of = -1).
 *   counts_raw [E]    assignments per expert before the capacity cut.
 *   kept       [E]    min(counts_raw, C).
 *   offsets    [E+1]  exclusive scan of kept; offsets[E] = S, the number of kept slots.
 *   perm       [min(T k, E C)]  perm[s] = token of slot s; expert e owns slots
 *                               offsets[e] .. offsets[e+1]-1 in token order.  Entries >= S
 *                               are not written.
 *   slot_of    [T, k] slot of assignment (t, j), or -1 when it was dropped.
 * Pure integer work: results are unique and bit-exact.  One thread block; no atomics.
 */
MOE_API moe_status moe_dispatch(const int32_t* topk_idx, int T, int E, int k, float capacity_factor,
                        int32_t* counts_raw, int32_t* kept, int32_t* offsets, int32_t* perm,
                        int32_t* slot_of, moe_stream_t stream);

/*
 * Dispatch of one shard of a token-sharded batch, with the whole batch's capacity rule.
 * The pages have no multi-GPU data-parallel layout of this layer (their own design is expert
 * parallelism); this entry is the one exchange step that token sharding needs so that
 * routing does not depend on how the batch is split (capacity as moe_capacity computes it,
 * ceil(cf T / E) of the whole batch, with drops in token order).
 *   The batch of T_global tokens is split over n_ranks callers in token order; this call
 *   holds shard `rank` (T tokens).  counts_all [n_ranks, E] int32 (device; nullable when
 *   rank == 0): the counts_raw of every shard in rank order, exchanged by the caller (for
 *   example an all_gather of each shard's counts_raw from moe_dispatch).
 *   C = ceil(cf T_global / E).  An assignment is kept iff (assignments to its expert in
 *   earlier shards) + (its rank within this shard) < C, so the kept / dropped decisions are
 *   those of moe_dispatch on the whole batch.
 *   Outputs as moe_dispatch, local to the shard: counts_raw / kept per expert for this
 *   shard, offsets / perm / slot_of over this shard's compact slots (perm holds local token
 *   indices), perm sized min(T k, E C).
 * Errors: MOE_ERR_INVALID_ARG for T_global < T, rank outside [0, n_ranks), or counts_all
 * NULL with rank > 0; otherwise as moe_dispatch.  T = 0 is a valid no-op.
 */
MOE_API moe_status moe_dispatch_sharded(const int32_t* topk_idx, int T, int E, int k,
                                        float capacity_factor, int T_global,
                                        const int32_t* counts_all, int n_ranks, int rank,
                                        int32_t* counts_raw, int32_t* kept, int32_t* offsets,
                                        int32_t* perm, int32_t* slot_of, moe_stream_t stream);

/*
 * Grouped expert FFN over the dispatched slots, unscaled:
 *   expert_out[s, :] = GeLU_tanh(tokens[perm[s], :] W1[e]) W2[e]   for s in expert e's slots.
 *   tokens [T, d], W1 [E, d, f], W2 [E, f, d], expert_out [S_max, d]: all in `dtype`.
 *   perm, offsets: as written by moe_dispatch.  S_max >= offsets[E] bounds the slot count
 *   (min(T k, E C) always suffices).  Rows >= offsets[E] of expert_out are not written.
 *   Bounds: the kernels clamp offsets to [0, S_max], so no row >= S_max of expert_out or of
 *   the workspace is ever written; offsets outside that range or decreasing, and perm
 *   entries outside [0, T), record MOE_ERR_DEVICE_BOUNDS in the workspace's status word
 *   (moe_status_read).
 *   workspace: >= 256 + S_max * f * sizeof(dtype) bytes, rounded up to a multiple of 256
 *   (the status word, then the hidden activations H [S_max, f]); moe_workspace_size of the
 *   same layer shape is always enough for S_max = min(T k, E C).
 * f16: hidden activations are rounded to f16 between the two GEMMs.
 */
MOE_API moe_status moe_expert_ffn(const void* tokens, const int32_t* perm, const int32_t* offsets,
                          const void* W1, const void* W2, moe_dtype dtype, int T, int d, int f,
                          int E, int S_max, void* expert_out, void* workspace, size_t ws_bytes,
                          moe_stream_t stream);

/*
 * Gate-weighted combine back to token order (DeepSpeed-MoE review, "Phenomenon2": the
 * outputs of the experts a token visits are summed; Residual-MoE adds a fixed MLP):
 *   out[t, :] = sum_j [slot_of[t,j] >= 0] topk_w[t,j] expert_out[slot_of[t,j], :]
 *               (+ residual_in[t, :] when residual_in is not NULL)
 * in fp32, j ascending, the residual added last, rounded once to `dtype`.
 *   expert_out [S, d], residual_in nullable [T, d], out [T, d]: all in `dtype`.
 */
MOE_API moe_status moe_combine(const void* expert_out, const int32_t* slot_of, const float* topk_w,
                       const void* residual_in, moe_dtype dtype, int T, int d, int k, void* out,
                       moe_stream_t stream);

/*
 * The whole layer, fused: gate, dispatch, expert GEMM1 + GeLU, expert GEMM2 with the
 * gate-weighted combine in its epilogue, and for MOE_MLP_RESIDUAL the dense MLP
 *   out[t] += GeLU(x_t Wr1) Wr2,   Wr1 [d, f_res], Wr2 [f_res, d]   (NULL for STANDARD),
 * computed by the same grouped-GEMM kernels as an extra group of all T tokens.
 *   tokens [T, d], W1 [E, d, f], W2 [E, f, d], out [T, d]: `dtype`.  Wg [d, E]: float32.
 *   topk_idx_out nullable [T, k], slot_of_out nullable [T, k]: routing, as moe_gate_topk /
 *   moe_dispatch define it.
 *   workspace >= moe_workspace_size(...) bytes; contents need no initialisation.
 *   out must not overlap tokens or the workspace: it is cleared before the experts' outputs
 *   are added into it.
 * Deterministic: repeated calls give identical bits.  Top-1 standard layers write each
 * output row once.  Where an output element has two addends (top-2, or one expert plus the
 * residual MLP), each is rounded to `dtype` and added into the cleared output: 0 + a is exact
 * and a + b commutes, so the order of the additions does not matter.  Top-2 with the residual
 * MLP (three addends) sums in fp32 in a fixed order and rounds once.
 */
MOE_API moe_status moe_layer_forward(const void* tokens, const float* Wg, const void* W1, const void* W2,
                             const void* Wr1, const void* Wr2, moe_dtype dtype, int T, int d,
                             int f, int E, int k, float capacity_factor, moe_mlp_type mlp_type,
                             int f_res, void* out, int32_t* topk_idx_out, int32_t* slot_of_out,
                             void* workspace, size_t ws_bytes, moe_stream_t stream);

/*
 * Synchronises `stream`, then returns the device-side status word of the most recent
 * moe_expert_ffn / moe_layer_forward / moe_adapter_forward / moe_adapter_backward call, or
 * moe_gate_topk_backward call with dWg or dtokens, on this workspace (MOE_OK, MOE_ERR_TIMEOUT
 * or MOE_ERR_DEVICE_BOUNDS), or MOE_ERR_CUDA if the synchronisation or the read failed.  Each of
 * those calls sets the word anew (of the empty ones the training calls; the others enqueue nothing).
 */
MOE_API moe_status moe_status_read(const void* workspace, moe_stream_t stream);

/* Static, human-readable name of a status code ("MOE_OK", ...). */
MOE_API const char* moe_status_string(moe_status status);

/*
 * Self-test of the device-side bounded wait that every pipeline wait in the library uses:
 * launches one block that waits on an mbarrier nothing ever arrives on, with a budget of
 * timeout_ns nanoseconds (1 .. 10^10) instead of the library's default of 2 s.  The wait
 * gives up, records MOE_ERR_TIMEOUT in the workspace's status word and the kernel returns
 * normally, leaving the context usable; read the result with moe_status_read.
 * workspace: >= 256 bytes.
 */
MOE_API moe_status moe_selftest_wait(void* workspace, uint64_t timeout_ns, moe_stream_t stream);

/*
 * Measurement hook (the pages have no counterpart): when `events` is not NULL, the calling
 * thread's next moe_layer_forward calls record events[0 .. 6] (cudaEvent_t handles created
 * by the caller) on their stream at the stage boundaries: [0] start, [1] after the gate
 * logits, [2] after softmax / top-k, [3] after dispatch, [4] after the first expert GEMM
 * (+ GeLU), [5] after the second expert GEMM (+ combine), [6] at the end.  n_events must be
 * 7, or 0 with events NULL to stop recording.  Thread-local; host only.
 */
#define MOE_STAGE_EVENTS 7
MOE_API moe_status moe_set_stage_events(void* const* events, int n_events);

/*
 * Measurement hook (the pages have no counterpart): the number of kernels this library has
 * enqueued in this process so far, counted on the host at each successful launch.  Inside a
 * stream capture a launch is counted once when captured (not per graph replay), so the
 * difference across a capture is the number of kernels per replay.  Never fails.
 */
MOE_API unsigned long long moe_kernel_launches(void);

/*
 * ---- Training the router and low-rank adapters of a layer whose experts stay as they are ----
 *
 * The pages have no counterpart of the calls from here to moe_adapter_backward: they are the
 * gradients of moe_gate_topk and moe_combine, the losses that keep a router balanced, and
 * low-rank adapters of many requests beside the layer (or any projection of its tokens).
 * An empty batch (T = 0) is valid for each: outputs with a row per token or slot have none, and
 * what is summed over the batch (counts, losses, dWg, dA, dB) is written as zeros.
 * Deterministic: equal calls give equal bits.  All sums are in float32 or wider; the softmax takes the
 * hardware's exponential, good to 2 + 1.2 |x - max| units of the last place.
 * They go with the staged calls (moe_gate_topk, moe_dispatch, moe_expert_ffn, moe_combine), whose
 * logits, gate weights and expert outputs they read; moe_layer_forward hands none of these out.  The
 * gradient of the expert FFN (dexpert_out to its tokens) and of the residual MLP is the caller's: what
 * these calls write to dtokens are the gate's and the adapters' addends of the tokens' gradient.
 */

/* Bytes of workspace of moe_balance_loss.  Host only; writes *bytes. */
MOE_API moe_status moe_balance_workspace_size(int T, int E, size_t* bytes);

/*
 * Router losses and per-expert counts of a batch routed by moe_gate_topk:
 *   p = softmax(logits[t, :]),  n = number of tokens that count,
 *   counts[e]    = #{(t, j): t counts, topk_idx[t, j] = e}    (before any capacity cut),
 *   prob_mean[e] = 1/n sum_t p[t, e],
 *   losses[0]    = E sum_e counts[e] / (n k) prob_mean[e]     (balance; 1 for a uniform router),
 *   losses[1]    = 1/n sum_t (log sum_e exp logits[t, e])^2   (z).
 *   logits     [T, E] float32, topk_idx [T, k] int32 (an index outside [0, E) is not counted).
 *   token_mask nullable [T] bytes: tokens with 0 (padding) do not count; what their rows hold
 *              (infinities, NaN) has no effect.
 *   n_valid    [1] int32: n.  n = 0 gives zero losses.
 * A row of -infinity only adds nothing to prob_mean and to the z loss, but counts in n.
 *   workspace: moe_balance_workspace_size bytes; contents need no initialisation.
 */
MOE_API moe_status moe_balance_loss(const float* logits, const int32_t* topk_idx,
                                    const uint8_t* token_mask, int T, int E, int k, int32_t* counts,
                                    float* prob_mean, float* losses, int32_t* n_valid,
                                    void* workspace, size_t ws_bytes, moe_stream_t stream);

/*
 * Bytes of workspace of moe_gate_topk_backward when it takes the gradient to Wg or the tokens.  The
 * bytes of a batch are enough for every smaller T.
 */
MOE_API moe_status moe_gate_backward_workspace_size(int T, int d, int E, moe_dtype dtype,
                                                    size_t* bytes);

/*
 * Gradient of moe_gate_topk's gate weights and of moe_balance_loss's losses:
 *   dlogits [T, E] = d/dlogits ( sum dtopk_w . topk_w + dlosses[0] balance + dlosses[1] z ),
 * with topk_idx and counts held constant, and from it
 *   dWg [d, E]     = tokens^T dlogits                               (float32),
 *   dtokens [T, d] = dtokens_in + dlogits Wg^T                      (`dtype`, rounded once).
 *   logits, topk_idx  as given to / written by moe_gate_topk (indices outside [0, E), or a pair
 *                     of equal ones, carry no gradient of their weights).
 *   dtopk_w    nullable [T, k] float32.
 *   dlosses    nullable [2] float32 (device): gradients of the two losses (their coefficients
 *              times what comes from above).  With it, counts [E] and n_valid [1] as
 *              moe_balance_loss wrote them; for a batch spread over several callers, both
 *              summed over the callers first.  NULL: counts and n_valid are not read.
 *   token_mask nullable [T]: rows of tokens with 0 are zero (dtokens: dtokens_in).
 *   dWg nullable (then tokens is not read), dtokens nullable (then Wg is not read), dtokens_in
 *   nullable (zero; may be dtokens itself).
 *   workspace: moe_gate_backward_workspace_size bytes; may be NULL when dWg and dtokens are.
 *   Otherwise no output overlaps an input (dtokens and tokens the same: MOE_ERR_INVALID_ARG).
 *   token_mask also leaves the masked tokens' rows out of dWg: what they hold has no effect.
 *   MOE_F16: dlogits and Wg may enter the products to 2^-23 of each value and 2^-36 of the largest of
 *   128 rows; in dWg a token's values below 2^-14 lose bits as if they were 2^-14.
 * Shapes: those of moe_gate_topk, T <= 2^30, and for dWg / dtokens d a multiple of 8 (MOE_F16) or
 * 4, at most 2^20.
 * Speed: MOE_F16 with E <= 256 runs on the 5th-generation tensor cores; MOE_F32, and dtokens of more
 * experts, take multiply-adds (T = 4096, d = 1024, both gradients: E = 256 40 us, E = 257 186 us).
 */
MOE_API moe_status moe_gate_topk_backward(const float* logits, const int32_t* topk_idx,
                                          const float* dtopk_w, const float* dlosses,
                                          const int32_t* counts, const int32_t* n_valid,
                                          const uint8_t* token_mask, const void* tokens,
                                          const float* Wg, moe_dtype dtype, int T, int d, int E,
                                          int k, float* dlogits, float* dWg, const void* dtokens_in,
                                          void* dtokens, void* workspace, size_t ws_bytes,
                                          moe_stream_t stream);

/*
 * Gradient of moe_combine.  For every assignment with s = slot_of[t, j] in [0, S_max):
 *   dexpert_out[s, :] = topk_w[t, j] dout[t, :]           (`dtype`, rounded once),
 *   dtopk_w[t, j]     = sum_i dout[t, i] expert_out[s, i] (float32; 0 for a dropped assignment).
 *   dout [T, d], expert_out and dexpert_out [S_max, d] in `dtype`.  Slots that no assignment
 *   names are left as they were.  dexpert_out nullable (then topk_w is not read), dtopk_w
 *   nullable (then expert_out is not read); not both.  residual_in's gradient is dout itself.
 *   dexpert_out does not overlap dout, nor expert_out.
 *   A slot that two assignments name (moe_dispatch names none twice) gets one of their rows.
 * Shapes: T <= 2^30, d <= 2^20.
 */
MOE_API moe_status moe_combine_backward(const void* dout, const void* expert_out,
                                        const int32_t* slot_of, const float* topk_w, moe_dtype dtype,
                                        int T, int d, int k, int S_max, void* dexpert_out,
                                        float* dtopk_w, moe_stream_t stream);

/*
 * Bytes of workspace that moe_adapter_forward and moe_adapter_backward need for this shape.  The
 * bytes of an S_max are enough for every smaller one (and any T).
 */
MOE_API moe_status moe_adapter_workspace_size(int T, int d_in, int d_out, int r, int N, int S_max,
                                              moe_dtype dtype, size_t* bytes);

/*
 * Low-rank adapters of many requests beside a shared projection.  For every slot s of adapter n
 * (offsets[n] <= s < offsets[n+1]) and its token t = perm[s]:
 *   hidden[s, :] = tokens[t, :] A[n]                         (float32),
 *   out[t, :]    = base[t, :] + scale[n] (hidden[s, :] B[n]) (`dtype`, rounded once).
 *   perm, offsets: as moe_dispatch writes them for the adapter index of each token in place of
 *   topk_idx (k = 1, E = N, capacity_factor = +INFINITY); an index outside [0, N) gives a token
 *   no adapter.  One plan serves every projection of a step.
 *   tokens [T, d_in], A [N, d_in, r], B [N, r, d_out], base (nullable: zero) and out [T, d_out]
 *   in `dtype`; scale [N] float32.  base may be out itself (the shared projection's result, in
 *   place).  Rows of out whose token has no adapter are left as they were.  Otherwise out
 *   overlaps no input (out and tokens the same: MOE_ERR_INVALID_ARG).  A token named by more
 *   than one slot (moe_dispatch names none twice) gets one of their results in each element; with
 *   base = out no token may be (a result that is written may be read as the other's base).
 *   hidden nullable [S_max, r] float32, for the backward pass; rows >= offsets[N] are not written.
 *   Bounds: as moe_expert_ffn's: no slot >= S_max is used, and offsets outside [0, S_max] or
 *   decreasing and perm entries outside [0, T) are skipped and recorded as
 *   MOE_ERR_DEVICE_BOUNDS in the workspace's status word.
 *   workspace: moe_adapter_workspace_size bytes; contents need no initialisation.
 * MOE_F16: hidden is given out in float32, and the second product takes it to 2^-23 (and 2^-39
 * of the row's largest value), so that out is what float32 sums give, rounded once.  (An infinite
 * weight makes what it enters infinite or NaN.)
 * Shapes: N <= 1024; r a multiple of 8, at most 128 (adapters of different ranks are padded with
 * zeros); d_in, d_out multiples of 8 (MOE_F16) or 4 (MOE_F32), at most 2^20; T, S_max <= 2^30.
 * Speed: long runs cost the same from r = 72 to 128, and 1.8 times r = 64 (16384 rows of 3584 columns:
 * 170 us and 96 us); MOE_F32 takes multiply-adds in tiles of 16 rows.
 */
MOE_API moe_status moe_adapter_forward(const void* tokens, const int32_t* perm,
                                       const int32_t* offsets, const void* A, const void* B,
                                       const float* scale, const void* base, moe_dtype dtype, int T,
                                       int d_in, int d_out, int r, int N, int S_max, void* out,
                                       float* hidden, void* workspace, size_t ws_bytes,
                                       moe_stream_t stream);

/*
 * Gradient of moe_adapter_forward, with dh[s, :] = dout[perm[s], :] B[n]^T:
 *   dtokens[t, :] = dtokens_in[t, :] + scale[n] (dh[s, :] A[n]^T)   (`dtype`, rounded once),
 *   dA[n] = scale[n] sum_s tokens[perm[s], :]^T dh[s, :],   dB[n] = scale[n] sum_s hidden[s, :]^T
 *   dout[perm[s], :]   (float32 [N, d_in, r] and [N, r, d_out]; zero for an adapter without slots).
 *   hidden: as moe_adapter_forward wrote it.  dtokens nullable; dtokens_in nullable (zero) and
 *   may be dtokens itself; dA nullable (then tokens is not read), dB nullable (then hidden is
 *   not read); not all three.  base's gradient is dout itself.
 *   dtokens overlaps neither dout nor tokens (the same: MOE_ERR_INVALID_ARG).
 *   With dtokens_in = dtokens no token is named by more than one slot.
 *   MOE_F16: dA and dB take dh and hidden to 2^-23 of each value and 2^-39 of the largest of 64 rows;
 *   values of tokens and dout below 2^-14 lose bits as if they were 2^-14.
 *   Everything else as moe_adapter_forward (dh in hidden's place).  MOE_F16, long runs: an infinite
 *   token or dout row makes its sums infinite or NaN.
 */
MOE_API moe_status moe_adapter_backward(const void* dout, const void* tokens, const float* hidden,
                                        const int32_t* perm, const int32_t* offsets, const void* A,
                                        const void* B, const float* scale, const void* dtokens_in,
                                        moe_dtype dtype, int T, int d_in, int d_out, int r, int N,
                                        int S_max, void* dtokens, float* dA, float* dB,
                                        void* workspace, size_t ws_bytes, moe_stream_t stream);

/*
 * Allocation-free variant of moe_expert_ffn (the pages have no counterpart).
 *
 * For callers that cannot allocate device memory where they run the layer: a plugin or
 * custom operator inside a host framework that owns all device memory and gives its
 * plugins no workspace, or a serving loop that forbids cudaMalloc after start-up because it
 * can synchronise the device.  They pass inputs and outputs only; the scratch (the hidden
 * activations H [S_max, f]) lives in a fixed 64 MiB array compiled into the library, which
 * every GPU that loads the library keeps until the process exits.
 *   Arguments and results: as moe_expert_ffn, without the workspace.
 *   Limit: S_max * f * sizeof(dtype) <= 64 MiB, else MOE_ERR_WORKSPACE (nothing runs).
 *   The first call on each device looks up the array's device address (with that device
 *   current) and keeps it; make that first call before any stream capture, and make no call
 *   on a device after a reset of it (cudaDeviceReset), which invalidates the kept address.
 *   All calls share the one array and it keeps the last call's contents: calls that
 *   overlap on the GPU race on it (order them on one stream).  Device-side wait timeouts
 *   are not reported by this variant (it has no status word to read).
 *   Calls no cudaMalloc, cudaFree or other allocating routine.
 */
MOE_API moe_status moe_expert_ffn_noalloc(const void* tokens, const int32_t* perm,
                                          const int32_t* offsets, const void* W1, const void* W2,
                                          moe_dtype dtype, int T, int d, int f, int E, int S_max,
                                          void* expert_out, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H_ */
