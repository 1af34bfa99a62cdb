/*
 * gdn.h -- C ABI of the chunked Gated DeltaNet (gated delta rule) forward and
 * backward for NVIDIA GB300 (sm_103a).
 *
 * The operation.  Per batch row b and value head j (key head kh = j / (Hv/Hk)),
 * with the state written transposed, h = S^T of shape d_k x d_v:
 *     h_t = exp(g_t) (I - beta_t k_t k_t^T) h_{t-1} + beta_t k_t v_t^T,
 *     o_t = h_t^T q_t,          h_{-1} = h0,  hT = h_{T-1}.
 * It is evaluated in chunks of `chunk` tokens through the WY/UT form: per chunk
 * the UT inverse T = (I + S)^-1 of S = tril(diag(beta) (K K^T * decay), -1)
 * (blockwise doubling ladder), w = T diag(beta exp(G)) K, u = T diag(beta) V,
 * the inter-chunk step h' = (exp(g_last) I - k_g^T w) h + k_g^T u = A h + B,
 * and the masked intra-chunk output.  Sources (pages' titles and sections):
 *   - the inter-chunk step as an affine map h' = A h + B and the composition
 *     law (A2,B2) o (A1,B1) = (A2 A1, A2 B1 + B2): issue "GatedDeltaNet does
 *     not support ici_context_parallelism", section "The recurrence is affine,
 *     so it can be parallelized";
 *   - the two-pass scan (fold each stretch of chunks into one (A, B), exclusive
 *     prefix, replay from the incoming state): PR "Shard the GatedDeltaNet
 *     sequence under ici_context_parallelism", description;
 *   - the ladder inverse, its analytic backward dS = -(T^T dT T^T) (strictly
 *     lower), the reverse chunk walk of the backward and initial/final state
 *     as first-class inputs/outputs: PR "Fuse the Gated Delta Net inter-chunk
 *     scan into a Pallas TPU kernel", section "Changes".
 *
 * Conventions for every entry point:
 *   - Pointers are device pointers (cudaMalloc'd, or any memory the device can
 *     address), contiguous, 16-byte aligned.  bf16 tensors are passed as
 *     void* to raw IEEE bfloat16 data.  The caller owns all memory; the
 *     library allocates nothing, keeps no state between calls and never
 *     synchronises the stream -- except gdn_chunk_fwd_noalloc, whose fixed
 *     scratch array (in the library's device image) and per-device address
 *     cache persist between calls (see its declaration), and the status
 *     readers, which synchronise.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  All work
 *     is enqueued on it asynchronously; outputs are valid once it has run.
 *   - Layouts: q, k [B, T, Hk, d_k]; v, o, dO, dv [B, T, Hv, d_v];
 *     g, beta, dg, dbeta [B, T, Hv]; h0, hT, dhT, dh0 [B, Hv, d_k, d_v];
 *     dq, dk [B, T, Hk, d_k].
 *   - Return value: GDN_OK, or a negative gdn_status.  Argument errors are
 *     detected on the host before anything is enqueued, so a failed call has
 *     no effect.  GDN_ERR_CUDA reports a launch failure (cudaGetLastError).
 *   - Supported sizes in this version: d_k = d_v = 128, chunk = 128, any
 *     T >= 0 (a ragged last chunk is zero-padded with g = 0, beta = 0, which
 *     leaves the state unchanged), Hv a multiple of Hk.  The forward entry
 *     points (gdn_chunk_fwd, its _timed and _ex variants without a saved
 *     buffer, gdn_chunk_fwd_noalloc, gdn_segment_fold, gdn_layer_fwd,
 *     gdn_debug_ut and their workspace sizes) also take chunk = 64 (PR "Shard
 *     the GatedDeltaNet sequence under ici_context_parallelism", review
 *     thread: forming each device's A_loc with 64-token chunks): the state
 *     then steps every 64 tokens.  The backward entry points, and a forward
 *     that keeps tiles for them, take chunk = 128 only (GDN_ERR_SHAPE
 *     otherwise); their results do not depend on the chunk size beyond
 *     rounding, so a backward with chunk = 128 serves a forward run with 64.
 *   - Workspace: the caller passes `ws` of at least the size the matching
 *     *_workspace_bytes call returns for the same arguments (256-byte aligned).
 *     Its contents on entry do not matter.  Its first 4 bytes are a status
 *     word: the call clears it, and a kernel sets bit 0 if one of its bounded
 *     waits gives up (gdn_workspace_status reads it).
 *   - Bounded waits: the kernels wait only inside one block (for their TMA
 *     copies, their tensor-core products and hand-offs between their warps);
 *     every such wait gives up after 2e9 SM cycles (about one second), so
 *     a fault can leave wrong outputs and a set status bit but never a hung
 *     GPU.
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gdn_status {
  GDN_OK = 0,
  GDN_ERR_ARG = -1,        /* null required pointer, misalignment, Hv % Hk != 0, negative size */
  GDN_ERR_SHAPE = -2,      /* unsupported d_k, d_v or chunk */
  GDN_ERR_WORKSPACE = -3,  /* workspace missing or smaller than required */
  GDN_ERR_CUDA = -4,       /* a kernel launch failed */
  GDN_ERR_TIMEOUT = -5,    /* a bounded in-kernel wait gave up (see gdn_workspace_status) */
  GDN_ERR_UNSUPPORTED = -6 /* device is not sm_103 / sm_100 class */
} gdn_status;

/* Human-readable text of a status code (static storage, never NULL). */
const char* gdn_strerror(int status);

/* Number of chunk segments the forward/backward use when n_segments == 0: one
 * when the chunks are few or the batch rows and value heads already keep a
 * quarter of the SMs busy with the one-segment walk (4 CTAs each), else enough
 * segments to fill the SMs about twice with the segment fold (8 CTAs per
 * segment and head), at least 8 chunks each. */
int gdn_default_segments(int B, int T, int Hv, int chunk);

/*
 * Workspace bytes of gdn_chunk_fwd / gdn_chunk_bwd for these arguments
 * (n_segments as it will be passed, 0 = automatic).  Returns 0 for invalid
 * sizes.
 */
size_t gdn_fwd_workspace_bytes(int B, int T, int Hk, int Hv, int d_k, int d_v, int chunk,
                               int n_segments);
size_t gdn_bwd_workspace_bytes(int B, int T, int Hk, int Hv, int d_k, int d_v, int chunk,
                               int n_segments);

/*
 * Forward.  Reads q, k, v (bf16), g, beta (fp32, g is the per-token log-gate,
 * exp(g) the decay), h0 (fp32, NULL = zero state); writes o (bf16) and hT
 * (fp32, NULL = not written).
 * n_segments: 1 = one sequential walk over the chunks per (b, value head);
 * S > 1 = the two-pass segment scan with S segments of whole chunks (segment
 * s holds chunks [floor(sN/S), floor((s+1)N/S)) of the N chunks); 0 = the
 * library's choice (gdn_default_segments).  Results agree across segment
 * counts up to rounding.
 */
int gdn_chunk_fwd(const void* q, const void* k, const void* v, const float* g,
                  const float* beta, const float* h0, void* o, float* hT, int B, int T,
                  int Hk, int Hv, int d_k, int d_v, int chunk, int n_segments, void* ws,
                  size_t ws_bytes, void* stream);

/*
 * Backward of gdn_chunk_fwd.  Takes the forward's inputs plus the output
 * cotangent dO (bf16, required) and the final-state cotangent dhT (fp32,
 * NULL = zero).  Writes dq, dk (bf16, summed over the value heads that share
 * each key head), dv (bf16), dg, dbeta (fp32) and dh0 (fp32, NULL = not
 * written).  The forward states are recomputed (nothing is saved from the
 * forward call).  n_segments as for the forward (it segments the reverse walk
 * of the state cotangent and the recomputation of the states).
 */
int gdn_chunk_bwd(const void* q, const void* k, const void* v, const float* g,
                  const float* beta, const float* h0, const void* dO, const float* dhT,
                  void* dq, void* dk, void* dv, float* dg, float* dbeta, float* dh0, int B,
                  int T, int Hk, int Hv, int d_k, int d_v, int chunk, int n_segments, void* ws,
                  size_t ws_bytes, void* stream);

/*
 * Keeping the forward's per-chunk quantities for the backward.  The backward
 * needs, per chunk, the forward's w, u, P and the UT inverse T; gdn_chunk_bwd
 * recomputes them (one launch of the preparation).  A training step that runs
 * the backward of the same inputs right after the forward can instead let the
 * forward keep them in a caller buffer `saved` of gdn_saved_bytes bytes (w, u,
 * P, T, the state entering every chunk and Delta = u - w h, bf16,
 * [B, Hv, ceil(T/chunk), 128, 128] each, and with segments the state entering
 * every segment, fp32 [B, Hv, S, 128, 128]) and pass it to the backward, which
 * then skips the preparation and the recompute of the states (and, with
 * segments, the fold and prefix that recompute the segments' entering states):
 * it runs the reverse walk of the state cotangent and the gradients only.  The pages' own fused kernel
 * keeps the inverse for its backward in the same way (PR "Fuse the Gated
 * Delta Net inter-chunk scan into a Pallas TPU kernel", section "Changes":
 * the backward's analytic inverse gradient takes T from the forward).
 *
 * gdn_chunk_fwd_ex / gdn_chunk_bwd_ex are gdn_chunk_fwd / gdn_chunk_bwd (and,
 * with events, their timing variants) with that buffer: saved = NULL gives
 * exactly the plain calls; otherwise the forward writes w, u, P, T into it and
 * the backward reads them there, and must be given the forward's inputs
 * unchanged (q, k, v, g, beta, h0, B, T, Hk, Hv, n_segments).  Results are
 * those of the plain calls.  saved is 16-byte aligned; a smaller saved_bytes
 * than gdn_saved_bytes (for the same n_segments) gives GDN_ERR_WORKSPACE.
 * Launch order of the backward with a saved buffer: reverse walk (with
 * segments: reverse fold, reverse prefix, reverse walk), gradients.
 */
size_t gdn_saved_bytes(int B, int T, int Hk, int Hv, int d_k, int d_v, int chunk, int n_segments);
int gdn_chunk_fwd_ex(const void* q, const void* k, const void* v, const float* g,
                     const float* beta, const float* h0, void* o, float* hT, int B, int T,
                     int Hk, int Hv, int d_k, int d_v, int chunk, int n_segments, void* saved,
                     size_t saved_bytes, void* ws, size_t ws_bytes, void* stream,
                     void* const* events, int n_events);
int gdn_chunk_bwd_ex(const void* q, const void* k, const void* v, const float* g,
                     const float* beta, const float* h0, const void* dO, const float* dhT,
                     void* dq, void* dk, void* dv, float* dg, float* dbeta, float* dh0, int B,
                     int T, int Hk, int Hv, int d_k, int d_v, int chunk, int n_segments,
                     const void* saved, size_t saved_bytes, void* ws, size_t ws_bytes,
                     void* stream, void* const* events, int n_events);

/*
 * One GatedDeltaNet layer's use of the rule, with the element-wise operations
 * around it (PR "Shard the GatedDeltaNet sequence under
 * ici_context_parallelism", description: the layer's "qkvz" activations
 * [B, T, H, D], of which q and k enter the rule normalised and z gates its
 * output; the pages do not define these operations further, so the plain
 * forms below are this library's reading):
 *   q_n = q / sqrt(sum q^2 + 1e-6), k_n likewise, per token and key head;
 *   beta = sigmoid(b), g = -softplus(a), per token and value head -- applied
 *     by the rule's kernels where they load the gates (the logits a and b
 *     are what the caller passes);
 *   o = the rule on (q_n, k_n, v, g, beta, h0)            (as gdn_chunk_fwd);
 *   y = o * silu(z), silu(z) = z sigmoid(z)                 (z NULL: y = o).
 * The forward never forms q_n, k_n: the preparation kernel takes 1/||q|| and
 * 1/||k|| of each raw row (fp32) and applies them to its products, and the
 * walk scales its rows by them, so the unit rows are exact to fp32 rather
 * than rounded to bf16.  The backward forms bf16 copies of q_n, k_n in its
 * workspace, runs the rule's backward on them and maps dq_n, dk_n back to
 * the raw rows.
 * Forward: q, k, v, z bf16 (layouts of gdn_chunk_fwd; z as v); a, b fp32
 * [B, T, Hv]; writes y (bf16), o (bf16, the ungated output the backward needs
 * when z is given; NULL = not kept) and hT (NULL = not written).
 * Backward: the forward's inputs, o (required when z is given), the output
 * cotangent dy and dhT (NULL = 0); writes dq, dk (bf16, raw q and k, summed over
 * the value heads of each key head), dv (bf16), da, db (fp32, the logits), dz
 * (bf16, required when z is given) and dh0 (NULL = not written).
 * ws: at least gdn_layer_workspace_bytes(backward, ...) bytes; its first word
 * is the rule's status word (gdn_workspace_status).  Other conventions as for
 * gdn_chunk_fwd / gdn_chunk_bwd.
 */
size_t gdn_layer_workspace_bytes(int backward, int B, int T, int Hk, int Hv, int d_k, int d_v,
                                 int chunk, int n_segments);
int gdn_layer_fwd(const void* q, const void* k, const void* v, const float* a, const float* b,
                  const void* z, const float* h0, void* y, void* o, float* hT, int B, int T, int Hk,
                  int Hv, int d_k, int d_v, int chunk, int n_segments, void* ws, size_t ws_bytes,
                  void* stream);
int gdn_layer_bwd(const void* q, const void* k, const void* v, const float* a, const float* b,
                  const void* z, const float* h0, const void* o, const void* dy, const float* dhT,
                  void* dq, void* dk, void* dv, float* da, float* db, void* dz, float* dh0, int B,
                  int T, int Hk, int Hv, int d_k, int d_v, int chunk, int n_segments, void* ws,
                  size_t ws_bytes, void* stream);

/*
 * Forward that allocates nothing and takes no workspace.  The pages have no
 * counterpart of this entry point; it exists for callers that may not
 * allocate device memory at call time and cannot lend a scratch buffer:
 * services that plan and lock all their device memory up front (where an
 * allocation could fail, fragment the plan, or stall the device while it
 * synchronises), and plug-ins whose host framework owns every byte of device
 * memory.  It computes exactly what gdn_chunk_fwd computes with
 * n_segments = 1 (same arguments otherwise, same results).
 *
 * Scratch: a fixed array inside the library's device image, sized for
 * GDN_NOALLOC_MAX_UNITS (batch x value head x chunk) units, i.e. the call
 * needs B * Hv * ceil(T / chunk) <= GDN_NOALLOC_MAX_UNITS (24 MiB of scratch);
 * larger problems are refused with GDN_ERR_WORKSPACE before anything is
 * enqueued.  Every GPU that loads the library keeps that array until the
 * process exits.
 * Set-up: a call looks up the array's device address on the current device
 * (cudaGetSymbolAddress) whenever `stream` is not capturing, and caches it per
 * device; a call made while `stream` is being captured uses that cache, so
 * make the first call on each device before any stream capture, and make one
 * again after a device reset (which reloads the library's device image at a
 * new address).
 * Sharing: all calls on a device use the same array, and its contents persist
 * from call to call.  Nothing in it needs to start at zero (each call writes
 * every scratch byte it reads before reading it), but calls whose executions
 * overlap on the GPU (different streams, or several host threads without
 * ordering) race on the array and may return wrong results: order them.
 * Never calls cudaMalloc, cudaFree or any allocating routine.
 * Failure detection: the call's kernels report a bounded wait that gave up in
 * the array's status word, which gdn_noalloc_status reads.
 */
#define GDN_NOALLOC_MAX_UNITS 256
int gdn_chunk_fwd_noalloc(const void* q, const void* k, const void* v, const float* g,
                          const float* beta, const float* h0, void* o, float* hT, int B, int T,
                          int Hk, int Hv, int d_k, int d_v, int chunk, void* stream);

/*
 * Status of the bounded in-kernel waits of the last gdn_chunk_fwd_noalloc
 * call on the current device: synchronises `stream` (pass the stream that
 * call used) and reads the status word of the fixed scratch array.  Returns
 * GDN_OK if no wait gave up, GDN_ERR_TIMEOUT if one did (that call's outputs
 * are then not valid), GDN_ERR_CUDA if the stream or the read failed.  The
 * pages have no counterpart.
 */
int gdn_noalloc_status(void* stream);

/*
 * Timing variants of gdn_chunk_fwd / gdn_chunk_bwd: identical results, plus
 * cudaEventRecord(events[i], stream) right after the library's i-th kernel
 * launch, for i < n_events (NULL entries are skipped).  The events are the
 * caller's (cudaEvent_t handles created by the caller).  Launch order:
 *   forward,  n_segments = 1:  prep, walk
 *   forward,  n_segments > 1:  prep, fold, segment prefix, walk
 *   backward, n_segments = 1:  prep, walks (state recompute beside the reverse
 *                              walk, one launch), gradients
 *   backward, n_segments > 1:  prep, fold, prefix, reverse fold, reverse prefix,
 *                              walks (the two replays, one launch), gradients
 * With T == 0 or B == 0 no kernel is launched and no event is recorded.
 * Pages: none (instrumentation of the same operations).
 */
int gdn_chunk_fwd_timed(const void* q, const void* k, const void* v, const float* g,
                        const float* beta, const float* h0, void* o, float* hT, int B, int T,
                        int Hk, int Hv, int d_k, int d_v, int chunk, int n_segments, void* ws,
                        size_t ws_bytes, void* stream, void* const* events, int n_events);
int gdn_chunk_bwd_timed(const void* q, const void* k, const void* v, const float* g,
                        const float* beta, const float* h0, const void* dO, const float* dhT,
                        void* dq, void* dk, void* dv, float* dg, float* dbeta, float* dh0, int B,
                        int T, int Hk, int Hv, int d_k, int d_v, int chunk, int n_segments,
                        void* ws, size_t ws_bytes, void* stream, void* const* events,
                        int n_events);

/*
 * Inclusive prefix of affine maps along n, per batch row:
 *   (A_out[i], B_out[i]) = (A_i, B_i) o (A_{i-1}, B_{i-1}) o ... o (A_0, B_0)
 * with (A2, B2) o (A1, B1) = (A2 A1, A2 B1 + B2), i.e. A_out[i] h + B_out[i] is
 * h pushed through maps 0..i in order.  This is the prefix the pages take over
 * the gathered per-device pairs (PR "Shard the GatedDeltaNet sequence ...",
 * description; issue "GatedDeltaNet does not support ...", composition law).
 * A, A_out: fp32 [batch, n, d_k, d_k]; B, B_out: fp32 [batch, n, d_k, d_v];
 * row-major.  The exclusive prefix and its application to an initial state
 * are the caller's.  Sizes: d_k = 128, d_v a multiple of 16 up to 128.
 * Out-of-place only (outputs must not overlap inputs).
 */
int gdn_affine_compose(const float* A, const float* B, float* A_out, float* B_out, int batch,
                       int n, int d_k, int d_v, void* stream);

/*
 * Per-segment affine maps of the inter-chunk recurrence (pass 1 of the
 * two-pass scan, returned to the caller).  The N = ceil(T/chunk) chunks of
 * each (b, value head) are split into n_segments segments of whole chunks
 * (segment s holds chunks [floor(sN/S), floor((s+1)N/S))), and each segment's
 * chunk maps h' = A_c h + B_c, A_c = exp(g_last) I - k_g^T w, B_c = k_g^T u, are
 * composed in order: for every segment
 *     A_s = A_{last} ... A_{first},   B_s = the state the segment leaves from h = 0,
 * so the state leaving segment s is A_s h_in + B_s.  A caller that holds a
 * sequence split across devices folds each device's chunks (n_segments = 1),
 * gathers the pairs, takes the exclusive prefix (gdn_affine_compose and one
 * application to h0) and replays with gdn_chunk_fwd from its incoming state.
 * Sources: PR "Shard the GatedDeltaNet sequence under ici_context_parallelism",
 * description (each device folds its chunks into one (A, B), the pairs are
 * gathered and prefix-composed), and the A-output design question in the
 * review thread of PR "Fuse the Gated Delta Net inter-chunk scan into a
 * Pallas TPU kernel" (A as an optional output beside B).
 * A_out: fp32 [B, Hv, n_segments, d_k, d_k] (NULL = not written);
 * B_out: fp32 [B, Hv, n_segments, d_k, d_v] (required).  Row-major.
 * 1 <= n_segments <= max(1, N), else GDN_ERR_ARG.  T = 0 gives (I, 0).
 * ws: at least gdn_fwd_workspace_bytes(B, T, Hk, Hv, d_k, d_v, chunk, 1)
 * bytes, with the status word as for the forward (gdn_workspace_status).
 */
int gdn_segment_fold(const void* k, const void* v, const float* g, const float* beta,
                     float* A_out, float* B_out, int B, int T, int Hk, int Hv, int d_k, int d_v,
                     int chunk, int n_segments, void* ws, size_t ws_bytes, void* stream);

/*
 * Single-token forms: one token per row, the row's state updated in place.
 * Per row r, value head j (key head kh = j / (Hv/Hk)) and state h:
 *   gdn_delta_step   h <- exp(g) (I - beta k k^T) h + beta k v^T,  o = h^T q
 *                    (one token of gdn_chunk_fwd's recurrence);
 *   gdn_decay_step   h <- exp(decay) h + k v^T,                   o = h^T q
 *                    (one token of gdn_decay_fwd's recurrence).
 * q, k [R, Hk, d_k] and v [R, Hv, d_v] bf16; g, beta [R, Hv] fp32; decay [Hv]
 * fp32 (the log-decay of each head); state [n_slots, Hv, d_k, d_v] fp32, read
 * and written; o [R, Hv, d_v] bf16.  Row r works on state slots[r] (int32;
 * NULL: state r).  A slot outside [0, n_slots) marks a row without a state (a
 * padded batch entry): its output is zero and no state is touched.  Two rows
 * with one slot give that state an undefined value.
 * q_stride, k_stride, v_stride: elements from a row to the next (at least
 * H * 128, a multiple of 8), so that q, k and v may be parts of one buffer.
 * No workspace.
 */
int gdn_delta_step(const void* q, const void* k, const void* v, const float* g, const float* beta,
                   float* state, const int* slots, void* o, int R, int n_slots, int Hk, int Hv,
                   int d_k, int d_v, long long q_stride, long long k_stride, long long v_stride,
                   void* stream);
int gdn_decay_step(const void* q, const void* k, const void* v, const float* decay, float* state,
                   const int* slots, void* o, int R, int n_slots, int Hk, int Hv, int d_k, int d_v,
                   long long q_stride, long long k_stride, long long v_stride, void* stream);

/*
 * Linear attention with a decay for each head, over packed sequences.  Per
 * sequence and value head j (key head kh = j / (Hv/Hk)), w = decay[j] <= 0:
 *     h_t = exp(w) h_{t-1} + k_t v_t^T,   o_t = h_t^T q_t,   h_{-1} = h0,   hT = h_{T-1}.
 * (minus infinity: only the newest row is kept).  The decays are constants of the
 * model: no gradient of them is formed.
 * q, k [total, Hk, d_k], v [total, Hv, d_v] bf16 (strides as for the
 * single-token forms); decay [Hv] fp32; h0, hT [n_seqs, Hv, d_k, d_v] fp32
 * (NULL = zero / not written); o [total, Hv, d_v] bf16.  Sequence s holds the
 * rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1 (int32 [n_seqs + 1] on the device,
 * ascending from 0 to total; lengths of zero are allowed); NULL = n_seqs
 * sequences of total / n_seqs rows.  max_seqlen: the longest sequence's length
 * or an upper bound of it; it sizes the split of long sequences over the SMs
 * (a value that is too small costs speed, not correctness).
 * Outputs must not overlap inputs, with one exception: hT may be h0 (and dh0 may
 * be dhT), the states then being replaced.  States that overlap otherwise are refused.
 * Backward: the forward's inputs, the output cotangent dO [total, Hv, d_v]
 * (bf16, contiguous) and dhT (fp32, NULL = zero); writes dq, dk [total, Hk, d_k]
 * (bf16, summed over the value heads of each key head), dv [total, Hv, d_v]
 * (bf16) and dh0 (fp32, NULL = not written).  Nothing is saved by the forward.
 * A sequence's results depend on its own rows alone, whatever the rows beside
 * it hold.  ws: at least gdn_decay_workspace_bytes(backward, ...) bytes, whose
 * first word is the status word of the bounded waits (gdn_workspace_status);
 * where that is all (256 bytes), ws may be NULL, and no status is kept.  A call without
 * rows starts no kernel and leaves that word as it was.
 */
size_t gdn_decay_workspace_bytes(int backward, int n_seqs, int total, int max_seqlen, int Hk,
                                 int Hv, int d_k, int d_v);
int gdn_decay_fwd(const void* q, const void* k, const void* v, const float* decay, const float* h0,
                  const int* cu_seqlens, void* o, float* hT, int n_seqs, int total, int max_seqlen,
                  int Hk, int Hv, int d_k, int d_v, long long q_stride, long long k_stride,
                  long long v_stride, void* ws, size_t ws_bytes, void* stream);
int gdn_decay_bwd(const void* q, const void* k, const void* v, const float* decay, const float* h0,
                  const void* dO, const float* dhT, const int* cu_seqlens, void* dq, void* dk,
                  void* dv, float* dh0, int n_seqs, int total, int max_seqlen, int Hk, int Hv,
                  int d_k, int d_v, long long q_stride, long long k_stride, long long v_stride,
                  void* ws, size_t ws_bytes, void* stream);

/*
 * Causal softmax attention over packed sequences with grouped heads (key head
 * h / (Hq/Hk) for query head h).  In a sequence of n queries and m keys, query i
 * sees the keys j <= i + m - n (the last query sees all of them):
 *     o_i = sum_j p_ij v_j,   p_ij = exp(scale q_i . k_j - lse_i),   lse_i = log sum_j exp(..).
 * n = m is a prompt, n < m a prompt or single tokens continuing m - n cached
 * keys.  A query that sees no key (n > m, or m = 0) has o = 0, lse = -inf and
 * passes no gradient.  One that sees a score of NaN or plus infinity (or one too large
 * for fp32) has o and lse NaN, however the keys are split.
 * Values of v are finite: a row of v that is not may make o NaN of queries that do not
 * see it, too (they count it zero times; lse is right).
 * q, o [total_q, Hq, d], k, v [total_k, Hk, d] bf16, d = 128, Hq a multiple of
 * Hk, at most 128 query heads to a key head (q_stride, k_stride, v_stride as for
 * the single-token forms); lse [total_q, Hq] fp32 (NULL = not written);
 * scale > 0.  cu_q, cu_k: int32 [n_seqs + 1] on the device, ascending from 0 to
 * total_q / total_k (NULL: equal lengths).  k_len: int32 [n_seqs] (NULL: all),
 * the used rows of each sequence's keys, for caches of fixed capacity; rows past
 * it may hold anything.  max_k: the longest sequence's keys or an upper bound; it
 * sizes the split of the keys over the SMs (a value that is too small, or much too
 * large, costs speed, not correctness).  Outputs must not overlap inputs.
 * Backward: the forward's inputs (without k_len), o and lse, and the output
 * cotangent dO [total_q, Hq, d] (bf16, contiguous); writes dq [total_q, Hq, d]
 * and dk, dv [total_k, Hk, d] (bf16, summed over the query heads of each key
 * head).  Sums have a fixed order: equal calls give equal results.
 * ws: at least gdn_attn_workspace_bytes(backward, ...) bytes, whose first word is
 * the status word of the bounded waits (gdn_workspace_status); where that is all
 * (256 bytes), ws may be NULL, and no status is kept.  A call without queries, and a
 * backward without keys, starts no kernel and leaves that word as it was.
 */
size_t gdn_attn_workspace_bytes(int backward, int n_seqs, int total_q, int total_k, int max_k,
                                int Hq, int Hk, int d);
int gdn_attn_fwd(const void* q, const void* k, const void* v, const int* cu_q, const int* cu_k,
                 const int* k_len, void* o, float* lse, int n_seqs, int total_q, int total_k,
                 int max_k, int Hq, int Hk, int d, float scale, long long q_stride,
                 long long k_stride, long long v_stride, void* ws, size_t ws_bytes, void* stream);
int gdn_attn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                 const void* dO, const int* cu_q, const int* cu_k, void* dq, void* dk, void* dv,
                 int n_seqs, int total_q, int total_k, int Hq, int Hk, int d, float scale,
                 long long q_stride, long long k_stride, long long v_stride, void* ws,
                 size_t ws_bytes, void* stream);

/*
 * Norms of query and key heads with the position rotation in the same pass.  Per
 * token t and head x [d] of q (weight q_weight) or k (k_weight):
 *     n = x w / sqrt(mean(x^2) + eps)          (no weight: n = x),
 *     y = n with its pairs j < n_pairs turned by
 *         positions[pair_axis[j]][t] * inv_freq[j]  radians:
 *         (a, b) -> (a cos - b sin, b cos + a sin).
 * Pair j is (n_j, n_{j + n_pairs}), or with interleaved != 0 (n_{2j}, n_{2j + 1});
 * values behind the first 2 n_pairs keep theirs.  n_pairs is a multiple of 8, at most
 * d / 2 (0: no rotation; positions and inv_freq may then be NULL).  positions: int32
 * [n_axes, n] on the device (several axes: time, height, width); inv_freq: fp32
 * [n_pairs] on the device, finite; pair_axis: n_pairs bytes on the HOST, each below
 * n_axes (NULL with one axis).  The angle's fraction of a turn is formed in 64 bits:
 * positions of any size keep it.  q, q_out [n, Hq, d], k, k_out [n, Hk, d] bf16, d =
 * 128, with strides between tokens as for the single-token forms; weights fp32 [d],
 * 16-byte aligned; squares and sums in fp32 (values beyond 1e18 overflow them).
 * q_out may be q, and k_out k, with equal strides; otherwise outputs must not overlap
 * inputs.
 * Backward: dq_out, dk_out are the cotangents of q_out and k_out, dq and dk those of q
 * and k (dq may be dq_out, dk may be dk_out, with equal strides).  q and k are the
 * forward's inputs, not read (and may be NULL) without a weight.  dq_weight, dk_weight:
 * fp32 [d], sums over tokens and heads in a fixed order (NULL: not wanted); they need
 * ws, of gdn_rope_workspace_bytes bytes.  Without them ws may be NULL.  No kernel of
 * these calls waits, and ws has no status word.
 *
 * gdn_rope_append is the forward that writes the keys, and the values v [n, Hk, d] as
 * they are, into a cache of n_pages pages of page_size rows each: token t into row
 * slots[t] % page_size of page slots[t] / page_size (slots: int32 [n] on the device;
 * a slot outside the cache is a padded token's, which is not written; two tokens must
 * not share one).  q_out is written for every token.
 *
 * Pages: k_pages, v_pages hold n_pages x page_size rows of Hk heads, bf16, at element
 * offset  page * strides->page + row * strides->row + head * strides->head, each stride
 * a multiple of 8, at least d; page_size a multiple of 16.
 */
typedef struct {
  long long page, row, head;
} gdn_page_strides;

int gdn_rope_fwd(const void* q, const void* k, const float* q_weight, const float* k_weight,
                 const int* positions, const float* inv_freq, const unsigned char* pair_axis,
                 void* q_out, void* k_out, int n, int Hq, int Hk, int d, int n_axes, int n_pairs,
                 int interleaved, float eps, long long q_stride, long long k_stride,
                 long long qo_stride, long long ko_stride, void* stream);
size_t gdn_rope_workspace_bytes(int n, int Hq, int Hk, int d);
int gdn_rope_bwd(const void* q, const void* k, const float* q_weight, const float* k_weight,
                 const int* positions, const float* inv_freq, const unsigned char* pair_axis,
                 const void* dq_out, const void* dk_out, void* dq, void* dk, float* dq_weight,
                 float* dk_weight, int n, int Hq, int Hk, int d, int n_axes, int n_pairs,
                 int interleaved, float eps, long long q_stride, long long k_stride,
                 long long dqo_stride, long long dko_stride, long long dq_stride,
                 long long dk_stride, void* ws, size_t ws_bytes, void* stream);
int gdn_rope_append(const void* q, const void* k, const void* v, const float* q_weight,
                    const float* k_weight, const int* positions, const float* inv_freq,
                    const unsigned char* pair_axis, void* q_out, void* k_pages, void* v_pages,
                    const int* slots, int n, int n_pages, int page_size, int Hq, int Hk, int d,
                    int n_axes, int n_pairs, int interleaved, float eps, long long q_stride,
                    long long k_stride, long long v_stride, long long qo_stride,
                    const gdn_page_strides* k_strides, const gdn_page_strides* v_strides,
                    void* stream);

/*
 * Softmax attention of new tokens over a paged cache: gdn_attn_fwd whose sequence s has
 * its key and value rows in pages.  Row j lies in page page_table[s][j / page_size] at
 * row j % page_size of k_pages and v_pages (layout: gdn_page_strides above); k_len[s]
 * rows are used, the new tokens' own among them (gdn_rope_append writes them), so that
 * the last query sees all of them, each one before it one fewer.  page_table: int32
 * [n_seqs, max_pages] on the device, table_stride entries between sequences; an entry
 * outside 0 .. n_pages - 1 is an absent page, whose keys nobody sees (a row that sees no
 * other has o = 0, lse = -inf).  k_len is held within max_pages * page_size (at most
 * 2^30).  Rows past k_len may hold anything.  Sequences may share pages.  q [total_q, Hq,
 * d], cu_q, o, lse, scale, max_k, status, scores and values that are not finite as for gdn_attn_fwd; max_q
 * bounds a sequence's new tokens as max_k does its keys (0: not known; up to 128 / (Hq/Hk)
 * it says that a kernel for few rows suits, which takes longer sequences too).  ws: at least
 * gdn_attn_paged_workspace_bytes(n_seqs, total_q, max_pages * page_size, max_q, max_k, Hq, Hk,
 * d) bytes, never NULL where there are queries.
 *
 * gdn_attn_paged_weights adds to each key the attention weight that it receives from the
 * same queries,
 *     weights[page][kh][row] += sum exp(scale q_i . k_j - lse_i)
 * over the queries i that see key j and the query heads of key head kh, with lse
 * [total_q, Hq] as gdn_attn_paged returned it (a row with lse = -inf adds nothing).
 * weights: fp32 [n_pages, Hk, page_size], contiguous.  A sequence's sum is formed in a
 * fixed order and added at once; where sequences share a page, or a table names one twice,
 * each adds its own, in no fixed order.  A row that a new key takes keeps the weight that it
 * had (of a key that was evicted, say): set it to zero where it is to count anew.  max_q and max_k bound a sequence's queries (0: not
 * known) and keys; they steer, as above.  ws: 256 bytes whose first word is the status
 * word, or NULL.  A call that has nothing to add starts no kernel.
 *
 * gdn_cache_evict drops the lightest keys.  Per sequence and key head the last min(recent,
 * budget) keys stay and of the others those with the largest weights, budget in all; of
 * equal weights the lowest index stays, NaN weighs least.  What stays moves in its order
 * into rows 0, 1, .. of the sequence's target pages to_table [n_seqs, to_pages] (int32,
 * to_stride entries between sequences, with to_pages * page_size rows for min(budget,
 * max_pages * page_size) keys): keys, values and weights.  to_table NULL or page_table (with
 * its stride): the sequence's own pages, in place.  Other rows keep what they hold.  new_len [n_seqs] receives
 * the keys that stay of each sequence (the same for all heads); it must not overlap k_len.
 * Keys on absent pages never stay; a row whose target page is absent is not written.  In
 * place, no page may occur twice in the tables; otherwise no target page may, nor may one
 * hold a key of any sequence of the call.  (A copy of page_table as to_table is such a case: rows
 * would be overwritten that others still read.)  ws: gdn_cache_evict_workspace_bytes(n_seqs, max_pages *
 * page_size, budget, Hk) bytes, without a status word (no kernel of it waits).
 */
size_t gdn_attn_paged_workspace_bytes(int n_seqs, int total_q, int max_rows, int max_q, int max_k,
                                      int Hq, int Hk, int d);
int gdn_attn_paged(const void* q, const void* k_pages, const void* v_pages, const int* page_table,
                   const int* k_len, const int* cu_q, void* o, float* lse, int n_seqs, int total_q,
                   int max_q, int max_k, int n_pages, int page_size, int max_pages, int Hq, int Hk,
                   int d, float scale, long long q_stride, const gdn_page_strides* k_strides,
                   const gdn_page_strides* v_strides, long long table_stride, void* ws,
                   size_t ws_bytes, void* stream);
int gdn_attn_paged_weights(const void* q, const void* k_pages, const float* lse,
                           const int* page_table, const int* k_len, const int* cu_q, float* weights,
                           int n_seqs, int total_q, int max_q, int max_k, int n_pages, int page_size,
                           int max_pages, int Hq, int Hk, int d, float scale, long long q_stride,
                           const gdn_page_strides* k_strides, long long table_stride, void* ws,
                           size_t ws_bytes, void* stream);
size_t gdn_cache_evict_workspace_bytes(int n_seqs, int max_rows, int budget, int Hk);
int gdn_cache_evict(void* k_pages, void* v_pages, float* weights, const int* page_table,
                    const int* to_table, const int* k_len, int* new_len, int n_seqs, int n_pages,
                    int page_size, int max_pages, int to_pages, int Hk, int d, int budget,
                    int recent, const gdn_page_strides* k_strides, const gdn_page_strides* v_strides,
                    long long table_stride, long long to_stride, void* ws, size_t ws_bytes,
                    void* stream);

/*
 * Debug export of the per-chunk UT quantities, for tests.  For every
 * (b, value head j, chunk c), in [B, Hv, N, ...] order with N = ceil(T/chunk):
 *   S_out [.., chunk, chunk] fp32  S = tril(diag(beta) (K K^T * decay), -1)
 *   T_out [.., chunk, chunk] fp32  T = (I + S)^-1 (the device's ladder)
 *   w_out [.., chunk, d_k]   bf16  w = T diag(beta exp(G)) K
 *   u_out [.., chunk, d_v]   bf16  u = T diag(beta) V
 * Any output may be NULL.  Rows of a ragged last chunk beyond T are the
 * zero-padding rows.  Uses no workspace.  With chunk = 64 the outputs are
 * the device's 128-row tiles, N = ceil(T/128) per (b, j), each holding two
 * chunks: S_out, T_out [.., 128, 128] block diagonal (chunk 2t in rows and
 * columns 0-63 of tile t, chunk 2t + 1 in 64-127, zeros elsewhere), w_out and
 * u_out [.., 128, d] (chunk 2t in rows 0-63, chunk 2t + 1 in rows 64-127).
 */
int gdn_debug_ut(const void* k, const void* v, const float* g,
                 const float* beta, float* S_out, float* T_out, void* w_out, void* u_out,
                 int B, int T, int Hk, int Hv, int d_k, int d_v, int chunk, void* stream);

/*
 * Status of the bounded in-kernel waits of the last gdn_chunk_fwd,
 * gdn_chunk_bwd call that used workspace `ws`.
 * The pages have no counterpart: it reports the failure detection of these
 * kernels.  Synchronises `stream` (the one exception to "never synchronises")
 * and reads the workspace's status word.  Returns GDN_OK if no wait gave up,
 * GDN_ERR_TIMEOUT if one did (the outputs of that call are then not valid),
 * GDN_ERR_ARG for a null ws, GDN_ERR_CUDA if the stream or the copy failed.
 */
int gdn_workspace_status(const void* ws, void* stream);

/*
 * Self-test of the bounded waits.  The pages have no counterpart.  Enqueues
 * one block whose wait on a barrier that nothing ever signals has to give up
 * after about limit_ns nanoseconds (1e3 <= limit_ns <= 1e10; counted in SM
 * cycles at the device's maximum clock, so longer at lower clocks); the kernel then sets
 * bit 0 of *status and returns normally (bit 1 would mean the wait completed,
 * which cannot happen), leaving the context usable.  status: one device int,
 * cleared by this call.  Synchronises `stream`.  Returns GDN_ERR_TIMEOUT when
 * the timeout was recorded (the expected outcome), GDN_OK if it was not,
 * GDN_ERR_ARG for a null status or a limit out of range, GDN_ERR_CUDA on a
 * CUDA error.
 */
int gdn_selftest_wait_timeout(long long limit_ns, int* status, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */
