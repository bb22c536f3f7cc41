/*
 * moe_gb300.h -- C ABI of the GB300 (sm_103a) MoE routing-layer library.
 *
 * One mixture-of-experts layer under batch-level routing control:
 *
 *   y(x) = sum_{j in Top-k(G(x))} G(x)_j * E_j(x)
 *       ("MACS: Modality-Aware Capacity Scaling for Efficient Multimodal MoE
 *        Inference", sec. 3.1, Eq. (1))
 *
 * computed as   moe_route        router GEMM + fp32 softmax + top-R ranking,
 *                                optionally fused with the SERE batch reroute
 *               moe_reroute_sere the SERE reroute on its own
 *               moe_route_dispatch
 *                                decode batches: moe_route (optionally with
 *                                SERE) and the uncapped dispatch in one launch
 *               moe_dispatch_capacity
 *                                expert-sorted permutation, optionally under a
 *                                weighted capacity with overflow reroute / drop
 *               moe_ffn_grouped  grouped SwiGLU expert FFN, combine fused in
 *               moe_combine      weighted combine of per-row expert outputs
 *               moe_token_weights
 *                                entropy-weighted token load for the capacity
 *                                dispatch, and the effective visual ratio
 *               moe_similarity_calibrate
 *                                the SERE similarity matrix from the experts'
 *                                outputs on calibration tokens
 *
 * and, beside that layer, the attention half of a decoder layer for serving:
 *
 *               moe_qk_norm_rope per-head norms of q and k, rotary positions
 *                                (one or several axes) and the append of k and
 *                                v to a paged cache held in 4 bits
 *               moe_attention_kv4  attention over that cache, for single
 *                                tokens, drafts and prompt chunks
 *               moe_kv4_read     cached tokens back as values
 *               moe_kv4_reserve, moe_kv4_assign, moe_kv4_compact
 *                                the cache's pages: growing, copying on write,
 *                                forking, reordering, freeing and packing
 *               moe_kv4_weigh, moe_kv4_evict
 *                                the attention weight that cached tokens draw,
 *                                and eviction of those that drew least
 *               moe_linear_w4, moe_w4_pack
 *                                products with weights in 4 bits (projections,
 *                                heads), and their rounding
 *               moe_verify_drafts
 *                                how many drafted tokens the target's logits
 *                                accept, and the token that follows
 *
 * Conventions for every entry point
 *  - Pointers named "host" are host memory; every other pointer is device
 *    memory (cudaMalloc / PyTorch CUDA tensors).  The caller owns all memory;
 *    the library allocates nothing, frees nothing and never synchronises.
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Calls are asynchronous on that stream; launch configurations
 *    depend only on the scalar arguments, so a sequence of calls can be
 *    captured into a CUDA graph.
 *  - Arguments are checked on the host before anything is launched.  A bad
 *    argument returns a negative moe_status_t and launches nothing.
 *  - Errors that depend on the data (non-finite logits, an out-of-range id,
 *    an internal wait that timed out) are written asynchronously into the
 *    optional device-side status word `st` (first error wins; clear it to
 *    zero before use).  Outputs of a call that set an error are unspecified.
 *  - Matrices are row-major and densely packed unless a leading dimension
 *    (`ld`) is given.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int moe_status_t;
#define MOE_OK 0
#define MOE_ERR_INVALID_ARG (-1)   /* a pointer, size, alignment or option is invalid */
#define MOE_ERR_UNSUPPORTED (-2)   /* valid but outside what the kernels support (see limits) */
#define MOE_ERR_CUDA (-3)          /* a CUDA launch or driver call failed */
#define MOE_ERR_WORKSPACE (-4)     /* workspace missing or smaller than moe_workspace_size() */

/* Device-side status word, written by kernels. */
typedef struct moe_dev_status {
    int32_t code;    /* MOE_DEV_* */
    int32_t detail;  /* code-specific: token index, expert id, or wait site */
} moe_dev_status;
#define MOE_DEV_OK 0
#define MOE_DEV_NONFINITE 1        /* a router logit, k or v was NaN or infinite (detail = token) */
#define MOE_DEV_TIMEOUT 2          /* a bounded on-chip wait gave up (detail = wait site) */
#define MOE_DEV_BAD_INDEX 3        /* an expert id, row, position or page was out of range (detail = value) */
#define MOE_DEV_NO_PAGES 4         /* the pool has too few free pages (detail = pages missing) */

#define MOE_DTYPE_F32 0
#define MOE_DTYPE_BF16 1

/* Compile-time limits of the library. */
#define MOE_MAX_EXPERTS 256        /* N */
#define MOE_MAX_RANKS 16           /* R (and k <= R) */

/* ---------------------------------------------------------------- */
/* moe_route                                                          */
/* ---------------------------------------------------------------- */
#define MOE_ROUTE_FROM_LOGITS 1u   /* `logits` is an input; x and w_router are not read */
#define MOE_ROUTE_RENORM_TOPK 2u   /* divide the first k gates by their fp32 sum */

/* SERE parameters ("SERE" expert rerouting, Xiaohongshu multi-image QA
 * inference article, sec. 4.1-4.2). */
typedef struct moe_sere_params {
    int k_primary;            /* K': ranks [0, K') are primaries, 1 <= K' <= k */
    float rho;                /* a secondary moves only if sim > rho (strict) */
    const float* sim;         /* [N][N] fp32 expert similarity, row = source expert */
    const uint8_t* protect;   /* [N] 0/1, nonzero = this source never moves; NULL = none */
    uint32_t* union_bitmap;   /* out [ceil(N/32)]: bit p set iff expert p is in the
                                 primary union P; may be NULL */
    int32_t* stats;           /* out [8]: union before, |P|, union after, moved, merged,
                                 kept-protected, kept-dissimilar, 0; may be NULL */
} moe_sere_params;

/*
 * Router scores, softmax gate and ranking.  "MACS" sec. 3.1, Eq. (1): the
 * router G(x) scores all N experts; the layer keeps the top-k and weights
 * each by its gate.
 *
 *   x          [T][H]  token activations, x_dtype BF16 or F32 (16-byte aligned)
 *   w_router   [N][H]  fp32 router weight
 *   logits     [T][N]  fp32; written (router GEMM, fp32 accumulation), or read
 *                      with MOE_ROUTE_FROM_LOGITS
 *   ids        [T][R]  int32 out: expert ids by logit descending, ties to the lower id
 *   gates      [T][R]  fp32 out: softmax gate of each ranked expert (over all N),
 *                      computed in a fixed fp32 order so that results are
 *                      reproducible bit for bit
 *   k                  the number of experts a token uses (k <= R); used by
 *                      MOE_ROUTE_RENORM_TOPK and by SERE
 *   sere               NULL, or SERE parameters: then R must equal k and the
 *                      reroute runs inside the same kernel as the ranking
 *                      (one CTA, T <= 4096), rewriting ids/gates in place:
 *                      moved slots take the target id, merged slots become
 *                      (-1, 0.0f) with the gate added to the slot that holds
 *                      the target.
 * Limits: 1 <= N <= 256, 1 <= k <= R <= min(16, N), T >= 0, H >= 1
 * (H % 8 == 0 for BF16 x, H % 4 == 0 for F32 x).
 */
moe_status_t moe_route(const void* x, int x_dtype, const float* w_router, int T, int H, int N, int R,
                       int k, uint32_t flags, float* logits, int32_t* ids, float* gates,
                       const moe_sere_params* sere, moe_dev_status* st, void* stream);

/*
 * Decode routing and dispatch in one launch: the results of moe_route with
 * R = k (and `sere`, if given) followed by the uncapped
 * moe_dispatch_capacity, bit for bit, for batches of up to 256 tokens.
 * "SERE" article sec. 4.2: the reroute feeds the fused MoE with no host round
 * trip; at decode sizes the ranking, reroute and permutation touch a few KB,
 * so they run in the last CTA of the router launch instead of in launches of
 * their own.
 *
 *   x, x_dtype, w_router, T, H, N, k, logits, ids, gates, sere
 *              as for moe_route with R = k (logits is a required output;
 *              flags: MOE_ROUTE_RENORM_TOPK only)
 *   counts, offsets, row_token, row_gate, active
 *              as for moe_dispatch_capacity with capacity_factor <= 0 and
 *              ld = k: rows ordered by (expert, token)
 *   workspace  moe_workspace_size(MOE_OP_ROUTE_DISPATCH, ...) bytes, 256-byte
 *              aligned, ZERO-FILLED before its first use (it holds a counter
 *              that every call leaves at zero); two calls must not use one
 *              workspace concurrently
 * Limits: 0 <= T <= 256, T * k <= 2048, 1 <= k <= min(16, N), N <= 256;
 * H % 8 == 0 for BF16 x, H % 4 == 0 for F32 x.
 */
moe_status_t moe_route_dispatch(const void* x, int x_dtype, const float* w_router, int T, int H, int N, int k,
                                uint32_t flags, float* logits, int32_t* ids, float* gates,
                                const moe_sere_params* sere, int32_t* counts, int32_t* offsets,
                                int32_t* row_token, float* row_gate, int32_t* active, void* workspace,
                                size_t ws_bytes, moe_dev_status* st, void* stream);

/*
 * One decode MoE layer in one call: moe_route_dispatch, then the grouped
 * SwiGLU FFN with the weighted combine fused in (y = sum_j G(x)_j E_j(x),
 * "MACS" sec. 3.1 Eq. (1); with `sere`, the "SERE" article's batch reroute,
 * sec. 4.1-4.2).  As soon as ranking ends, while the routing launch still
 * reroutes and permutes, the FFN starts streaming the weights of a published
 * set of experts: without SERE the union of the ranked experts; with SERE
 * its primary union P (sec. 4.1: primaries are never rerouted), or the whole
 * union before the reroute when that union's phase-1 units fit one wave of
 * the SMs, or two waves while P's would fill at most a third of one and the
 * other experts' more than one (an expert that then moves costs only its
 * phase 1).  The other experts and the down projections wait for the final
 * routing.  Results equal moe_route_dispatch followed by moe_ffn_grouped
 * with MOE_FFN_FUSE_COMBINE (up to the fp32 summation order of y).
 *
 *   x, w_router, sere, logits, ids, gates, counts, offsets, row_token,
 *   row_gate, active: as moe_route_dispatch (x is BF16, [T][H])
 *   w_gate, w_up [N][I][H], w_down [N][H][I]  bf16 expert weights
 *   y          [T][H] fp32 out: zeroed first when ffn_flags has
 *              MOE_FFN_ZERO_Y, else the layer output is added into it
 *   route_flags  MOE_ROUTE_RENORM_TOPK or 0
 *   ffn_flags    MOE_FFN_ZERO_Y or 0 (the combine is always fused)
 *   route_ws   moe_workspace_size(MOE_OP_ROUTE_DISPATCH, ...) bytes
 *   ffn_ws     moe_workspace_size(MOE_OP_FFN, T, H, I, N, k, k, 0, BF16) bytes
 *              both 256-byte aligned and ZERO-FILLED before their first use
 *              (every call leaves their counters at zero); a pair of
 *              workspaces serves one call at a time.
 * Limits: 1 <= T <= 64, T * k <= 2048, N <= 256, 1 <= k <= min(16, N),
 * H % 128 == 0, I % 128 == 0, pointers 16-byte aligned.  Errors: argument
 * errors return before anything is launched; data-dependent errors and
 * bounded waits that ran out go to st.
 */
moe_status_t moe_decode_layer(const void* x, const float* w_router, const void* w_gate, const void* w_up,
                              const void* w_down, int T, int H, int I, int N, int k, uint32_t route_flags,
                              uint32_t ffn_flags, const moe_sere_params* sere, float* logits, int32_t* ids,
                              float* gates, int32_t* counts, int32_t* offsets, int32_t* row_token,
                              float* row_gate, int32_t* active, float* y, void* route_ws, size_t route_ws_bytes,
                              void* ffn_ws, size_t ffn_ws_bytes, moe_dev_status* st, void* stream);

/*
 * SERE batch reroute on given routing ("SERE" article, sec. 4.1: the union P
 * of every token's top-K' primary experts is the shared candidate set; every
 * secondary outside P whose source is not protected (sec. 4.2) moves to its
 * most similar member of P when that similarity exceeds rho; ties to the
 * lower id; a token that already holds the target gets the gate added).
 *
 *   ids, gates [T][ld] in/out (the first k columns are used); same rewrite
 *   rules as moe_route with `sere`.  One CTA; T <= 4096.
 */
moe_status_t moe_reroute_sere(int32_t* ids, float* gates, int ld, int T, int N, int k,
                              const moe_sere_params* sere, moe_dev_status* st, void* stream);

/* ---------------------------------------------------------------- */
/* moe_dispatch_capacity                                              */
/* ---------------------------------------------------------------- */
#define MOE_SLOT_KEPT 0
#define MOE_SLOT_REROUTED 1
#define MOE_SLOT_DROPPED 2

/*
 * Expert-sorted permutation, optionally under a weighted capacity.
 *
 * Uncapped (capacity_factor <= 0): every slot with id >= 0 among the first k
 * columns of ids becomes one row.  Capped ("MACS" sec. 3.1 Eq. (3) and
 * sec. 3.2 Eq. (6)): token weights w are taken in fixed point
 * w_q = rint(w * 2^24); S = sum w_q; C = floor(((double)S * k) *
 * capacity_factor / N).  Each expert admits its (token, slot) pairs in
 * (gate desc, token asc) order while the cumulative w_q stays <= C.  Then, in
 * rounds i = 0 .. R-k-1, every token with an overflowed slot offers its
 * lowest-rank overflowed slot (with that slot's gate) to its rank-(k+i)
 * expert, which admits offers in the same order while load + cumulative
 * w_q <= C.  Slots left over are dropped (the "MACS" Fig. 1 overflow path:
 * reroute locally, else drop).
 *
 *   ids, gates   [T][ld]  ranked routing (ld >= R when capped, >= k otherwise)
 *   token_w      [T] fp32 >= 0, or NULL (all 1); capped mode only (e.g. the
 *                      entropy weights of moe_token_weights)
 *   modality_bias [N] int8, or NULL: per-expert capacity ("MACS" sec. 3.3:
 *                      m_j = +1 visual, -1 text, 0 shared expert).  The page
 *                      stops before its scaling formula; this library reads it
 *                      as C_j = floor(c * (1 + m_j * (R_v - 1/2))) with
 *                      c = ((double)S * k) * capacity_factor / N unfloored, so
 *                      m_j = 0 or R_v = 1/2 keep the static C.  Capped mode only.
 *   r_v          [1] fp32 device scalar in [0, 1] (the effective visual ratio of
 *                      moe_token_weights); required with modality_bias.  A bias
 *                      outside {-1, 0, 1} or a ratio outside [0, 1] is reported
 *                      in st and that expert keeps the static C.
 *   counts       [N]      out: rows per expert
 *   offsets      [N+1]    out: exclusive prefix of counts
 *   row_token    [T*k]    out: token of each row, rows ordered by (expert, token)
 *   row_gate     [T*k]    out: gate of each row
 *   active       [N+1]    out: active[0] = experts with rows, active[1..] their ids ascending
 *   out_ids, out_gates [T][k] out (may be NULL): final expert and gate per slot,
 *                      (-1, 0.0f) for empty or dropped slots
 *   slot_row     [T][k]   out (may be NULL): row index of each slot, -1 if none
 *   slot_status  [T][k]   out (may be NULL): MOE_SLOT_*; capped mode only
 *   load_q       [N]      out (may be NULL): final weighted load in 2^-24 units
 *   cap_q        [1]      out (may be NULL): the static C in 2^-24 units
 *   workspace    device scratch of moe_workspace_size(MOE_OP_DISPATCH, ...) bytes
 * Limits: N <= 256, k <= R <= min(16, N); capped mode T <= 16384.
 */
moe_status_t moe_dispatch_capacity(const int32_t* ids, const float* gates, int ld, int T, int N, int k,
                                   int R, const float* token_w, float capacity_factor,
                                   const int8_t* modality_bias, const float* r_v, int32_t* counts,
                                   int32_t* offsets, int32_t* row_token, float* row_gate, int32_t* active,
                                   int32_t* out_ids, float* out_gates, int32_t* slot_row,
                                   uint8_t* slot_status, int64_t* load_q, int64_t* cap_q, void* workspace,
                                   size_t ws_bytes, moe_dev_status* st, void* stream);

/*
 * moe_dispatch_capacity_static -- the same dispatch as moe_dispatch_capacity,
 * for callers that cannot allocate device memory.  The paper has no
 * counterpart; this is an interface of this library only.
 *
 * Who needs it: code that is not allowed to call cudaMalloc or to hold a
 * workspace of its own, for example a plugin inside a serving engine that
 * hands out all device memory from its own pool, or code running while a
 * stream is captured into a CUDA graph under a capture mode that forbids
 * allocation calls.  Such a caller still passes its inputs and outputs; only
 * the scratch memory moves into the library.
 *
 * Scratch: one file-scope device array of MOE_STATIC_DISPATCH_SCRATCH_BYTES
 * (4.5 MiB), present on every GPU that loads the library until the process
 * exits.  It is enough for every size with T <= MOE_STATIC_DISPATCH_MAX_T
 * (2048 tokens) and the limits of moe_dispatch_capacity; larger T returns
 * MOE_ERR_UNSUPPORTED and launches nothing.  No call allocates or frees.
 * The first call on a device looks up the array's device address (with that
 * device current) and caches it; make that first call before any stream
 * capture.  Every call on a device shares the one array: calls whose work
 * overlaps on the GPU (two streams, or two host threads) race and give wrong
 * results, so serialise them.  Each call clears the parts of the array that
 * must start at zero, so leftovers of the previous call do no harm.
 *
 * Arguments, outputs and errors are those of moe_dispatch_capacity without
 * `workspace` and `ws_bytes`.
 */
#define MOE_STATIC_DISPATCH_MAX_T 2048
#define MOE_STATIC_DISPATCH_SCRATCH_BYTES (4608u * 1024u)
moe_status_t moe_dispatch_capacity_static(const int32_t* ids, const float* gates, int ld, int T, int N, int k,
                                          int R, const float* token_w, float capacity_factor,
                                          const int8_t* modality_bias, const float* r_v, int32_t* counts,
                                          int32_t* offsets, int32_t* row_token, float* row_gate,
                                          int32_t* active, int32_t* out_ids, float* out_gates,
                                          int32_t* slot_row, uint8_t* slot_status, int64_t* load_q,
                                          int64_t* cap_q, moe_dev_status* st, void* stream);

/* ---------------------------------------------------------------- */
/* moe_ffn_grouped                                                    */
/* ---------------------------------------------------------------- */
#define MOE_FFN_FUSE_COMBINE 1u    /* out is y[T][H] fp32: y[t] += gate * E_e(x_t) per row */
#define MOE_FFN_ZERO_Y 2u          /* with FUSE_COMBINE: zero y first */

/*
 * Grouped SwiGLU expert FFN ("MACS" sec. 3.1 Eq. (1), E_j(x) =
 * W_down_j (silu(W_gate_j x) * (W_up_j x))) over the rows of
 * moe_dispatch_capacity, only for active experts.
 *
 *   x       [T][H]     activations, dtype BF16 or F32 (same dtype as the weights)
 *   w_gate  [N][I][H], w_up [N][I][H], w_down [N][H][I]  expert weights
 *   offsets [N+1], row_token [T*k], row_gate [T*k], active [N+1]  from dispatch
 *   out     FUSE_COMBINE: y [T][H] fp32 (accumulated into); otherwise
 *           rows_out [T*k][H] fp32, row r = E_e(x_token(r)) without the gate
 *   workspace  device scratch of moe_workspace_size(MOE_OP_FFN, ...) bytes,
 *           256-byte aligned.  BF16 needs it: a work counter, one counter
 *           per (expert, token chunk), three more counters and the bf16
 *           SwiGLU activations of every row (T*k*I*2 bytes plus a few KiB);
 *           F32 needs none.  ZERO-FILL it once before its first use: the
 *           counters must start at zero, and every call (including one that
 *           reports an error in st) leaves them at zero again, so nothing
 *           needs clearing between calls.  Two calls in flight at once must
 *           not share a workspace.
 *   flags   MOE_FFN_ZERO_Y: y is zeroed inside the same launch (in chunks,
 *           all of them before any row is added into it).
 * BF16 runs on the tensor cores (tcgen05, TMA-fed) with fp32 accumulation;
 * the SwiGLU activation is rounded to bf16 before the down projection.
 * F32 runs a CUDA-core kernel in fp32.
 * Limits BF16: H % 128 == 0, I % 128 == 0, all pointers 16-byte aligned;
 * rows_out mode needs FUSE_COMBINE off and is accumulated, so zero it first.
 * Limits F32: (H + I) * 4 <= 227 KiB (a row's x and activations are held
 * in shared memory); larger sizes return MOE_ERR_UNSUPPORTED.
 */
moe_status_t moe_ffn_grouped(const void* x, int dtype, const void* w_gate, const void* w_up,
                             const void* w_down, int T, int H, int I, int N, int k, const int32_t* offsets,
                             const int32_t* row_token, const float* row_gate, const int32_t* active,
                             uint32_t flags, float* out, void* workspace, size_t ws_bytes,
                             moe_dev_status* st, void* stream);

/*
 * Expert similarity from calibration tokens (SERE article sec. 4.2: the
 * similarity matrix is prepared offline as the Frobenius similarity of the
 * experts' outputs on calibration data):
 *
 *   sim[i][j] = <E_i(X), E_j(X)>_F / (||E_i(X)||_F ||E_j(X)||_F)
 *
 * with E_e(X) the [n][H] SwiGLU outputs of expert e on the calibration
 * tokens X.  The diagonal is 1; a pair with an expert whose output is all
 * zero gets 0.  Every expert's output on every token comes from the grouped
 * tcgen05 FFN; they are rounded to bf16 and the Gram matrix E E^T runs on the
 * tensor cores split over the SMs, summed and normalised in double.  The
 * result feeds moe_sere_params.sim (the matrix is exactly symmetric).
 *
 *   x          [n][H] bf16 calibration tokens
 *   w_gate, w_up, w_down   bf16 expert weights as in moe_ffn_grouped
 *   sim        [N][N] fp32 out
 *   workspace  moe_workspace_size(MOE_OP_CALIBRATE, n, H, I, N, 1, 1, 0,
 *              MOE_DTYPE_BF16) bytes, 256-byte aligned
 * Limits: 2 <= N <= 128, H % 128 == 0, I % 128 == 0, n * N and n * H below 2^31.
 */
moe_status_t moe_similarity_calibrate(const void* x, int n, const void* w_gate, const void* w_up,
                                      const void* w_down, int H, int I, int N, float* sim, void* workspace,
                                      size_t ws_bytes, moe_dev_status* st, void* stream);

/*
 * Entropy-weighted token load ("MACS" sec. 3.2 Eqs. (4)-(5) and sec. 3.3
 * Eq. (7)): the per-token load weights that moe_dispatch_capacity takes as
 * token_w, and the batch's effective visual ratio.
 *
 *   x          [T][H] token features z (the layer's input rows), BF16 or F32,
 *              16-byte aligned, H % 8 == 0
 *   is_visual  [T] uint8, nonzero = visual token, 0 = text token
 *   delta      sensitivity of the entropy-to-weight map (finite)
 *   eps        added to the standard deviation (> 0)
 *   entropy    [T] fp32 out: Shannon entropy (natural log) of Softmax(z), every token
 *   token_w    [T] fp32 out: sigmoid(-delta * (H - mu) / (sigma + eps)) for
 *              visual tokens, where mu and sigma are the mean and population
 *              standard deviation of the visual tokens' entropies in this
 *              batch; 1 for text tokens
 *   r_v        [1] fp32 out (may be NULL): sum of visual weights / sum of all
 *              weights (0 when T == 0)
 *   workspace  moe_workspace_size(MOE_OP_TOKEN_WEIGHTS, T, ...) bytes (24 bytes
 *              per 8 tokens + 16 per 256 tokens + 16), 256-byte aligned; no
 *              initial contents needed
 * Entropies and weights are computed in fp32 (one warp per token for the
 * entropy, exponentials in base 2); the statistics (count, sum and sum of
 * squares of the visual entropies) and the two weight sums of R_v are added
 * up as 64-bit fixed-point integers (entropy in 2^-32, its square in 2^-24,
 * weights in 2^-32 units), so results do not depend on summation order and
 * are reproducible bit for bit; the population variance is formed from them
 * exactly in 128-bit integers, then mean, standard deviation and R_v in
 * fp32.  T is at most 2^24 (MOE_ERR_UNSUPPORTED beyond), which keeps those
 * sums in range.  Two calls must not share a workspace concurrently (it
 * holds a completion counter).
 * A token whose entropy comes out non-finite sets MOE_DEV_NONFINITE (detail =
 * token) in st: any non-finite feature does so, and so can a row with
 * features of magnitude 2^126 or more (its base-2 exponents overflow fp32).
 */
moe_status_t moe_token_weights(const void* x, int x_dtype, int T, int H, const uint8_t* is_visual, float delta,
                               float eps, float* entropy, float* token_w, float* r_v, void* workspace,
                               size_t ws_bytes, moe_dev_status* st, void* stream);

/*
 * Weighted combine ("MACS" Eq. (1)): y[t] = sum_r gate[t][r] * rows_out[slot_row[t][r]]
 * over the slots r < k with slot_row >= 0, in slot order (deterministic).
 *   rows_out [M][H] fp32, slot_row [T][k], slot_gate [T][k], y [T][H] fp32 out.
 */
moe_status_t moe_combine(const float* rows_out, const int32_t* slot_row, const float* slot_gate, int T,
                         int H, int k, float* y, void* stream);

/*
 * Residual rounding between stacked layers: y[i] = bf16(x[i]), round to
 * nearest, ties to even, for i < n.  In a stack of layers the FFN adds
 * sum_j G_j E_j(x) ("MACS" Eq. (1)) into the fp32 residual (moe_ffn_grouped
 * with MOE_FFN_FUSE_COMBINE and without MOE_FFN_ZERO_Y), and the next
 * layer's routing and FFN read bf16 tokens; this is that rounding, as a
 * launch that overlaps its neighbours (programmatic dependent launch).
 *   x [n] fp32 in, y [n] bf16 out (device, 16-byte aligned, caller-owned);
 *   n a multiple of 8.  Bad sizes or alignment return MOE_ERR_INVALID_ARG
 *   with no launch; n = 0 is a no-op.
 */
moe_status_t moe_residual_to_bf16(const float* x, void* y, long long n, void* stream);

/* ---------------------------------------------------------------- */
/* The cache in 4 bits                                                */
/* ---------------------------------------------------------------- */
#define MOE_KV4_PAGE 64            /* tokens of a page */
#define MOE_KV4_BLOCK 16           /* neighbouring numbers of a head that share a scale */

/*
 * One layer's cache of keys and values in 4 bits, in pages of 64 tokens.
 *
 * A block of 16 neighbouring numbers y of a head is held as
 *     z = y * (1/hs)          hs = k_scale[head] or v_scale[head], 1 if NULL
 *     s = e4m3(max|z| * (1/6))   8 bits, nearest, at most 448
 *     c = e2m1(z * (1/s))        4 bits each, nearest, at most 6 (0 if s is 0)
 * and stands for c * s * hs.  Each operation is one fp32 operation, rounded
 * to nearest; 1/6 is the fp32 nearest to it.  c * s has at most 6 significant
 * bits, so it is exact in fp16 and bf16.  4.5 bits a number in all.
 *
 * pages   [n_pages][n_kv][64 * (D + D/8)] bytes, 16-byte aligned; a head's
 *         part of a page holds, in this order (D = head_dim; i, e = number of
 *         the head; tok = token of the page, g = tok % 8, j = tok / 2):
 *           key codes    [64][D/2]: byte tok*(D/2) + i/2, even i in the low half
 *           key scales   block b = t*(D/64) + r (t < 4):
 *                        byte ((t*8 + g)*8 + tok/8)*(D/64) + r
 *           value codes  e = g'*(D/8) + u (g' < 8): byte
 *                        (((j/4)*8 + g')*4 + j%4)*(D/8) + u, even tok in the low half
 *           value scales block b: byte ((b*4 + j%4)*8 + j/4)*2 + tok%2
 *         (each lane of a warp then finds what its tensor-core fragments need
 *         in 16-byte runs, and a head's part of a page is one bulk copy).
 * page_table [S][max_pages] page of every 64 tokens of a sequence, -1 = none
 * seq_len    [S] tokens of each sequence
 * Bytes of a page that no token has been written to may hold anything.
 */
typedef struct moe_kv4_cache {
    void* pages;
    const int32_t* page_table;
    const int32_t* seq_len;
    const float* k_scale;   /* [n_kv] > 0, or NULL */
    const float* v_scale;   /* [n_kv] > 0, or NULL */
    int32_t n_pages;
    int32_t max_pages;      /* columns of page_table */
    int32_t S;
    int32_t n_kv;
    int32_t head_dim;       /* D: 64 or 128 */
} moe_kv4_cache;

/* Bytes of one page of one layer (all heads); 0 for unsupported sizes. */
size_t moe_kv4_page_bytes(int n_kv, int head_dim);

/*
 * Rotary positions.  Pair i of a head (a, b) becomes
 *     (a cos - b sin, b cos + a sin),  (cos, sin) = table[p][i],
 * where p = positions[axis[i]][token].  Pairs are (i, i + rot/2), or
 * (2i, 2i + 1) with `pairs`; numbers from rot on pass through.  The table
 * brings any frequency scaling, and far positions keep the precision that
 * its maker gave them.
 */
typedef struct moe_rope_params {
    const float* table;        /* [n_pos][rot/2][2] (cos, sin), 16-byte aligned */
    const int32_t* positions;  /* [axes][T], or NULL: the token's place in its sequence (needs a cache) */
    const uint8_t* axis;       /* [rot/2] axis of each pair (e.g. time, height, width), 8-byte aligned, or NULL: axis 0 */
    int32_t n_pos;
    int32_t rot;               /* rotated numbers: a multiple of 32, at most head_dim */
    int32_t axes;              /* rows of positions */
    int32_t pairs;             /* nonzero: neighbours form the pairs */
} moe_rope_params;

/*
 * Norms of q and k for each head, rotary positions, and the append to the
 * cache, in one launch.
 *
 *   qkv      [T][ld] rows of n_q query heads, n_kv key heads and n_kv value
 *            heads of D numbers, BF16 or F32 (16-byte aligned, ld * size a
 *            multiple of 16)
 *   q_weight, k_weight  [D] fp32: y = x * (1/sqrt(mean(x^2) + eps)) * weight for
 *            each head; NULL = that side is not normed
 *   rope     NULL = no rotation
 *   q_out    [T][ld_q], n_q heads, same dtype as qkv; may be qkv itself (with
 *            ld_q = ld)
 *   k_out    [T][ld_k], n_kv heads, or NULL; may be qkv's key part
 *   cache, q_start  NULL, or the cache that k and v are appended to: rows
 *            q_start[s] .. q_start[s+1]-1 (q_start [S+1], ascending) are the
 *            last tokens of sequence s, whose seq_len already counts them and
 *            whose pages are there (moe_kv4_reserve).  A row whose place would
 *            be negative (a sequence of length 0 in a padded batch) is not
 *            appended.  The key is quantised from its fp32 value after the
 *            rotation, the value from its input.
 * Arithmetic is fp32, rounded once to the outputs' type; the sum of a key's
 * squares is carried in two fp32 words, so that a key's code does not depend
 * on the order of the sum.  A NaN or infinite k or v is stored as zero and
 * reported (MOE_DEV_NONFINITE, detail = row).  A token with a position outside
 * the table is reported (MOE_DEV_BAD_INDEX, detail = the position, -1 for an
 * axis that has none) and nothing of it is written, neither outputs nor cache;
 * a page outside the pool is reported (detail = page) and not written.
 * Limits: D is 64 or 128; n_q >= 0, n_kv >= 1, n_q + 2 n_kv <= 1024.
 */
moe_status_t moe_qk_norm_rope(const void* qkv, int dtype, long long ld, int T, int n_q, int n_kv, int head_dim,
                              const float* q_weight, const float* k_weight, float eps,
                              const moe_rope_params* rope, void* q_out, long long ld_q, void* k_out,
                              long long ld_k, const moe_kv4_cache* cache, const int32_t* q_start,
                              moe_dev_status* st, void* stream);

/*
 * The cached tokens q_start[s] .. q_start[s+1]-1 of moe_qk_norm_rope's rows
 * (a sequence's last tokens) as values c * s * hs, rounded to bf16.
 *   k_out, v_out  [T][n_kv][D] bf16; either may be NULL.  Rows without a
 *                 place in the cache are zero.
 */
moe_status_t moe_kv4_read(const moe_kv4_cache* cache, const int32_t* q_start, int T, void* k_out, void* v_out,
                          moe_dev_status* st, void* stream);

/*
 * Attention over the cache: for row q_start[s] + i of sequence s, at place
 * p = seq_len[s] - (q_start[s+1] - q_start[s]) + i, and head h (key head
 * h / (n_q / n_kv)),
 *     out = sum_j softmax_j(scale * q . k_j) v_j   over p - window < j <= p
 * (window 0: all j <= p).  A row that sees nothing (p < 0) gives zeros.
 *
 *   q        [T][ld_q] bf16, n_q heads of D (16-byte aligned, ld_q % 8 == 0)
 *   max_new  an upper bound of the rows of a sequence; it only chooses the
 *            kernels
 *   out      [T][ld_out] bf16, n_q heads of D
 *   lse      [T][n_q] fp32 out: log of the sum of exp(scale * q . k_j), -inf for
 *            a row that sees nothing; may be NULL
 *   workspace  moe_attention_kv4_workspace() bytes, 256-byte aligned, ZERO-FILLED
 *            before its first use (every call leaves its counters at zero, at
 *            places that no size changes: one buffer serves calls of any
 *            sizes in turn); serves one call at a time.  2.7 MB for D = 128 while
 *            T * (n_q / n_kv) <= 256, else 45 MB
 * The products run on the tensor cores in fp16 (q scaled by a power of two of
 * its row, the cached numbers exact) with fp32 sums; softmax in fp32, its
 * probabilities rounded to fp16 before the second product.  Results are
 * reproducible bit for bit.  A page outside the pool, a length beyond the
 * table or a bad q_start is reported (MOE_DEV_BAD_INDEX) and nothing is read
 * through it; that sequence's rows of out and lse are then unspecified.
 * After MOE_DEV_TIMEOUT the workspace has to be zero-filled again.
 * Rows of no sequence are not written.
 * Limits: D is 64 or 128; n_q <= 1024, a multiple of n_kv; S <= 16384; window + T below
 * 2^31 where a table is longer than the window.
 */
moe_status_t moe_attention_kv4(const void* q, long long ld_q, int T, int n_q, const moe_kv4_cache* cache,
                               const int32_t* q_start, int max_new, float scale, int window, void* out,
                               long long ld_out, float* lse, void* workspace, size_t ws_bytes,
                               moe_dev_status* st, void* stream);
size_t moe_attention_kv4_workspace(int T, int n_q, int n_kv, int head_dim);

/*
 * The pages of a cache of several layers.  A page number names the same page
 * in every layer; ref counts the table entries that hold it (a caller may add
 * references of its own), 0 = free.  Entries of a row beyond a sequence's
 * pages are -1.
 */
typedef struct moe_kv4_pool {
    void* pages;               /* layer l's pages start at pages + l * layer_stride */
    long long layer_stride;    /* bytes, a multiple of 16 */
    long long page_bytes;      /* bytes of a page of one layer, a multiple of 16 */
    int32_t* page_table;       /* [S][max_pages] */
    int32_t* seq_len;          /* [S] */
    int32_t* ref;              /* [n_pages] */
    int32_t n_layers;
    int32_t n_pages;
    int32_t max_pages;
    int32_t S;
} moe_kv4_pool;

/*
 * Room for n_new[s] more tokens of every sequence (0: unchanged; negative:
 * the sequence loses its last -n_new[s] tokens and the pages that it no
 * longer needs).  Where a sequence grows into a partly filled page that
 * others hold too, it first gets a copy of it (of every layer); of the
 * sequences that share such a page in this call the last keeps it if nobody
 * else holds it.  Pages are taken from the free ones in ascending order, in
 * the order of the sequences, a copy before new pages.  Pages freed by the call
 * are free for the next one.  All or nothing: with too few free pages
 * (MOE_DEV_NO_PAGES), or a length beyond the table or a held page outside the
 * pool (MOE_DEV_BAD_INDEX, detail = sequence), nothing changes.
 *   workspace  moe_kv4_pool_workspace(S, n_pages) bytes, 256-byte aligned; holds
 *            nothing between calls, so one buffer serves pools of any sizes in turn;
 *            serves one call at a time.
 * Limits: S <= 4096.
 */
moe_status_t moe_kv4_reserve(const moe_kv4_pool* pool, const int32_t* n_new, void* workspace, size_t ws_bytes,
                             moe_dev_status* st, void* stream);

/*
 * Every sequence becomes what parent[s] was before the call: its table row
 * and length; -1 = empty.  Pages gain and lose references accordingly; none
 * is copied.  So parent = s keeps, another sequence's number forks it (or
 * reorders beams), -1 frees.  A parent outside [-1, S) is reported
 * (MOE_DEV_BAD_INDEX) and its sequence kept.  Limits: S <= 4096.
 */
moe_status_t moe_kv4_assign(const moe_kv4_pool* pool, const int32_t* parent, moe_dev_status* st, void* stream);

/*
 * Packs the pool: with n pages in use, those numbered n and above move, in
 * ascending order, to the free pages below n, in every layer: the k-th of them
 * to the k-th free one.  Tables and references follow (a caller that holds
 * pages of its own finds their new numbers by that rule from the references
 * before the call).  A table entry other than -1 that names no page in use is
 * reported (MOE_DEV_BAD_INDEX, detail = entry) and stays.
 * n_live [1] out (may be NULL): n.
 *   workspace  as for moe_kv4_reserve.
 */
moe_status_t moe_kv4_compact(const moe_kv4_pool* pool, int32_t* n_live, void* workspace, size_t ws_bytes,
                             moe_dev_status* st, void* stream);
size_t moe_kv4_pool_workspace(int S, int n_pages);

/* ---------------------------------------------------------------- */
/* Eviction from the cache by the attention that its tokens draw      */
/* ---------------------------------------------------------------- */
/*
 * The attention weight that cached tokens draw: for every token j of sequence s
 *     score[s][j] += sum over rows i and heads h of exp(scale * q_i . k_j - lse[i][h])
 * over the rows q_start[s] + i that see token j, as moe_attention_kv4 lets them
 * (places, window, key heads); with that call's lse the exponentials are its
 * probabilities.  A row whose lse is -inf sees nothing and adds nothing.
 *
 *   q, ld_q, q_start, scale, window  as for moe_attention_kv4
 *   last     count only the last `last` rows of each sequence; 0 = all
 *   lse      [T][n_q] fp32
 *   score    [S][ld_score] fp32, ld_score >= max_pages * 64; entries beyond a
 *            sequence's tokens are not touched
 *   fresh    nonzero: the entries of the rows' own tokens (the last of the
 *            sequence) are set instead of added to.  With one score for all
 *            layers the first layer's call is fresh and the others add.
 *   max_new  an upper bound of the rows of a sequence; one with more is reported
 *            (MOE_DEV_BAD_INDEX, detail = sequence) and adds nothing
 *   workspace  moe_kv4_weigh_workspace() bytes, 256-byte aligned; holds nothing between
 *            calls, so one buffer serves calls of any sizes in turn; serves one call at a
 *            time; may be NULL where that is 0
 * The cache's values are not read.  Products run on the tensor cores with fp32
 * sums, keys exact: in fp16 with q scaled by a power of two of its row, or, where a
 * sequence has many rows, in bf16 (q as it is).  Exponentials and their sums are
 * fp32, added in an order that depends on the sizes, the sequences' lengths and rows and the
 * device's number of SMs alone, so results are reproducible bit for bit.  A page outside the pool, a length beyond the table
 * or a bad q_start is reported (MOE_DEV_BAD_INDEX) and adds nothing.
 * Limits: those of moe_attention_kv4.
 */
moe_status_t moe_kv4_weigh(const void* q, long long ld_q, int T, int n_q, const moe_kv4_cache* cache,
                           const int32_t* q_start, int max_new, const float* lse, float scale, int window,
                           int last, float* score, long long ld_score, int fresh, void* workspace,
                           size_t ws_bytes, moe_dev_status* st, void* stream);
size_t moe_kv4_weigh_workspace(int S, int T, int n_q, int n_kv, int head_dim, int max_pages);

/*
 * Eviction: every sequence with more than budget[s] tokens keeps that many --
 * its first `sinks`, its last `recent`, and of the others those with the
 * highest scores (equal ones: the earlier first; a NaN counts as lowest) -- in
 * their order, moved to its front in every layer.  Keys and values are moved as
 * they are (a rotated key keeps the position that it was turned to).  The
 * pages behind are released.  budget[s] < 0, or at least the sequence's tokens:
 * the sequence stays as it is.
 *
 *   head_dim  D of the pool's caches (64 or 128; page_bytes is n_kv * 64 * (D + D/8))
 *   score    [S][ld_score] fp32, ld_score >= max_pages * 64: the kept tokens'
 *            entries move with them, those behind are set to 0 up to the old length
 *   budget   [S] int32; at least sinks + recent where the sequence has more tokens
 *   kept     [S][ld_kept] int32 out, or NULL: the place that each token had
 *            before (of every sequence), -1 from its new length on
 * Pages in front of the first evicted token's stay as they are.  Of the others
 * a page that only one table entry holds is rewritten in place; one that
 * others hold too is left, and a free one taken for it (ascending, in the order
 * of sequences and places).  In a rewritten page the codes and scales behind the last
 * token are zero.  Pages freed by the call are free for the next one.  All or
 * nothing: with too few free pages (MOE_DEV_NO_PAGES, detail = how many more), or a
 * length beyond the table, a held page outside the pool or a budget below
 * sinks + recent (MOE_DEV_BAD_INDEX, detail = sequence), nothing changes and
 * nothing is written, kept included.
 *   workspace  moe_kv4_evict_workspace() bytes, 256-byte aligned; holds nothing
 *            between calls, so one buffer serves pools of any sizes in turn; serves one call
 *            at a time.
 * Limits: S <= 4096; tables of at most 2^31 - 1 tokens a sequence.
 */
moe_status_t moe_kv4_evict(const moe_kv4_pool* pool, int head_dim, float* score, long long ld_score,
                           const int32_t* budget, int sinks, int recent, int32_t* kept, long long ld_kept,
                           void* workspace, size_t ws_bytes, moe_dev_status* st, void* stream);
size_t moe_kv4_evict_workspace(int S, int max_pages, int n_pages);

/* ---------------------------------------------------------------- */
/* Products with weights in 4 bits                                    */
/* ---------------------------------------------------------------- */
/*
 * Weights [N][K] in 4 bits: number (n, k) stands for c * s * row_scale[n], c an
 * e2m1 code and s the e4m3 scale of columns 16 (k/16) .. + 15 of its row.
 *
 * tiles  [ceil(N/128)][ceil(K/128)][9216] bytes, 16-byte aligned.  In a tile
 *        (r, k = row and column in it, c = k / 32): the code of (r, k) is in the
 *        16-byte run at
 *            (r/8)*512 + c*128 + ((r%8) ^ (2c))*16,
 *        eight columns to a 32-bit word, the even ones in its lower half, the
 *        j-th two (j = k%8/2) in bits 15 8 7 6, 12 5 4 3, 9 2 1 0 or
 *        14 13 11 10 of a half (sign, then magnitude from its high bit); the
 *        scale of (r, k) is byte 8192 + r*8 + k/16.  Codes and scales beyond N or K are zero.
 *        (Three of four codes then become bf16 with a shift and a mask.)
 */
typedef struct moe_w4 {
    void* tiles;
    float* row_scale;   /* [N], or NULL: 1 */
    int32_t N;
    int32_t K;
} moe_w4;

/* Bytes of the tiles; 0 for sizes below 1. */
size_t moe_w4_bytes(int N, int K);

/*
 * Packs weights: row_scale[n] = max|w[n]| / 2688 (1 where that is below 2^-100),
 * z = w * (1/row_scale), and codes and scales of z as in the cache (above): s =
 * e4m3(max|z| * (1/6)), c = e2m1(z * (1/s)), every operation one fp32 operation.
 *   w   [N][ld] BF16 or F32
 *   out tiles and row_scale (not NULL) are written
 * A NaN or infinite weight is packed as zero and reported (MOE_DEV_NONFINITE,
 * detail = row).
 */
moe_status_t moe_w4_pack(const void* w, int dtype, long long ld, const moe_w4* out, moe_dev_status* st, void* stream);

/*
 * y[t][n] = row_scale[n] * sum_k x[t][k] c[n][k] s[n][k/16] + bias[n]  (+ y[t][n])
 *
 *   x     [T][ld_x] bf16, K numbers a row (any alignment; rows that start at
 *         16-byte boundaries are read faster)
 *   bias  [N] fp32, or NULL
 *   y     [T][ld_y] BF16 or F32, N numbers a row; must not overlap x
 *   add   nonzero: added to what y holds (F32 only), e.g. a residual
 *   st    an internal wait that gave up (MOE_DEV_TIMEOUT); no number of x or w is reported
 * Products are exact, sums fp32, results rounded once to y's type.  Sums are added
 * in an order that depends on the sizes and the device's number of SMs alone, not on
 * where rows start, so results are reproducible bit for bit.
 * Limits: N, K <= 2^24, T <= 2^20.
 */
moe_status_t moe_linear_w4(const void* x, long long ld_x, int T, const moe_w4* w, const float* bias, void* y,
                           int y_dtype, long long ld_y, int add, moe_dev_status* st, void* stream);

/* ---------------------------------------------------------------- */
/* Verification of drafted tokens                                     */
/* ---------------------------------------------------------------- */
/*
 * How many of each sequence's drafted tokens the target accepts, and the token
 * that follows them; tokens are then distributed as the target's.
 *
 * Rows q_start[s] .. q_start[s+1]-1 of a step are a sequence's newest known
 * token and its n drafts behind it.  logits of a row are the target's for the
 * place behind it, so row r decides on the draft tokens[r+1].  With p the
 * target's and q the drafting model's distribution at a row, the draft x is
 * accepted if uniform[r+1] * q(x) < p(x); the first one that is not ends
 * the run, and the next token is drawn from max(p - q, 0); with all accepted it
 * is drawn from the last row's p.  uniform[q_start[s]] draws it: of the tokens
 * in order, the first whose cumulated weight exceeds uniform * the sum.
 *
 *   logits        [T][ld] BF16 or F32, V numbers a row (any alignment)
 *   draft_logits  [T][ld_draft], same type: row r's distribution is the one that
 *                 tokens[r+1] was drawn from (a sequence's last row is not read);
 *                 NULL: drafts without a distribution, q = 1 at the draft
 *   tokens        [T] int32; uniform [T] fp32 from [0, 1)
 *   temperature   [S] fp32, or NULL: 1.  Below 2^-60 (0 among it): greedy -- a draft
 *                 is accepted if it is the target's strongest (of equal ones the lowest
 *                 number), and so is the next token
 *   accepted      [S] int32 out: accepted drafts
 *   next          [S] int32 out: the token that follows; -1 for a sequence without rows
 *   n_new         [S] int32 out, or NULL: accepted - n, what moe_kv4_reserve takes to
 *                 cut the refused drafts' tokens from the cache
 *   workspace     moe_verify_workspace() bytes, 256-byte aligned; holds nothing between calls; serves
 *                 one call at a time
 * A logit of -inf is a token that cannot be.  A row with a NaN, with +inf or
 * without a finite logit is reported (MOE_DEV_NONFINITE, detail = row; T + row for
 * draft_logits), and so is a temperature that is NaN, negative or infinite
 * (detail = -1 - sequence) and a draft outside [0, V) (MOE_DEV_BAD_INDEX, detail = row):
 * such a sequence has accepted 0 and next -1.  A bad q_start is reported (MOE_DEV_BAD_INDEX, detail = sequence)
 * and its sequence counts as without rows; where starts around it give a row to several sequences,
 * the row is weighed for the first of them, and one with another temperature has accepted 0 and next -1.
 *
 * Whole numbers decide, so that results do not depend on the order of a sum:
 * with m the row's maximum, it = log2(e) / temperature,
 *     t = max((logit - m) * it, -60),  n = rint(t),  f = t - n
 *     w = 2^n * (((((c6 f + c5) f + c4) f + c3) f + c2) f + c1) f + c0,  c_i = ln(2)^i / i!
 * each operation one fp32 operation (the series' steps fused), W = rint(w 2^42), Z the sum
 * of a row's W, p(x) = W/Z in fp64; max(p - q, 0) is rint(max(w_p i_p - w_q i_q, 0) 2^42) with i =
 * 2^42/Z rounded to fp32, or p's W with the draft's set to 0 when draft_logits is NULL; where all of
 * it is 0, p's W.  The cumulated weight is compared with floor(uniform * sum) in fp64, at most sum - 1.
 * Limits: V <= 2^20, T <= 2^16, S <= 16384.
 */
moe_status_t moe_verify_drafts(const void* logits, int dtype, long long ld, int T, int V, const int32_t* tokens,
                               const float* uniform, const int32_t* q_start, int S, const void* draft_logits,
                               long long ld_draft, const float* temperature, int32_t* accepted, int32_t* next,
                               int32_t* n_new, void* workspace, size_t ws_bytes, moe_dev_status* st, void* stream);
size_t moe_verify_workspace(int T, int S, int V);

/* ---------------------------------------------------------------- */
/* Workspace sizes and status strings                                 */
/* ---------------------------------------------------------------- */
#define MOE_OP_DISPATCH 1
#define MOE_OP_FFN 2
#define MOE_OP_CALIBRATE 3   /* moe_similarity_calibrate: T = calibration tokens n */
#define MOE_OP_TOKEN_WEIGHTS 4   /* moe_token_weights: depends on T only */
#define MOE_OP_ROUTE_DISPATCH 5  /* moe_route_dispatch: a fixed 512 bytes */

/* Bytes of device workspace that `op` needs for these sizes (0 if none).
 * capped != 0 asks for the capacity-mode size of MOE_OP_DISPATCH; dtype
 * selects the FFN kernel.  Returns 0 for invalid arguments. */
size_t moe_workspace_size(int op, int T, int H, int I, int N, int k, int R, int capped, int dtype);

/* Static string for a status code (host or device MOE_DEV_* codes are
 * told apart by the `device` flag). */
const char* moe_status_string(int code, int device);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
