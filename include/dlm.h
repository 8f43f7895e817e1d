/*
 * dlm.h -- C ABI of the MI355X (gfx950) hot path of token-level pre-gated
 * dynamic LoRA adapters (AdaFuse: "Accelerating Dynamic Adapter Inference via
 * Token-Level Pre-Gating and Fused Kernel Optimization").
 *
 * Three operations, and below them what trains their adapters:
 *   dlm_pregate  one top-2 routing decision per token, made once and reused by
 *                every adapted layer (AdaFuse digest, section 2-ga "token-level
 *                pre-gating"; English abstract, "decide-once, apply-everywhere").
 *   dlm_switch   one launch that removes the previous token's gated adapters
 *                from every adapted weight of every layer and merges the current
 *                token's, in place (digest section 2-na "fused adapter
 *                switching": concatenated adapters, parallel GEMM in one
 *                kernel, in-place update, prefetch).
 *   dlm_sgmm     the unmerged batched form for rows with different expert sets,
 *                y += sum_k g_k (x A_k^T) B_k^T, segmenting rows by their set
 *                (digest section 2-na names the SGMM, "segmented gather matrix
 *                multiplication", kernel).
 *   dlm_route    routing from logits (top k of up to 512 experts, biased, in
 *                groups) and dlm_route_backward, the gradient of its weights;
 *   dlm_sgmm_group_backward  the gradients of the grouped SGMM: its inputs',
 *                its banks' and its gates';
 *   dlm_adamw_*  AdamW over many tensors in one launch, with fp32 or 8-bit
 *                moments;
 *   dlm_balance  the router's balance loss over packed sequences, its counts, and
 *                dlm_balance_backward, its gradient;
 *   dlm_muon_*   a step of momentum orthogonalised by Newton-Schulz products over
 *                many matrices;
 *   dlm_i8_*     the frozen base's products in 8-bit integers, and their input
 *                gradients.
 *
 * Conventions (all calls):
 *   - Pointers are DEVICE pointers unless marked (host).  The caller owns every
 *     buffer and every stream; `stream` is a hipStream_t passed as void*
 *     (NULL = the legacy default stream).  Calls only enqueue work on `stream`
 *     and return; device-side failures are reported through the status calls.
 *   - Layouts are row-major.  Adapted weight W is [d_out][d_in]; expert bank A
 *     is [E][r][d_in] (A_e = the LoRA "down" matrix), B is [E][d_out][r] (B_e =
 *     the LoRA "up" matrix); the delta of expert e is B_e A_e.
 *   - An expert set is two slots (idx[2] int32, g[2] fp32).  idx = -1 is an
 *     empty slot; a NULL set pointer is the empty set.  Slot order does not
 *     change results of dlm_switch (the kernel orders the slots itself).
 *   - dtype: DLM_F32 or DLM_BF16 for every floating tensor of a call (x, Wr,
 *     W, A, B, y); gates g are always fp32, indices int32.
 *   - bf16 arithmetic: bf16 operands, fp32 accumulation; results are rounded
 *     to bf16 once, to nearest even.
 *   - Every call validates its arguments on the host before touching the GPU;
 *     on a negative status nothing was enqueued and no memory was changed.
 *     dlm_last_error() gives a text for the last failure of the calling thread.
 *   - Thread safety: calls on distinct handles / workspaces may run
 *     concurrently; one handle or workspace must not be used by two calls in
 *     flight at once (the caller orders its streams).
 */
#ifndef DLM_H
#define DLM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    DLM_OK = 0,
    DLM_EINVAL = -1,     /* null pointer, bad count, bad value */
    DLM_ESHAPE = -2,     /* a size out of the supported range, or sizes whose
                            launch grid would exceed 2^32 - 1 work-items (refused
                            before anything is launched) */
    DLM_EDTYPE = -3,     /* unknown or unsupported dtype */
    DLM_EALIGN = -4,     /* a pointer or row pitch not 16-byte aligned (bf16 fast path) */
    DLM_EWORKSPACE = -5, /* workspace missing or too small */
    DLM_EHIP = -6,       /* a HIP runtime call failed */
    DLM_EDEVICE = -7,    /* the device rejected an expert set (index out of range,
                            non-finite gate); reported by the status calls */
    DLM_ENOMEM = -8      /* a host or device allocation failed */
} dlm_status;

typedef enum { DLM_F32 = 0, DLM_BF16 = 1 } dlm_dtype;

/* Compile-time limits of the library. */
#define DLM_MAX_EXPERTS 32
#define DLM_MAX_RANK 128
#define DLM_MAX_CENTROIDS 1024   /* per adapter, dlm_pregate_centroid */

/* Text of the calling thread's last non-OK status (static storage). */
const char* dlm_last_error(void);

/* Library version string. */
const char* dlm_version(void);

/* ------------------------------------------------------------------ router */

/*
 * Top-2 pre-gate for T tokens (digest section 2-ga: a lightweight top-2 router
 * at the first layer selects each token's expert set; the set is then reused by
 * every layer).
 *   x  [T][d]  token activations at the first layer (dtype)
 *   Wr [d][E]  router weight (dtype)
 *   idx [T][2] out, int32: slot 0 = expert with the largest logit l = x.Wr,
 *              slot 1 = largest of the rest; equal logits -> lower index.
 *   g   [T][2] out, fp32: softmax over all E renormalised over the kept two,
 *              i.e. g0 = 1/(1+exp(l1-l0)), g1 = 1 - g0 (computed in binary64,
 *              rounded once to fp32).
 * Logits accumulate in binary64 (the products of fp32/bf16 inputs are exact),
 * so the decision is exact up to the summation order.  idx is always in
 * [0, E) and idx[t][0] != idx[t][1], also for non-finite inputs.
 * Requires 2 <= E <= DLM_MAX_EXPERTS, d >= 1, 0 <= T < 2^31 (T = 0 enqueues
 * nothing).
 */
int dlm_pregate(const void* x, const void* Wr, int64_t T, int64_t d, int32_t E,
                int32_t dtype, int32_t* idx, float* g, void* stream);

/*
 * Training-free nearest-centroid pre-gate (the ARIADNE page: each adapter is
 * represented by centroids of its training data's embeddings; the input's
 * embedding is compared with them and the closest adapter is chosen), with the
 * same output format as dlm_pregate so it feeds dlm_switch / dlm_sgmm as is:
 *   x [T][d], C [E][J][d] (row-major, dtype; C adapter-major: J centroids of
 *   adapter 0, then adapter 1, ...).  Adapter distance = min over its J
 *   centroids of sum_k (x_k - c_k)^2, accumulated in binary64 with a fixed
 *   reduction order.  idx[t] = {nearest adapter (ties -> lower index), -1},
 *   g[t] = {1, 0}.
 * Requires 1 <= E <= DLM_MAX_EXPERTS, 1 <= J <= DLM_MAX_CENTROIDS, d >= 1,
 * 0 <= T < 2^31.  One launch on `stream`, no allocation.
 */
int dlm_pregate_centroid(const void* x, const void* C, int64_t T, int64_t d, int32_t E,
                         int32_t J, int32_t dtype, int32_t* idx, float* g, void* stream);

/*
 * Routing from router logits for any number of experts (the top-2 pre-gate's
 * general form, for routers whose product is computed elsewhere and for
 * training; k = 2 with E <= DLM_MAX_EXPERTS gives sets that dlm_switch and
 * dlm_sgmm take as they are):
 *   s      softmax(l) over the available experts of the row, or sigmoid(l)
 *   key    s + bias (bias [E] fp32 or NULL: it steers the choice, for balance,
 *          and is not part of the weights)
 *   groups n_groups runs of E / n_groups experts, each ranked by its best key
 *          (group_top 1) or the sum of its best two (group_top 2); the best
 *          keep_groups of them stay (n_groups = 1: all experts)
 *   idx    [T][k] the k largest keys of the kept groups, descending
 *   g      [T][k] scale * s_i, or with renorm scale * s_i / sum_j s_j over the
 *          chosen (0 where that sum is 0)
 * Equal keys go to the lower index.  Without a bias (and with group_top 1) the
 * logits themselves are compared, exactly; otherwise keys are binary64 values
 * and two within 2^-43 of their size may count as equal.  Scores and sums are
 * binary64; g is rounded to fp32 once.  (A sigmoid below e^-700 counts as 0.)
 * A logit of -inf or NaN marks an expert that is not available to the row: its
 * score is 0 and it is never chosen; +inf counts as the largest fp32 value.  A
 * row with fewer than k available experts in its kept groups ends in empty
 * slots (idx -1, g 0); a padding row of -inf has only those.
 *   logits [T] rows of E (dtype), ld elements apart (ld >= E)
 *   counts [E] int32 or NULL: the number of rows that chose each expert is
 *          ADDED to it (the load a balance bias is steered by)
 * One launch on `stream`, no allocation.  T = 0 enqueues nothing.
 */
#define DLM_MAX_ROUTE_EXPERTS 512
#define DLM_MAX_ROUTE_K 16
#define DLM_MAX_ROUTE_GROUPS 32
typedef enum { DLM_SOFTMAX = 0, DLM_SIGMOID = 1 } dlm_score;
typedef struct {
    int32_t k;            /* 1 .. min(DLM_MAX_ROUTE_K, keep_groups * E / n_groups) */
    int32_t score;        /* dlm_score */
    int32_t n_groups;     /* 1 .. DLM_MAX_ROUTE_GROUPS, dividing E */
    int32_t keep_groups;  /* 1 .. n_groups */
    int32_t group_top;    /* 1 or 2 */
    int32_t renorm;       /* 0 or 1 */
    float scale;
} dlm_route_cfg;
int dlm_route(const void* logits, int64_t ld, const float* bias, int64_t T, int32_t E, int32_t dtype,
              const dlm_route_cfg* cfg, int32_t* idx, float* g, int32_t* counts, void* stream);

/*
 * The gradient of dlm_route's weights: given dg [T][k] = dLoss/dg for the
 * choice idx [T][k], dlogits [T] rows of E (dtype, ldd elements apart) =
 * dLoss/dlogits, every element of the rows written.  The choice itself has no
 * gradient.  Entries of idx outside [0, E) are empty slots, and so are those
 * that name an expert that is not available; an expert named twice
 * counts twice.  binary64 inside, rounded once.  cfg as for dlm_route (its
 * groups only bound k).  One launch on `stream`, no allocation.
 */
int dlm_route_backward(const void* logits, int64_t ld, const int32_t* idx, const float* dg, int64_t T, int32_t E,
                       int32_t dtype, const dlm_route_cfg* cfg, void* dlogits, int64_t ldd, void* stream);

/*
 * The router's balance loss over packed sequences, with the counts it steers by.
 * Rows offsets[q] .. offsets[q + 1] - 1 are sequence q (offsets [n_seq + 1] int32 on
 * the device, not decreasing, within [0, T]; NULL: all T rows are one sequence).
 *   p      softmax(l) over the available experts of the row, or sigmoid(l) over its
 *          sum there; a logit of -inf or NaN marks an expert that is not available,
 *          as for dlm_route, and a row without any (padding) belongs to nothing
 *   and per sequence, over its n rows that have an expert:
 *   counts [n_seq][E] int32: the slots of idx [T][k] that name expert e (entries
 *          outside [0, E), or that name an expert not available, are empty)
 *   rows   [n_seq] int32: n
 *   probs  [n_seq][E] fp32: the mean of p_e
 *   loss   [2] fp32: alpha * mean over the sequences of sum_e f_e probs_e with
 *          f_e = E counts_e / (k n), which is alpha for a balanced router, and
 *          zeta * mean over the sequences of the mean of (log sum_e exp l_e)^2
 * A sequence without rows counts as 0 in both means.  zeta must be 0 for sigmoid
 * scores.  Everything is written, not added to; also for T = 0.  p is fp32, its sums
 * binary64; bitwise reproducible.  Two launches (one for a single sequence of few
 * rows), no allocation.
 * workspace: >= dlm_balance_workspace_size(T, E, n_seq) bytes, 256-byte aligned, of
 * any content.
 */
#define DLM_MAX_BALANCE_SEQS 65536
typedef struct {
    int32_t k;     /* slots of a row of idx: 1 .. DLM_MAX_ROUTE_K */
    int32_t score; /* dlm_score */
    float alpha, zeta;
} dlm_balance_cfg;
int dlm_balance_workspace_size(int64_t T, int32_t E, int32_t n_seq, size_t* bytes);
int dlm_balance(const void* logits, int64_t ld, const int32_t* idx, const int32_t* offsets, int32_t n_seq, int64_t T,
                int32_t E, int32_t dtype, const dlm_balance_cfg* cfg, float* loss, int32_t* counts, int32_t* rows,
                float* probs, void* workspace, size_t ws_bytes, void* stream);

/*
 * The gradient of loss[0] dloss[0] + loss[1] dloss[1] (dloss [2] fp32 on the device,
 * NULL = 1, 1) with the counts held constant: dlogits [T] rows of E (dtype, ldd
 * elements apart) are written, or with accumulate != 0 added to (it joins
 * dlm_route_backward's), rounded once.  Rows of no sequence are left as they are;
 * padding rows and experts not available get 0.  counts and rows are dlm_balance's,
 * or their sums over several processes' batches (the loss is then that of the joint
 * batch, and the processes' gradients add up to its).  One launch, no allocation.
 * T = 0 enqueues nothing.
 */
int dlm_balance_backward(const void* logits, int64_t ld, const int32_t* counts, const int32_t* rows, const int32_t* offsets,
                         int32_t n_seq, int64_t T, int32_t E, int32_t dtype, const dlm_balance_cfg* cfg, const float* dloss,
                         int32_t accumulate, void* dlogits, int64_t ldd, void* stream);

/* ------------------------------------------------------------ fused switch */

/* One adapted weight and its expert bank. */
typedef struct {
    void* W;        /* [d_out][d_in], updated in place by dlm_switch */
    const void* A;  /* [E][r][d_in] */
    const void* B;  /* [E][d_out][r] */
    int64_t d_out;
    int64_t d_in;
} dlm_proj;

typedef struct dlm_layers dlm_layers;

/*
 * Build the table of every adapted weight of every layer (L*P entries) that
 * one dlm_switch call updates.  Copies the host descriptors to a small device
 * table plus a device error word.  The buffers themselves stay owned by the
 * caller and must outlive the handle.
 *   projs (host) [n]; E in [1, DLM_MAX_EXPERTS]; r in [1, DLM_MAX_RANK];
 *   scale = the LoRA scale s multiplying every delta.
 * bf16: every W/A/B pointer 16-byte aligned and every d_in a multiple of 8.
 * bf16 with r in 17..64: the handle also allocates and fills a packed copy of
 * every A bank (E * ceil(d_in/64) * 64 * 16*ceil(r/16) bf16 per weight, about
 * the size of A) that the switch stages into LDS with direct copies; the
 * device is synchronised before returning.  The copy is taken here: after
 * changing an A bank in place call dlm_layers_repack.  Otherwise does not
 * synchronise.  All of it is freed by destroy.  *out (host) receives the handle.
 */
int dlm_layers_create(const dlm_proj* projs, int32_t n, int32_t E, int32_t r,
                      float scale, int32_t dtype, dlm_layers** out);

/* Free the handle's device memory (synchronises the device first). */
int dlm_layers_destroy(dlm_layers* h);

/*
 * Refresh the handle's packed A copies from the caller's A banks: one launch
 * per weight on `stream`, no allocation (no-op when the handle keeps none).
 */
int dlm_layers_repack(dlm_layers* h, void* stream);

/*
 * One fused switch over every weight of the handle, one kernel launch:
 *   W <- round( W - s*sum_{k in old} g_k B_k A_k + s*sum_{k in new} g_k B_k A_k )
 * (digest section 2-na: remove the previous token's adapters and merge the
 * current token's, on concatenated adapter matrices, in place).  The sets are
 * read from DEVICE memory (idx[2] int32, g[2] fp32; NULL = empty set), so a
 * router output can feed the switch with no host synchronisation.  Each
 * slot's product is accumulated separately in fp32 and scaled by s*g_k in
 * fp32; the old and new halves use the same expression, so a switch to the
 * same set leaves W bitwise unchanged.
 * A set with an index outside [-1, E) or a non-finite gate on a used slot is
 * rejected on the device: no weight is written and the handle's error word is
 * set (read it with dlm_layers_status).
 * No allocation; one launch on `stream`.  Reads the packed A copy where the
 * handle keeps one, so A banks changed after create need dlm_layers_repack.
 */
int dlm_switch(dlm_layers* h, const int32_t* old_idx, const float* old_g,
               const int32_t* new_idx, const float* new_g, void* stream);

/* Number of kernel launches one dlm_switch call makes (always 1). */
int dlm_switch_launches(const dlm_layers* h);

/* -------------------------------------------- merged-weight products */

/*
 * The decode step after a switch: each adapted projection is the product of
 * its merged weight with the layer input, y_i = W_i x_i (Chinese digest,
 * "technical framework": the fused kernel merges the selected adapters into
 * the backbone and carries out the computation in a single kernel).
 *
 * Bind one input and one output vector to every weight of the handle:
 *   x (host) [n] device pointers, x_i [d_in_i] in the handle's dtype (bf16:
 *   16-byte aligned); y (host) [n] device pointers, y_i [d_out_i] fp32, not
 *   overlapping x_i or W_i.  The device is synchronised first (launches in
 *   flight on any stream finish with the previous binding), then the pointers
 *   are copied into the device table; the buffers stay owned by the caller.  bf16 handles with
 *   r <= 16 also get a partial-product buffer (sum of ceil(d_in_i/256) *
 *   d_out_i floats), and every handle a buffer for dlm_gemv_unmerged's rank
 *   vectors (sum of ceil(d_in_i/2048) * 2 r floats), freed by destroy.
 *   Binding again replaces the vectors.
 */
int dlm_layers_bind_vectors(dlm_layers* h, const void* const* x, float* const* y);

/*
 * y_i = W_i x_i for every weight (fp32 accumulation, one rounding to fp32 per
 * lane sum, then a fixed-order reduction: bitwise reproducible).  One launch,
 * no allocation.  DLM_EINVAL if no vectors are bound.
 */
int dlm_gemv(dlm_layers* h, void* stream);

/*
 * dlm_switch followed by y_i = W'_i x_i with the new (rounded) weights.  bf16
 * with r <= 16: one fused kernel reads each W once, writes W' and forms
 * per-256-column partial products, and a second launch adds each row's
 * partials in column order.  Otherwise the switch and dlm_gemv's kernel run
 * back to back.  Two launches either way, no allocation.  A set the switch
 * rejects leaves W and y unchanged (the error word is set as for dlm_switch).
 */
int dlm_switch_gemv(dlm_layers* h, const int32_t* old_idx, const float* old_g,
                    const int32_t* new_idx, const float* new_g, void* stream);

/* Number of kernel launches one dlm_switch_gemv call makes (always 2). */
int dlm_switch_gemv_launches(const dlm_layers* h);

/*
 * The decode product with one set's adapters left unmerged: for every weight
 * with its bound vectors,
 *   y_i = W_i x_i + s * sum_k g_k * B_{e_k,i} (A_{e_k,i} x_i)          (fp32 y)
 * W is not modified.  The set is made once per token and applied by every
 * adapted layer (AdaFuse, KR digest section 2-ga, token-level pre-gating); the
 * adapters are the per-row gated LoRA product of the SGMM formula, applied
 * to the token's input here instead of merged into W.
 *   idx [2] int32, g [2] fp32 (device): the set, in dlm_switch's format.
 * Two launches, no allocation: the rank vectors' partials A_e x per (weight,
 * 2048-wide K slice, group of 8 rank vectors) into the handle's buffer
 * (dlm_layers_bind_vectors), then the product, each output row adding its adapters' B row times the slices'
 * sum (slices added in order; every result bitwise reproducible, and the
 * same for the set's two slots in either order).  A set dlm_switch would
 * reject leaves y unchanged and sets the error word (dlm_layers_status).
 * DLM_EINVAL if no vectors are bound or idx / g is null.
 */
int dlm_gemv_unmerged(dlm_layers* h, const int32_t* idx, const float* g, void* stream);

/* Number of kernel launches one dlm_gemv_unmerged call makes (always 2). */
int dlm_gemv_unmerged_launches(const dlm_layers* h);

/*
 * Synchronise `stream`, then read and clear the handle's device error word:
 * *code (host) = DLM_OK or DLM_EDEVICE.
 */
int dlm_layers_status(dlm_layers* h, int32_t* code, void* stream);

/* ------------------------------------------------------------------- SGMM */

/*
 * Workspace bytes dlm_sgmm / dlm_sgmm_group_run need for T rows, problems with
 * d_in up to d_in_max, E experts, rank r and n_problems problems sharing one
 * set of rows: row segmentation, the shrink's per-K-slice partial results
 * (fp32, [n_problems][ceil(d_in_max / 2048)][T][2][r]) and the device status
 * word.  *bytes is host memory.
 */
int dlm_sgmm_workspace_size(int64_t T, int64_t d_in_max, int32_t E, int32_t r,
                            int32_t n_problems, size_t* bytes);

/*
 * Batched unmerged adapters for rows with different expert sets:
 *   y[t] <- round( y[t] + sum_k s*g[t][k] * B_{idx[t][k]} (A_{idx[t][k]} x[t]) )
 *   x [T][d_in], y [T][d_out] (in place, must not overlap x),
 *   idx [T][2] int32 (-1 = empty slot), g [T][2] fp32,
 *   A [E][r][d_in], B [E][d_out][r].
 * Launches: segment (rows sorted by their unordered expert pair, 32-row
 * tiles, the experts each tile uses; a per-1024-row count launch first when
 * T > 8192), shrink (v = x A^T on the tile's experts
 * over 2048-wide K slices staged through LDS 512 columns at a time, bf16
 * MFMA, fp32 partial results kept in the workspace), a K-slice sum in a fixed
 * order (only when d_in > 2048 and r > 64) and
 * expand (y += (s g v) B^T, MFMA with v*s*g split into two bf16 terms, fp32
 * accumulate, one bf16 rounding of y; up to rank 64 it adds the K slices'
 * partials of its tile itself, in the same fixed order).  A bf16 call with at most 4 rows (a
 * decode step) skips the segmentation: with one problem a single launch, in
 * which each 1024-column group computes the rows' rank vectors (fp32 dot
 * products over all of K) and adds s*g*v*B^T to its columns with one rounding;
 * with several, one launch for the rank vectors per 2048-wide K slice and one
 * for the columns.  A bf16 call with 5 to 64 rows and no K-slice sum launch
 * has no segmentation launch either: every shrink and expand workgroup orders
 * the rows itself, in the same order (one wave, one row per lane), so the
 * results are those of the segmented launches bit for bit.  Results are
 * bitwise reproducible run to run.
 * Rows whose two slots are empty are not touched.
 * What is not finite in a bank reaches the rows that choose its expert, no others.
 * A row with an index outside [-1, E) or a non-finite gate on a used slot makes
 * the whole call a no-op on y and sets the workspace status word (read it with
 * dlm_sgmm_status).
 * bf16: x, y, A, B 16-byte aligned; d_in and d_out multiples of 8.
 * workspace: >= dlm_sgmm_workspace_size(T, d_in, E, r, 1) bytes, 256-byte aligned.
 * T = 0 enqueues nothing and looks at no buffer (they may be null).
 */
int dlm_sgmm(const void* x, const int32_t* idx, const float* g, const void* A,
             const void* B, void* y, int64_t T, int64_t d_in, int64_t d_out, int32_t E,
             int32_t r, float scale, int32_t dtype, void* workspace, size_t ws_bytes,
             void* stream);

/*
 * dlm_sgmm for callers that cannot allocate device memory at all (code being
 * captured into a HIP graph, tight serving loops, harnesses that forbid
 * hipMalloc): the same launches and results as dlm_sgmm, with the workspace in
 * the library's own scratch array instead of a caller buffer.  The array is a
 * static device array of DLM_SGMM_NOALLOC_SCRATCH_BYTES, held by every device
 * that loads the library until the process ends; its device address is looked
 * up on the first call on a device (which is when the runtime places the array
 * in that device's memory).  The call itself allocates nothing.
 *   status (device, may be NULL): receives 0 when every row's set was valid,
 *     nonzero when the device rejected one (then y is left unchanged) -- the
 *     workspace status word of dlm_sgmm, written where the caller can read it.
 * Every other argument as for dlm_sgmm.  `stream` must belong to the current
 * device (DLM_EINVAL otherwise).  A call whose workspace
 * (dlm_sgmm_workspace_size(T, d_in, E, r, 1)) exceeds the array returns
 * DLM_EWORKSPACE before anything is enqueued.
 * All calls on one device share that device's array and each call overwrites
 * it: calls that can overlap on one device (different streams, or several host
 * threads) race and give wrong results; order them on one stream.
 */
#define DLM_SGMM_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
int dlm_sgmm_noalloc(const void* x, const int32_t* idx, const float* g, const void* A,
                     const void* B, void* y, int64_t T, int64_t d_in, int64_t d_out, int32_t E,
                     int32_t r, float scale, int32_t dtype, int32_t* status, void* stream);

/* One problem of a grouped SGMM: every problem shares the rows' sets. */
typedef struct {
    const void* x;  /* [T][d_in] */
    const void* A;  /* [E][r][d_in] */
    const void* B;  /* [E][d_out][r] */
    void* y;        /* [T][d_out], in place */
    int64_t d_in;
    int64_t d_out;
} dlm_sgmm_problem;

typedef struct dlm_sgmm_group dlm_sgmm_group;

/*
 * Register n problems (e.g. every adapted projection of every layer) that are
 * run together on the same rows' expert sets: the decide-once routing means
 * one segmentation serves all of them.  Copies the descriptors (host) to a
 * small device table; x, B and y stay owned by the caller and are used in place.
 * bf16: the handle also keeps a packed copy of every distinct A bank
 * (Ap[e][k/8][rho][8] = A[e][rho][k..k+8), the same size as A, allocated and
 * filled here; the device is synchronised before returning), so that the shrink
 * reads A in contiguous runs.  The copy is taken at create time: after
 * changing an A bank in place call dlm_sgmm_group_repack.
 */
int dlm_sgmm_group_create(const dlm_sgmm_problem* probs, int32_t n, int32_t E, int32_t r,
                          float scale, int32_t dtype, dlm_sgmm_group** out);
int dlm_sgmm_group_destroy(dlm_sgmm_group* h);

/*
 * Refresh the handle's packed A copies from the caller's A banks: one launch
 * per distinct bank on `stream`, no allocation (no-op for fp32 groups).
 */
int dlm_sgmm_group_repack(dlm_sgmm_group* h, void* stream);

/*
 * Run every problem of the group for T rows: one segment launch shared by all
 * problems (none up to 64 rows without a K-slice sum, as for dlm_sgmm), then
 * one shrink, one K-slice sum (only when some d_in > 2048 and r > 64) and one
 * expand launch covering all problems.
 * workspace: >= dlm_sgmm_workspace_size(T, max d_in, E, r, n_problems) bytes.
 */
int dlm_sgmm_group_run(dlm_sgmm_group* h, const int32_t* idx, const float* g, int64_t T,
                       void* workspace, size_t ws_bytes, void* stream);

/*
 * Gradients of the group's product (training the adapters and the router that
 * gates them).  Bind every problem's buffers once:
 *   dy (host) [n] device pointers, dy_i [T][d_out_i] = dLoss/dy_i (dtype)
 *   dx (host) [n] device pointers or NULL, dx_i [T][d_in_i] (dtype): the
 *      adapters' share is ADDED to it, in place (it joins what the base product
 *      left there); NULL entries are not wanted.  Problems that read one x may
 *      share one dx: their shares are added in problem order, each with a
 *      rounding of its own
 *   dA, dB (host) [n] device pointers, dA_i [E][r][d_in_i], dB_i [E][d_out_i][r]
 *      fp32
 * bf16: all 16-byte aligned.  The handle allocates memory for the banks'
 * transposes (the banks' size); the device is synchronised first.  The buffers
 * stay owned by the caller.  Binding again replaces them (calls captured into
 * graphs before then read freed tables: capture them again).
 */
int dlm_sgmm_group_bind_grads(dlm_sgmm_group* h, const void* const* dy, void* const* dx, float* const* dA,
                              float* const* dB);

/*
 * The backward pass of the group for T rows and their sets: with u = A_e x and
 * w = B_e^T dy for the expert e of a row's slot k,
 *   dx[t] <- round( dx[t] + sum_k s g_k A_e^T w )     (rows with a set; others untouched)
 *   dg[t][k] = s sum_problems u . w   ([T][2] fp32 or NULL; 0 for an empty slot)
 *   dA_e = s sum g w x[t]^T,  dB_e = s sum g dy[t] u^T   (over the slots with e;
 *          written whole, 0 for an expert no row chose, or with accumulate != 0 added to)
 * bf16: bf16 operands, fp32 sums; s g u and s g w enter dA and dB as three bf16
 * terms (24 bits), s g w enters dx as two.  An infinity among them, or in x or dy,
 * may become NaN.
 * What is not finite in a bank reaches the rows that choose its expert, no others.
 * Reads the banks as they are, and refreshes the packed A copies that the
 * forward call reads on the way.  Every result is bitwise reproducible.  A set the forward call would reject leaves all of
 * them unchanged and sets the workspace status word (dlm_sgmm_status).  T = 0
 * writes zeros to dA and dB unless accumulate, and looks at nothing else.
 * workspace: >= dlm_sgmm_group_backward_workspace_size(h, T) bytes (asked once
 * the buffers are bound; it serves any smaller T too), 256-byte aligned.  No
 * allocation.  Launches: segmentation with the banks' transposes, shrink, expand
 * (with the outer products' coefficients), outer products with dg, and for bf16 and
 * more than a few hundred rows the sum of their parts; one more each for T > 8192, for the K-slice sum above rank
 * 64, and for every further problem that shares the same dx.
 */
int dlm_sgmm_group_backward_workspace_size(const dlm_sgmm_group* h, int64_t T, size_t* bytes);
int dlm_sgmm_group_backward(dlm_sgmm_group* h, const int32_t* idx, const float* g, float* dg, int64_t T,
                            int32_t accumulate, void* workspace, size_t ws_bytes, void* stream);

/*
 * Synchronise `stream`, then read and clear the workspace status word:
 * *code (host) = DLM_OK or DLM_EDEVICE.  Besides a rejected expert set, the
 * one-launch shrink + expand sets it if an expand work item waited about a
 * second for its shrink items (status 2) or found they ran on another XCD
 * (status 3); y is then not to be trusted.  Neither happens when the device
 * starts workgroups in order and round-robin over its XCDs.
 */
int dlm_sgmm_status(void* workspace, int32_t* code, void* stream);

/*
 * Number of kernel launches one dlm_sgmm, dlm_sgmm_noalloc or
 * dlm_sgmm_group_run call makes for T rows and n_problems problems of rank r
 * with d_in up to d_in_max: 0 for T = 0; for bf16 with T <= 4, 1 (one problem)
 * or 2; for bf16 up to rank 64, a multiple of 8, with
 * n_problems x ceil(T / 32) >= 256 (and d_in_max up to 4095 x 2048), the segmentation (2 launches when T > 8192,
 * else 1) and one launch running the shrink and the expand; otherwise for bf16
 * with T <= 64 and no K-slice sum, 2 (shrink and expand); else the
 * segmentation, the shrink, the K-slice sum (bf16 with d_in_max > 2048 and
 * r > 64 only) and the expand.  Returns -1 (with the last
 * error set) for a negative T, d_in_max < 1, r outside [1, DLM_MAX_RANK],
 * n_problems < 1 or an unknown dtype.
 */
int dlm_sgmm_launches(int64_t T, int64_t d_in_max, int32_t r, int32_t n_problems, int32_t dtype);

/* ---------------------------------------------------------- 8-bit products */

/*
 * Rows as 8-bit codes with a scale each: x [T][d] (dtype) ->
 *   q [T][d] int8:  127 x / max|x| of the row, to the nearest whole number (decided on
 *                   the exact quotient; a half goes towards 0)
 *   scale [T] fp32: max|x| / 127
 * A row of zeros has scale 0; a row that is not finite has codes 0 and scale NaN.  The
 * form that dlm_i8_group_create takes weights in.  One launch, no allocation.
 */
int dlm_i8_quantize(const void* x, int64_t T, int64_t d, int32_t dtype, int8_t* q, float* scale, void* stream);

/* One product of a frozen base weight that is held in 8 bits. */
typedef struct {
    const void* x;        /* [T][d_in] */
    const int8_t* W;      /* [d_out][d_in] codes */
    const float* w_scale; /* [d_out] */
    void* y;              /* [T][d_out], written */
    int64_t d_in;         /* 1 .. 131072 */
    int64_t d_out;
} dlm_i8_problem;

typedef struct dlm_i8_group dlm_i8_group;

/*
 * Register n products that run together (the base's share of the problems that a
 * dlm_sgmm_group then adds the adapters' to).  The handle keeps a copy of every W (padded
 * to 16 rows and 128 columns, in the layout its kernels read) and w_scale, taken here;
 * the caller's may be freed.  x and y stay the caller's.  x, y and every pointer need
 * their element's alignment only (16 bytes and sizes a multiple of 8 are faster).
 * Synchronises the device.
 */
int dlm_i8_group_create(const dlm_i8_problem* probs, int32_t n, int32_t dtype, dlm_i8_group** out);

/* Free the handle's device memory (synchronises the device first). */
int dlm_i8_group_destroy(dlm_i8_group* h);

/*
 * y[t][o] = round( s_t w_scale[o] sum_k q[t][k] W[o][k] ) for T rows of every problem, with
 * q and s the row's codes and scale as dlm_i8_quantize makes them.  The sum is exact; the
 * factors are applied in fp32, w_scale's first.  A row of x that is not finite gives NaN in
 * its row of y, and nothing else.  Two launches (the codes, once for problems that share an x; the
 * products), no allocation; one for up to four rows whose codes fit a workgroup's LDS (four
 * of 11008 columns do), while 1, 2 or 4 (the rows, 4 for three) times the 16-channel tiles
 * of all products are at most 2048.  Up to 64 rows the weights are read once, straight into
 * the products' operands.  T = 0 enqueues nothing.
 * workspace: >= dlm_i8_group_workspace_size(h, T) bytes, 256-byte aligned, of any content.
 */
int dlm_i8_group_workspace_size(const dlm_i8_group* h, int64_t T, size_t* bytes);
int dlm_i8_group_run(dlm_i8_group* h, int64_t T, void* workspace, size_t ws_bytes, void* stream);

/*
 * The gradient of the inputs, W held: dx = sum over the problems that share it of
 * dy_i (w_scale_i W_i), with dy in 8 bits too.  Bind once:
 *   dy (host) [n] device pointers, dy_i [T][d_out_i]; dx (host) [n] device pointers,
 *   dx_i [T][d_in_i]; NULL entries of dx (and their dy) are not wanted.  Problems of one
 *   d_in may share a dx (at most 131072 output channels, each problem's counted as a
 *   multiple of 64): their products dy_i[t][o] w_scale_i[o], side by side, are one row of
 *   codes with one scale, formed from the exact products (of fp32 dy a code can be one off
 *   where its quotient lies within 2^-50 of a half of it).
 * The handle allocates the weights' transposes (the weights' size).  Synchronises the
 * device.  Binding again replaces the buffers (calls captured into graphs before then read
 * freed tables: capture them again).
 */
int dlm_i8_group_bind_grads(dlm_i8_group* h, const void* const* dy, void* const* dx);

/*
 * dx[t][i] = round( s_t sum_o q[t][o] W[o][i] ) for T rows, written, or with accumulate != 0
 * added to dx before the rounding.  Otherwise as dlm_i8_group_run; the workspace's size is
 * asked once the buffers are bound.
 */
int dlm_i8_group_backward_workspace_size(const dlm_i8_group* h, int64_t T, size_t* bytes);
int dlm_i8_group_backward(dlm_i8_group* h, int64_t T, int32_t accumulate, void* workspace, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------ AdamW */

/* One tensor of an AdamW step. */
typedef struct {
    void* p;           /* [n] parameter (p_dtype), updated in place */
    const void* g;     /* [n] gradient (g_dtype) */
    float* master;     /* [n] fp32 copy of a bf16 parameter, updated in place (the
                          parameter becomes its rounding), or NULL */
    void* m;           /* [n] first moment: fp32, or int8 codes with 8-bit states */
    void* v;           /* [n] second moment: fp32, or uint8 codes */
    float* m_scale;    /* [ceil(n / 256)] one scale per block (8-bit states only) */
    float* v_scale;
    int64_t n;
    float weight_decay;
} dlm_adamw_param;

typedef struct {
    float lr;
    double beta1, beta2; /* in [0, 1) */
    float eps;           /* > 0, with 8-bit states at least 2^-126 */
} dlm_adamw_cfg;

typedef struct dlm_adamw dlm_adamw;

/*
 * Register n tensors (the adapter banks of every layer, a router's weight) that
 * one AdamW step updates together.  Copies the descriptors to a small device
 * table; the buffers stay owned by the caller, must outlive the handle, and no
 * written one may overlap another.  step = steps already taken (0 at the start
 * of training): the count lives on the device from here on.  seed: of the
 * 8-bit states' rounding noise.
 * state_bits 32: m and v are fp32.  state_bits 8: blocks of 256 consecutive
 * elements share a scale each,
 *   m = m_scale sign(q) (q / 127)^2      v = v_scale (c / 255)^4
 * rounded stochastically (the stored value's mean is the exact one), a positive
 * v to a code of at least 1; all-zero codes and scales are zero moments.
 * Tensors may be of any size and alignment of their element (aligned to four
 * elements they are faster).
 */
int dlm_adamw_create(const dlm_adamw_param* params, int32_t n, int32_t p_dtype, int32_t g_dtype, int32_t state_bits,
                     int64_t step, uint32_t seed, dlm_adamw** out);

/* Free the handle's device memory (synchronises the device first). */
int dlm_adamw_destroy(dlm_adamw* h);

/*
 * One step over every tensor, one launch, no allocation:
 *   t <- t + 1,  g' = grad_scale g,  m <- b1 m + (1 - b1) g',  v <- b2 v + (1 - b2) g'^2
 *   w <- w (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
 * w = the master where there is one, else the parameter; lr = cfg's times
 * *lr_scale.  lr_scale and grad_scale are DEVICE floats or NULL (1): a captured
 * step reads them, and t, on every replay.
 * fp32 throughout (8-bit moments: binary64 between their codes); m and v of
 * this step enter w before they are rounded to codes.
 * An element whose new v is not finite in fp32 (a g' infinite, NaN, or past about
 * 1.8e19 / sqrt(1 - b2), which is 5.8e20 for b2 = 0.999) is left unchanged, with
 * 8-bit states its whole block of 256, and the error word is set.
 */
int dlm_adamw_step(dlm_adamw* h, const dlm_adamw_cfg* cfg, const float* lr_scale, const float* grad_scale, void* stream);

/*
 * Synchronise `stream`, then read the step count and read and clear the error
 * word: *step, *code (host) = DLM_OK or DLM_EDEVICE (some gradient was not finite).
 */
int dlm_adamw_status(dlm_adamw* h, int64_t* step, int32_t* code, void* stream);

/*
 * The fp32 values that n 8-bit moments stand for (checkpoints, inspection):
 * m_out [n], v_out [n].  One launch on `stream`.
 */
int dlm_adamw_read_state(const int8_t* m, const uint8_t* v, const float* m_scale, const float* v_scale, int64_t n,
                         float* m_out, float* v_out, void* stream);

/* ------------------------------------------------------------------- muon */

/* One tensor of a muon step: `count` matrices, one behind the other. */
typedef struct {
    void* p;           /* [count][rows][cols] parameter (p_dtype), updated in place */
    const void* g;     /* gradient (g_dtype), of the same shape */
    float* master;     /* fp32 copy of a bf16 parameter, updated in place (the
                          parameter becomes its rounding), or NULL */
    float* m;          /* momentum, fp32 */
    int64_t count, rows, cols;
    float weight_decay;
    float scale;       /* of the orthogonalised update */
} dlm_muon_param;

#define DLM_MAX_MUON_SIDE 512
#define DLM_MAX_MUON_STEPS 10
typedef struct {
    float lr;
    double momentum;   /* in [0, 1) */
    int32_t nesterov;  /* 0 or 1 */
    float eps;         /* > 0 */
    int32_t steps;     /* 1 .. DLM_MAX_MUON_STEPS */
    double coefs[DLM_MAX_MUON_STEPS][3]; /* a, b, c of every step */
} dlm_muon_cfg;

typedef struct dlm_muon dlm_muon;

/*
 * Register n tensors of matrices (every expert's A and B is one, a router's weight
 * another) that one step of orthogonalised momentum updates together.  Copies the
 * descriptors to the device and allocates a step's scratch memory; the buffers stay
 * owned by the caller, must outlive the handle, and no written one may overlap
 * another.  The smaller side of a matrix is at most DLM_MAX_MUON_SIDE, the other at
 * most 2^30, and a tensor has at most 2^40 elements.  Any sizes and
 * alignments of their element (cols a multiple of 4 and tensors aligned to four
 * elements are faster).
 * The scratch memory, for all tensors at once, by a matrix's smaller side n and longer
 * side d: n up to 16, 32 and 64: 2, 6 and 20 KB for every 512 of d (every 256 where n is
 * above 16 and pieces are few), and 2, 8 and 32 KB; above, with N = n rounded up to a
 * multiple of 64: 4 bytes an element (u), (N / 64 + 1) N bytes for each of d rounded up to
 * a multiple of 256, and 48 N^2 bytes.  A weight of rank 16 so takes 1/4 byte, of rank 128
 * 7, of rank 512 13.
 */
int dlm_muon_create(const dlm_muon_param* params, int32_t n, int32_t p_dtype, int32_t g_dtype, dlm_muon** out);

/* Free the handle's device memory (synchronises the device first). */
int dlm_muon_destroy(dlm_muon* h);

/*
 * One step over every matrix of every tensor, no allocation:
 *   g' = grad_scale g,  m <- beta m + (1 - beta) g',  u = nesterov ? beta m + (1 - beta) g' : m
 *   X = u / (|u| + eps),  then `steps` times  X <- a X + (b A + c A^2) X,  A = X X^T
 *   w <- w (1 - lr wd) - lr scale X
 * with |u| the Frobenius norm, w = the master where there is one, else the parameter;
 * lr = cfg's times *lr_scale.  lr_scale and grad_scale are DEVICE floats or NULL (1): a
 * captured step reads them on every replay.  m and u are fp32; the products are formed
 * on the smaller side in binary64 and X is rounded to fp32 once.
 * Coefficients with |a| above 1 raise weak directions, and the rounding of A in them, by
 * a^2 a step: with five steps of (3.4445, -4.775, 2.0315) X is off by less than its own
 * rounding, with ten by 1e-4 in directions below 1e-5 of the strongest.
 * A matrix whose u is not finite, or whose X coefficients drive out of fp32's range, is left
 * unchanged, momentum too, and the error word is set.  Bitwise reproducible.
 * Launches: three for the matrices with a smaller side up to 16, three up to 32, three
 * up to 64 (three for all of these where they are few), and 3 + 3 steps for those above.
 */
int dlm_muon_step(dlm_muon* h, const dlm_muon_cfg* cfg, const float* lr_scale, const float* grad_scale, void* stream);

/*
 * Synchronise `stream`, then read and clear the error word: *code (host) = DLM_OK or
 * DLM_EDEVICE (some matrix was not finite).
 */
int dlm_muon_status(dlm_muon* h, int32_t* code, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DLM_H */
