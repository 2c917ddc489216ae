/*
 * lrmoe.h -- C ABI of the MI355X (gfx950) pruned MoE expert backward.
 *
 * The library implements, for the experts local to one GPU, the backward of
 * one expert projection y = W_e phi under LRMoE's pruning:
 *
 *   1. quota     q_e pairs kept per expert, fixed before the backward
 *                ("LRMoE: Trimming Backward Work in Memory-Bound MoE Training",
 *                section "Backward demand is not a constant").
 *   2. score     R_u = alpha_u^2 * ||g_t||^2 * ||phi_u||^2 for each routed pair
 *                u = (t, e) (same article, section "LRM: a decomposable
 *                contribution score").
 *   3. select    per expert, the q_e pairs with the highest R_u
 *                ("LRMoE poda a passagem reversa do MoE ...", bullet on
 *                selection by the LRM metric).
 *   4. compact   kept g rows, phi rows and alpha packed into contiguous,
 *                expert-segmented, unpadded buffers (English article, section
 *                "The part that is easy to get wrong"; Portuguese write-up,
 *                bullet on physical compaction).
 *   5. GEMMs     dW_e = sum_kept (alpha_u g_t) phi_u^T and
 *                dphi_u = alpha_u W_e^T g_t, written back to the original pair
 *                layout (English article, "LRM: ..." for the per-pair outer
 *                product; Portuguese write-up, compaction bullet, for the
 *                return to the original layout).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Pairs are expert-sorted: pairs [off_e, off_e + n_e) belong to local
 *    expert e, off_e = n_0 + ... + n_{e-1}.  Pair index u is the row of phi.
 *  - Tensors are dense row-major.  g is [T, d_out], phi is [P, d_in], W is
 *    [E, d_out, d_in] (W_e maps phi in R^d_in to y in R^d_out), dW is
 *    [E, d_out, d_in] float32, dphi is [P, d_in] float32.
 *  - Storage type of g, phi, W and of the compacted g_c, phi_c is given by
 *    lrmoe_problem.dtype (bfloat16 or float32).  Arithmetic is float32
 *    (bf16 matrix cores with float32 accumulation for the GEMMs).
 *  - Counts and quotas are HOST arrays, read during the call only.  Every
 *    other pointer is a DEVICE pointer, used asynchronously in the order of
 *    `stream` (a hipStream_t; NULL means the null stream).  The caller owns
 *    all memory; the library allocates nothing and keeps no state between
 *    calls, so calls on different streams may run concurrently if their
 *    buffers are disjoint.  Outputs must not alias inputs.
 *  - Device pointers must be 16-byte aligned.  d_out and d_in must be
 *    multiples of 8 (bf16) or 4 (float32).
 *  - Row indices are a precondition the host cannot check (they live in
 *    device memory): 0 <= g_row_index[u] < T and 0 <= phi_row_index[u] <
 *    T_phi.  The kernels still bound every index they read, so a violation
 *    does not fault: a g or phi row whose index is out of range reads as a
 *    row of zeros (score 0, zero compacted row), and a perm entry outside
 *    0..P-1 is skipped.  A call that reads g rows for P > 0 pairs needs
 *    T >= 1 (LRMOE_ERR_SHAPE otherwise), and one that reads phi through a
 *    row index for M > 0 kept pairs needs 1 <= T_phi < 2^31.
 *  - Errors: every host-detectable problem is reported before anything is
 *    launched, and no entry point aborts or prints.  A failed kernel launch
 *    returns LRMOE_ERR_HIP; faults inside kernels surface at the caller's
 *    next synchronisation.
 */
#ifndef LRMOE_H
#define LRMOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LRMOE_ABI_VERSION 6
#define LRMOE_MAX_EXPERTS 256

typedef enum {
  LRMOE_OK = 0,
  LRMOE_ERR_NULL = 1,      /* a required pointer is NULL                     */
  LRMOE_ERR_INVALID = 2,   /* bad expert count, quota or policy              */
  LRMOE_ERR_SHAPE = 3,     /* sizes inconsistent or out of range             */
  LRMOE_ERR_ALIGN = 4,     /* pointer or row length misaligned               */
  LRMOE_ERR_DTYPE = 5,     /* unknown storage type                           */
  LRMOE_ERR_WORKSPACE = 6, /* workspace smaller than lrmoe_workspace_size    */
  LRMOE_ERR_HIP = 7,       /* a HIP runtime call or launch failed            */
  LRMOE_ERR_SCRATCH = 8    /* more scratch than the static buffer holds
                              (lrmoe_score_select_compact_noalloc)           */
} lrmoe_status;

typedef enum { LRMOE_F32 = 0, LRMOE_BF16 = 1 } lrmoe_dtype;

typedef enum {
  /* keep floor(n_e * num / den) pairs of every expert (C-level Cx is
   * num/den = (100 - x)/100; C0 keeps everything)                          */
  LRMOE_QUOTA_RATIO = 0,
  /* a fixed number of pairs for the layer call, shared in proportion to
   * demand: q_e = min(n_e, floor(n_e * budget_pairs / P))                  */
  LRMOE_QUOTA_BUDGET = 1
} lrmoe_quota_mode;

typedef struct {
  int32_t mode;          /* lrmoe_quota_mode                                */
  int64_t num, den;      /* RATIO: 0 <= num <= den, den > 0                 */
  int64_t budget_pairs;  /* BUDGET: >= 0                                    */
} lrmoe_quota_policy;

/* How the GEMMs fold alpha into the weight gradient.  alpha multiplies the
 * reduction index of dW_e = sum_j (alpha_j g_j) phi_j^T, so it enters an
 * operand before the matrix cores (the narrower of g and phi carries it).
 * EXACT (0): alpha*x is split into a bf16 high part and a bf16 residual and
 *   both are multiplied (two matrix-core passes for dW), so dW carries
 *   float32-level error (about 2^-16 relative per term).
 * BF16 (1): alpha*x is rounded once to bf16 (the rounding a bf16 training
 *   step applies); one pass, up to 2^-8 relative per term.
 * F16 (2): one pass on float16 matrix cores (the same rate as bf16): the
 *   other operand converts from bf16 exactly, alpha*x is rounded once to
 *   float16 (2^-11 relative per term, eight times finer than bf16).  Both
 *   are scaled per expert by powers of two taken from the largest row norm
 *   over the expert's kept rows (a bound of the largest magnitude), so any
 *   bf16 range maps into float16's; the product is unscaled exactly.  bf16
 *   storage only (float32 storage uses EXACT).
 * dphi always applies alpha in float32 after the product.  float32 storage
 * always splits both operands (three bf16 passes). */
typedef enum { LRMOE_DW_EXACT = 0, LRMOE_DW_BF16 = 1, LRMOE_DW_F16 = 2 } lrmoe_dw_mode;

/* Scoring rule of lrmoe_score_select_compact.  LRM is the method's metric
 * R_u = alpha_u^2 * ||g_t||^2 * ||phi_u||^2.  The others are the ablation
 * baselines the pages compare it with ("LRMoE: Trimming Backward Work in
 * Memory-Bound MoE Training", section "What the measurements show"): the
 * squared norm of the upstream gradient alone, ||g_t||^2, and its absolute
 * magnitude, read here as the L1 norm sum_i |g_t,i| (the Euclidean norm
 * would rank pairs exactly like the squared norm).  Random dropping, the
 * third baseline, takes caller-drawn scores through lrmoe_select_compact.
 * The gradient-only rules read no phi row.  Sums are float32. */
typedef enum {
  LRMOE_SCORE_LRM = 0,
  LRMOE_SCORE_GRAD_SQNORM = 1,
  LRMOE_SCORE_GRAD_L1 = 2
} lrmoe_score_mode;

typedef struct {
  int32_t E;               /* local experts, 1 .. LRMOE_MAX_EXPERTS          */
  int32_t dtype;           /* lrmoe_dtype                                    */
  int64_t P;               /* routed pairs, 0 <= P < 2^31                     */
  int64_t T;               /* rows of g (T == P when every pair has its row) */
  int32_t d_out;           /* length of g rows = rows of W_e                 */
  int32_t d_in;            /* length of phi rows = columns of W_e            */
  const int64_t* counts;   /* host [E]: n_e, sum = P                          */
  const int64_t* quotas;   /* host [E]: q_e, 0 <= q_e <= n_e                  */
  int32_t dw_mode;         /* lrmoe_dw_mode                                  */
  int32_t score_mode;      /* lrmoe_score_mode (0 = LRM)                     */
  int64_t T_phi;           /* rows of phi when a phi_row_index is passed
                              (lrmoe_gather_compact, lrmoe_gather_backward);
                              ignored otherwise, where phi has P rows        */
} lrmoe_problem;

/* ABI version of the loaded library (LRMOE_ABI_VERSION at build time). */
int32_t lrmoe_abi_version(void);

/* Static English text for a status code (never NULL). */
const char* lrmoe_status_string(lrmoe_status s);

/* Step 1 (host only, no GPU): quotas_out[e] from counts[e] under `policy`.
 * Integer arithmetic, floor rounding, no minimum of one (an expert with one
 * pair at C20 keeps none).  The quota is fixed for the whole layer call.
 * Errors: NULL pointers; E outside 1..LRMOE_MAX_EXPERTS, a negative count or
 * a bad policy -> LRMOE_ERR_INVALID. */
lrmoe_status lrmoe_plan_quota(int32_t E, const int64_t* counts,
                              const lrmoe_quota_policy* policy,
                              int64_t* quotas_out);

/* Step 1 on the device, from the forward's routing instead of host counts
 * (the quota is fixed before the backward from how many pairs reached each
 * expert -- "LRMoE poda a passagem reversa do MoE e acelera o treinamento
 * em 21-45%", bullet "Cotas antes do calculo").
 *   expert_ids   int32 [n_ids] device: local expert index of every routed
 *                pair, any order; an index outside 0..E-1 is not routed and
 *                is counted in *invalid_out instead
 *   counts_out   int64 [E] device: n_e
 *   quotas_out   int64 [E] device: q_e, the same integer rules and results
 *                as lrmoe_plan_quota on counts_out (budget P = sum n_e)
 *   seg_offsets_out int64 [E+1] device: exclusive prefix sum of q_e (the
 *                last entry is M)
 *   invalid_out  int64 [1] device or NULL
 * Asynchronous on `stream`; device pointers 16-byte aligned.  Errors (before
 * any launch): NULL policy or required pointer, misalignment, E outside
 * 1..LRMOE_MAX_EXPERTS or a bad policy (LRMOE_ERR_INVALID), n_ids outside
 * 0..2^31-1 (LRMOE_ERR_SHAPE). */
lrmoe_status lrmoe_plan_quota_device(int32_t E, const int32_t* expert_ids, int64_t n_ids,
                                     const lrmoe_quota_policy* policy, int64_t* counts_out,
                                     int64_t* quotas_out, int64_t* seg_offsets_out,
                                     int64_t* invalid_out, void* stream);

/* Workspace bytes needed by every call of this problem that takes a
 * workspace (one buffer may serve all of them when they run in order on one
 * stream).  Validates the problem like the calls that use it.  The size is
 * returned through bytes_out, so that a bad problem is reported as a status
 * like everywhere else. */
lrmoe_status lrmoe_workspace_size(const lrmoe_problem* pb, size_t* bytes_out);

/* Steps 2-4.  Inputs: alpha f32 [P]; g [T, d_out]; phi [P, d_in];
 * g_row_index int32 [P] gives the g row of each pair (NULL when T == P and
 * pair u uses row u).
 * Outputs (M = sum of quotas, known to the caller from the host quotas):
 *   scores      f32 [P]   R_u (float32 arithmetic, norms summed in float32)
 *   keep        u8  [P]   1 if the pair is kept
 *   seg_offsets i32 [E+1] exclusive prefix sum of the quotas
 *   perm        i32 [M]   original pair index of each compacted row; segments
 *                         in ascending expert order, ascending pair index
 *                         inside a segment
 *   g_c [M, d_out], phi_c [M, d_in], alpha_c f32 [M]: bit-exact copies of the
 *                         kept rows
 *   dphi_zero   f32 [P, d_in] or NULL: rows of dropped pairs are set to 0 (the
 *                         kept rows are left for lrmoe_grouped_backward)
 * Selection: the q_e-th largest score of expert e is the threshold tau_e;
 * every pair above it is kept and pairs equal to it are kept in ascending
 * pair index until q_e pairs are kept.  Scores must be finite. */
lrmoe_status lrmoe_score_select_compact(
    const lrmoe_problem* pb, const int32_t* g_row_index, const float* alpha,
    const void* g, const void* phi, float* scores, uint8_t* keep,
    int32_t* seg_offsets, int32_t* perm, void* g_c, void* phi_c, float* alpha_c,
    float* dphi_zero, void* workspace, size_t ws_bytes, void* stream);

/* lrmoe_score_select_compact for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): no workspace argument.  The selection's scratch -- used when
 * an expert has more than 24576 pairs: three radix-digit histograms and the
 * select state per expert (33 KiB) and two counts per 4096-pair chunk --
 * lives in a static device array of the library, 8 MiB, which every GPU the
 * library runs on holds until the process ends.  Problems that need more
 * (about 240 experts or more, with one of them above 24576 pairs) are
 * rejected with LRMOE_ERR_SCRATCH before anything is launched.  The call allocates nothing; on its first call on a
 * device it looks up that device's copy of the array (the current device,
 * which `stream` must belong to).  Nothing in the scratch needs to start at
 * zero: every call writes what it later reads.  All calls on one GPU share
 * that GPU's array, so calls that overlap in time on one GPU (different
 * streams, or different host threads) race and must not be issued.
 * Arguments, results and other errors as for lrmoe_score_select_compact. */
lrmoe_status lrmoe_score_select_compact_noalloc(
    const lrmoe_problem* pb, const int32_t* g_row_index, const float* alpha,
    const void* g, const void* phi, float* scores, uint8_t* keep,
    int32_t* seg_offsets, int32_t* perm, void* g_c, void* phi_c, float* alpha_c,
    float* dphi_zero, void* stream);

/* Steps 3-4 on caller-provided scores (float32 [P], finite; -0.0 counts as
 * 0.0), for scoring rules other than LRM.  Arguments as above. */
lrmoe_status lrmoe_select_compact(
    const lrmoe_problem* pb, const float* scores, const int32_t* g_row_index,
    const float* alpha, const void* g, const void* phi, uint8_t* keep,
    int32_t* seg_offsets, int32_t* perm, void* g_c, void* phi_c, float* alpha_c,
    float* dphi_zero, void* workspace, size_t ws_bytes, void* stream);

/* Steps 2-3 without compaction: scores, keep flags, seg_offsets and perm as
 * in lrmoe_score_select_compact, no row is moved.  For the zero-masked dense
 * alternative below. */
lrmoe_status lrmoe_score_select(
    const lrmoe_problem* pb, const int32_t* g_row_index, const float* alpha,
    const void* g, const void* phi, float* scores, uint8_t* keep,
    int32_t* seg_offsets, int32_t* perm, void* workspace, size_t ws_bytes,
    void* stream);

/* Zero-masked dense alternative to compaction (what the pages argue against:
 * masking the surplus rows of full-size tensors saves neither time nor
 * memory -- "LRMoE poda a passagem reversa do MoE e acelera o treinamento em
 * 21-45%", the paragraph after the bullets).  alpha_masked f32 [P] = alpha
 * where keep, 0 where dropped; perm_identity int32 [P] (or NULL) = 0..P-1.
 * Running lrmoe_grouped_backward with quotas = counts, perm_identity,
 * alpha_masked and the uncompacted g (one row per pair) and phi yields the
 * same dW and dphi as the compacted path, dropped dphi rows included (0).
 * Errors: NULL / misaligned pointers, P outside 0..2^31-1. */
lrmoe_status lrmoe_mask_alpha(int64_t P, const uint8_t* keep, const float* alpha,
                              float* alpha_masked, int32_t* perm_identity, void* stream);

/* Step 4 alone, for a second projection of the same pairs that inherits an
 * existing keep set (the gate/up projection of the expert MLP: a pair whose
 * down-projection input gradient is zero has zero gate/up gradient, so it is
 * not rescored).  pb describes the second projection (its d_out, d_in, T and
 * dtype; the same counts and quotas); perm and keep come from an earlier
 * lrmoe_score_select_compact.  g_row_index / phi_row_index (int32 [P], or
 * NULL for row u of pair u) pick the source rows of g and phi; the kept
 * rows are copied bit for bit into g_c [M, d_out] and phi_c [M, d_in], alpha
 * into alpha_c [M], and dphi_zero (or NULL) gets zero rows for dropped
 * pairs.  g and g_c may both be NULL: only phi rows and alpha are gathered
 * (the gate/up output gradient of lrmoe_grouped_backward_glu is already
 * compacted). */
lrmoe_status lrmoe_gather_compact(
    const lrmoe_problem* pb, const int32_t* perm, const uint8_t* keep,
    const int32_t* g_row_index, const int32_t* phi_row_index,
    const float* alpha, const void* g, const void* phi, void* g_c,
    void* phi_c, float* alpha_c, float* dphi_zero, void* stream);

/* lrmoe_gather_compact followed by lrmoe_grouped_backward on the same
 * buffers, for a projection on an inherited keep set (the gate/up projection
 * above), in one call.  With bf16 storage the gather also writes the GEMM's
 * operand planes from the rows it moves (as in lrmoe_pruned_backward), bit
 * for bit the separate calls' results.  g and g_c are required here; dphi is
 * both the zero target of dropped rows and the output of kept rows (or
 * NULL); dropped rows of at least 512 MiB in all are cleared inside the
 * grouped GEMM launch, as in lrmoe_pruned_backward.  workspace:
 * lrmoe_workspace_size bytes.  Errors as for the two calls. */
lrmoe_status lrmoe_gather_backward(
    const lrmoe_problem* pb, const int32_t* perm, const uint8_t* keep,
    const int32_t* g_row_index, const int32_t* phi_row_index,
    const float* alpha, const void* g, const void* phi, const void* W,
    void* g_c, void* phi_c, float* alpha_c, float* dW, float* dphi,
    void* workspace, size_t ws_bytes, void* stream);

/* Step 5: variable-length grouped GEMMs over the compacted buffers.
 *   dW   f32 [E, d_out, d_in]: fully overwritten (zero for q_e = 0)
 *   dphi f32 [P, d_in] or NULL: rows perm[j] receive alpha_c[j] W_e^T g_c[j];
 *        other rows are not touched (see dphi_zero above).
 * W is [E, d_out, d_in] in the storage type; segments are given by the host
 * quotas of pb. */
lrmoe_status lrmoe_grouped_backward(
    const lrmoe_problem* pb, const int32_t* perm, const float* alpha_c,
    const void* g_c, const void* phi_c, const void* W, float* dW, float* dphi,
    void* workspace, size_t ws_bytes, void* stream);

/* The expert MLP's activation backward, chained on the compacted layout.
 * The models trained in "What the measurements show" ("LRMoE: Trimming
 * Backward Work in Memory-Bound MoE Training": Qwen3-30B-A3B,
 * GLM4.5-106B-A12B) have gated-MLP experts whose down projection reads
 * phi = SiLU(a) * b, a and b being the saved gate and up pre-activations.
 * The pages do not spell this step out (a reading); they only say that the
 * original layout is restored after the compacted GEMMs ("LRMoE poda a
 * passagem reversa do MoE e acelera o treinamento em 21-45%", compaction
 * bullet), which this entry point postpones past the activation backward.  Same as lrmoe_grouped_backward for dW (the down projection's),
 * but instead of dphi it writes, for every compacted row j (pair
 * u = perm[j] of expert e), with d = W_e^T g_c[j] before the routing weight:
 *   dgu_c[j] = [ d * b_u * SiLU'(a_u)  |  d * SiLU(a_u) ]
 * SiLU'(a) = s (1 + a (1 - s)), s = sigmoid(a), computed in float32.  dgu_c
 * is [M, 2 d_in], gate half first: the gate/up projection's output gradient,
 * already compacted.  Its storage follows pb->dw_mode: float32 (unrounded)
 * unless dw_mode is LRMOE_DW_BF16, where each entry is rounded once to bf16
 * (the single-rounding mode, with that mode's error bound).  The chain ends
 * with lrmoe_gather_compact (g = g_c = NULL) of the gate/up projection's
 * inputs x, then, with the same perm and alpha_c (alpha applied once,
 * there), lrmoe_grouped_backward_gate_up on the float32 dgu_c, or
 * lrmoe_grouped_backward with g_c = dgu_c on the bf16 one.  No
 * original-layout dphi is written and none needs zeroing.
 *   act_a, act_b  bf16 [P, d_in], pair-indexed like phi.
 * act_a, act_b and dgu_c may be NULL when no pair is kept (M = 0).  bf16
 * storage only (LRMOE_ERR_DTYPE otherwise); other errors as for
 * lrmoe_grouped_backward. */
lrmoe_status lrmoe_grouped_backward_glu(
    const lrmoe_problem* pb, const int32_t* perm, const float* alpha_c,
    const void* g_c, const void* phi_c, const void* W, float* dW,
    const void* act_a, const void* act_b, void* dgu_c, void* workspace,
    size_t ws_bytes, void* stream);

/* The gate/up projection's backward at the end of the MLP chain above: the
 * same products as lrmoe_grouped_backward (dW [E, d_out, d_in] of the gate/up
 * weight, dx rows perm[j] of [P, d_in], alpha applied once) with the float32
 * output gradient dgu_c [M, d_out] of lrmoe_grouped_backward_glu (d_out = 2
 * d_in of the down projection) as g_c, and bf16 x_c [M, d_in] and W
 * [E, d_out, d_in].  alpha * dgu_c is split into a bf16 high part and
 * residual (hi only when dw_mode is LRMOE_DW_BF16) that feed both products,
 * so the gradient handed over keeps float32-level precision.  dx may be NULL
 * (dW only).  pb->dtype must be LRMOE_BF16 (LRMOE_ERR_DTYPE otherwise);
 * workspace: lrmoe_workspace_size of pb; other errors as for
 * lrmoe_grouped_backward. */
lrmoe_status lrmoe_grouped_backward_gate_up(
    const lrmoe_problem* pb, const int32_t* perm, const float* alpha_c, const float* dgu_c,
    const void* x_c, const void* W, float* dW, float* dx, void* workspace, size_t ws_bytes,
    void* stream);

/* Steps 2-5 in one call: lrmoe_score_select_compact followed by
 * lrmoe_grouped_backward on the same buffers, with the same arguments and
 * results (dphi is both the zero target of dropped rows and the output of
 * kept rows; NULL for dW only).  With bf16 storage the gather also writes the
 * GEMM's operand planes (alpha times the narrower compacted operand, as bf16
 * hi and, in exact mode, lo) from the rows it moves, so no separate pass
 * reads the compacted operand again; the planes and every result are bit for
 * bit those of the two separate calls.  When the dropped pairs' dphi rows
 * hold at least 512 MiB ((P - M) * d_in * 4 bytes), the grouped GEMM launch
 * clears them beside its tiles instead of the gather (same results).
 * workspace: lrmoe_workspace_size bytes.  Errors as for the two calls. */
lrmoe_status lrmoe_pruned_backward(
    const lrmoe_problem* pb, const int32_t* g_row_index, const float* alpha,
    const void* g, const void* phi, const void* W, float* scores, uint8_t* keep,
    int32_t* seg_offsets, int32_t* perm, void* g_c, void* phi_c, float* alpha_c,
    float* dW, float* dphi, void* workspace, size_t ws_bytes, void* stream);

/* Per-kernel timing.  Each entry point below launches a fixed sequence of
 * kernels; for every non-NULL pair, `before` and `after` (hipEvent_t created
 * by the caller with timing enabled) are recorded on `stream` right before
 * and right after that kernel's launch.  Kernels not launched for a problem
 * (an empty range) leave their events unrecorded.
 *   lrmoe_score_select_compact_timed: [0] score  [1] select+scan  [2] gather
 *   lrmoe_select_compact_timed:       [1] select+scan  [2] gather
 *   lrmoe_grouped_backward_timed,
 *   lrmoe_grouped_backward_glu_timed,
 *   lrmoe_grouped_backward_gate_up_timed:
 *                                     [0] operand prologue  [1] grouped GEMM
 *                                     [2] split-K reduction
 *   lrmoe_pruned_backward_timed:      [0] score  [1] select+scan  [2] gather
 *                                     [3] grouped GEMM  [4] split-K reduction
 *                                     [5] operand prologue (float32 storage)
 *   lrmoe_gather_backward_timed:      [2] gather  [3] grouped GEMM
 *                                     [4] split-K reduction
 *                                     [5] operand prologue (float32 storage) */
#define LRMOE_TIMING_SLOTS 8
typedef struct {
  void* before[LRMOE_TIMING_SLOTS];
  void* after[LRMOE_TIMING_SLOTS];
} lrmoe_timing;

/* lrmoe_score_select_compact with per-kernel events (timing may be NULL). */
lrmoe_status lrmoe_score_select_compact_timed(
    const lrmoe_problem* pb, const int32_t* g_row_index, const float* alpha,
    const void* g, const void* phi, float* scores, uint8_t* keep,
    int32_t* seg_offsets, int32_t* perm, void* g_c, void* phi_c, float* alpha_c,
    float* dphi_zero, void* workspace, size_t ws_bytes, void* stream,
    const lrmoe_timing* timing);

/* lrmoe_select_compact with per-kernel events (timing may be NULL). */
lrmoe_status lrmoe_select_compact_timed(
    const lrmoe_problem* pb, const float* scores, const int32_t* g_row_index,
    const float* alpha, const void* g, const void* phi, uint8_t* keep,
    int32_t* seg_offsets, int32_t* perm, void* g_c, void* phi_c, float* alpha_c,
    float* dphi_zero, void* workspace, size_t ws_bytes, void* stream,
    const lrmoe_timing* timing);

/* lrmoe_grouped_backward with per-kernel events (timing may be NULL). */
lrmoe_status lrmoe_grouped_backward_timed(
    const lrmoe_problem* pb, const int32_t* perm, const float* alpha_c,
    const void* g_c, const void* phi_c, const void* W, float* dW, float* dphi,
    void* workspace, size_t ws_bytes, void* stream, const lrmoe_timing* timing);

/* lrmoe_pruned_backward with per-kernel events (timing may be NULL). */
lrmoe_status lrmoe_pruned_backward_timed(
    const lrmoe_problem* pb, const int32_t* g_row_index, const float* alpha,
    const void* g, const void* phi, const void* W, float* scores, uint8_t* keep,
    int32_t* seg_offsets, int32_t* perm, void* g_c, void* phi_c, float* alpha_c,
    float* dW, float* dphi, void* workspace, size_t ws_bytes, void* stream,
    const lrmoe_timing* timing);

/* lrmoe_gather_backward with per-kernel events (timing may be NULL). */
lrmoe_status lrmoe_gather_backward_timed(
    const lrmoe_problem* pb, const int32_t* perm, const uint8_t* keep,
    const int32_t* g_row_index, const int32_t* phi_row_index,
    const float* alpha, const void* g, const void* phi, const void* W,
    void* g_c, void* phi_c, float* alpha_c, float* dW, float* dphi,
    void* workspace, size_t ws_bytes, void* stream, const lrmoe_timing* timing);

/* lrmoe_grouped_backward_glu with per-kernel events (timing may be NULL). */
lrmoe_status lrmoe_grouped_backward_glu_timed(
    const lrmoe_problem* pb, const int32_t* perm, const float* alpha_c,
    const void* g_c, const void* phi_c, const void* W, float* dW,
    const void* act_a, const void* act_b, void* dgu_c, void* workspace,
    size_t ws_bytes, void* stream, const lrmoe_timing* timing);

/* lrmoe_grouped_backward_gate_up with per-kernel events (timing may be NULL). */
lrmoe_status lrmoe_grouped_backward_gate_up_timed(
    const lrmoe_problem* pb, const int32_t* perm, const float* alpha_c, const float* dgu_c,
    const void* x_c, const void* W, float* dW, float* dx, void* workspace, size_t ws_bytes,
    void* stream, const lrmoe_timing* timing);

/* ------------------------------------------------------------------------
 * The forward side: what produces the pairs, projection inputs and
 * pre-activations that the backward above reads, and the gradients of the
 * steps around it.
 *
 *   gate      router logits -> expert ids and weights of each token
 *   sort      ids -> pairs in expert order (counts, segments, rows, alpha)
 *   dispatch  token rows -> pair rows          (gradient: sum over a token)
 *   product   z_u = W_e x_u + bias, y_u = act(z_u) + residual, per expert
 *                                              (gradient of the epilogue; the
 *             product's own is lrmoe_grouped_backward with quotas = counts)
 *   combine   pair rows -> weighted token rows (gradient: rows and weights)
 *
 * The rules above hold here too (dense row-major, device pointers 16-byte
 * aligned, row lengths multiples of 8 (bf16) or 4 (float32), outputs not
 * aliasing inputs, nothing allocated, errors before any launch).  Expert
 * counts and segments stay on the device: nothing visits the host between
 * these calls, so a layer's forward and the gradients declared here can be
 * captured in a graph.  (The products' gradients take counts and quotas from
 * the host, as all of the pruned backward does.)  A graph that is replayed
 * beside other calls needs a workspace of its own.
 *
 * The gate's ids are those of the whole router row.  A rank that holds experts
 * first .. first + n - 1 sorts ids - first with E = n: ids below 0 or from n
 * on belong to other ranks.
 * ------------------------------------------------------------------------ */

#define LRMOE_MAX_GATE_EXPERTS 1024 /* experts of a router row               */
#define LRMOE_MAX_TOPK 64           /* slots of a token                      */

typedef enum { LRMOE_GATE_SOFTMAX = 0, LRMOE_GATE_SIGMOID = 1 } lrmoe_gate_score;

typedef struct {
  int64_t T;       /* tokens, T * K < 2^31                                   */
  int32_t E;       /* experts of a row, 1 .. LRMOE_MAX_GATE_EXPERTS          */
  int32_t K;       /* slots, 1 .. min(E, LRMOE_MAX_TOPK)                     */
  int32_t dtype;   /* lrmoe_dtype of the logits                              */
  int32_t score;   /* lrmoe_gate_score                                       */
  int32_t renorm;  /* non-zero: weights of the chosen experts sum to scale   */
  float scale;     /* factor on every weight                                 */
} lrmoe_gate;

/* Top-k gate.  logits [T, E] (any E: a row need not be 16-byte aligned).
 * Selection key of expert e: its logit x_e, or with select_bias (float32 [E],
 * sigmoid score only, else LRMOE_ERR_INVALID) sigmoid(x_e) + select_bias[e]
 * in float64.  The K largest keys, best first, ties to the lower expert:
 *   ids      int32 [T, K]
 *   weights  float32 [T, K]: scale * the score of the chosen experts, softmax
 *            over the row (SOFTMAX) or sigmoid (SIGMOID); with renorm
 *            normalised over the chosen ones instead.  The bias enters the
 *            selection only.
 * A logit of -inf or NaN masks its expert (+inf counts as the largest finite
 * value); so does a NaN or -inf key.  Where fewer than K experts are left,
 * the last slots hold id -1 and weight 0. */
lrmoe_status lrmoe_gate_topk(const lrmoe_gate* gt, const void* logits, const float* select_bias,
                             int32_t* ids, float* weights, void* stream);

/* Gradient of the gate's weights: dlogits [T, E] in the logits' type, fully
 * overwritten, from dweights float32 [T, K] at the ids of lrmoe_gate_topk (or
 * any others: a slot with an id outside 0..E-1 carries nothing, and an
 * expert standing in two slots gets the sum of both).  The selection itself
 * has no gradient. */
lrmoe_status lrmoe_gate_topk_backward(const lrmoe_gate* gt, const void* logits,
                                      const int32_t* ids, const float* dweights, void* dlogits,
                                      void* stream);

/* Workspace bytes of lrmoe_route_sort (0 for few pairs). */
lrmoe_status lrmoe_route_sort_workspace(int64_t T, int32_t K, int32_t E, size_t* bytes_out);

/* Stable sort of the T * K slots by expert.  ids int32 [T, K], local expert
 * indices; a slot whose id is outside 0..E-1 is routed elsewhere.  With P
 * the slots routed here (= seg_offsets[E], known on the device only):
 *   counts       int64 [E]
 *   seg_offsets  int32 [E + 1]
 *   row_index    int32 [T * K]: token of each pair in expert order, pairs of
 *                one expert in ascending slot order; -1 behind the last pair
 *   pos          int32 [T, K]: each slot's place in that order, -1 elsewhere
 *   alpha        float32 [T * K] or NULL: weights (float32 [T, K]) in that
 *                order, 0 behind the last pair
 * T * K < 2^31; E <= LRMOE_MAX_EXPERTS; K <= LRMOE_MAX_TOPK. */
lrmoe_status lrmoe_route_sort(int64_t T, int32_t K, int32_t E, const int32_t* ids,
                              const float* weights, int64_t* counts, int32_t* seg_offsets,
                              int32_t* row_index, int32_t* pos, float* alpha, void* workspace,
                              size_t ws_bytes, void* stream);

/* xp[pos[t, k]] = x[t]: x [T, D], xp [P, D] of one type.  P is the capacity
 * of xp: a place outside 0..P-1 is skipped, and rows no slot names are left
 * as they were.  Two slots must not share a place.  (lrmoe_grouped_forward
 * can read x through row_index instead, without this copy.) */
lrmoe_status lrmoe_dispatch(int32_t dtype, int64_t T, int32_t K, int32_t D, int64_t P,
                            const void* x, const int32_t* pos, void* xp, void* stream);

/* dx[t] = sum_k dxp[pos[t, k]] (float32 sum in ascending k, one rounding):
 * dxp [P, D] of type dtype (float32 for lrmoe_grouped_backward's dphi), dx
 * [T, D] of type out_dtype, fully overwritten. */
lrmoe_status lrmoe_dispatch_backward(int32_t dtype, int32_t out_dtype, int64_t T, int32_t K,
                                     int32_t D, int64_t P, const void* dxp, const int32_t* pos,
                                     void* dx, void* stream);

/* y[t] = residual[t] + sum_k weights[t, k] * yp[pos[t, k]] (float32, one
 * rounding): yp [P, D], y [T, D], residual [T, D] or NULL, of one type;
 * weights float32 [T, K].  A token without a place gets its residual, or 0. */
lrmoe_status lrmoe_combine(int32_t dtype, int64_t T, int32_t K, int32_t D, int64_t P,
                           const void* yp, const int32_t* pos, const float* weights,
                           const void* residual, void* y, void* stream);

/* Gradient of lrmoe_combine from dy [T, D]: dyp[pos[t, k]] = weights[t, k] *
 * dy[t] ([P, D]; rows no slot names are left as they were) and dweights
 * float32 [T, K] = <dy[t], yp[pos[t, k]]> (0 without a place).  (The
 * residual's gradient is dy.)  Two slots must not share a place. */
lrmoe_status lrmoe_combine_backward(int32_t dtype, int64_t T, int32_t K, int32_t D, int64_t P,
                                    const void* dy, const void* yp, const int32_t* pos,
                                    const float* weights, void* dyp, float* dweights,
                                    void* stream);

/* Activation of the grouped product's epilogue.  GELU is the exact one (with
 * the error function).  SWIGLU: the first half of W_e's rows gives the gate
 * a, the second half b; y = SiLU(a) * b. */
typedef enum {
  LRMOE_ACT_NONE = 0,
  LRMOE_ACT_RELU = 1,
  LRMOE_ACT_SILU = 2,
  LRMOE_ACT_GELU = 3,
  LRMOE_ACT_SWIGLU = 4
} lrmoe_act;

typedef struct {
  int32_t E;      /* experts, 1 .. LRMOE_MAX_EXPERTS                         */
  int32_t dtype;  /* storage of x, W, bias, residual, y and pre-activations  */
  int64_t P;      /* pair rows (capacity), 0 <= P < 2^31                     */
  int64_t T;      /* rows of x (T == P without a row_index)                  */
  int32_t d_out;  /* rows of W_e (2 F for SWIGLU)                            */
  int32_t d_in;   /* columns of W_e                                          */
  int32_t act;    /* lrmoe_act                                               */
} lrmoe_forward;

/* y_u = act(W_e x_{row(u)} + bias_e) + residual_u for the pairs u of expert
 * e, seg_offsets[e] <= u < seg_offsets[e + 1] (device int32 [E + 1],
 * ascending, at most P; rows behind the last segment are left as they were).
 * F = d_out, or d_out / 2 for SWIGLU.
 *   row_index  int32 [P] device or NULL (row u): an index outside 0..T-1
 *              reads a zero row
 *   x [T, d_in], W [E, d_out, d_in], bias [E, d_out] or NULL,
 *   residual [P, F] or NULL, y [P, F]
 *   pre_a [P, F] (and pre_b, both or none, for SWIGLU): W x + bias before the
 *              activation, in the layout lrmoe_act_backward and
 *              lrmoe_grouped_backward_glu read; NULL: not stored
 * One segment (E = 1) is the dense product of a shared expert.  float32
 * accumulation and epilogue, one rounding; float32 storage multiplies in
 * float32. */
lrmoe_status lrmoe_grouped_forward(const lrmoe_forward* fw, const int32_t* seg_offsets,
                                   const int32_t* row_index, const void* x, const void* W,
                                   const void* bias, const void* residual, void* y, void* pre_a,
                                   void* pre_b, void* stream);

/* Workspace bytes of lrmoe_act_backward when dbias is asked for. */
lrmoe_status lrmoe_act_backward_workspace(const lrmoe_forward* fw, size_t* bytes_out);

/* Gradient of the epilogue, from dy [P, F]:
 *   dz     [P, d_out] of type dz_dtype (the storage type, or float32 for the
 *          unrounded hand-off to lrmoe_grouped_backward_gate_up): dy act'(a),
 *          for SWIGLU [dy b SiLU'(a) | dy SiLU(a)]; rows behind the last
 *          segment are left as they were
 *   dbias  float32 [E, d_out] or NULL: sum of the unrounded dz over the
 *          expert's rows (0 without rows), in an order that does not depend
 *          on timing
 * pre_a (and pre_b for SWIGLU) as stored by lrmoe_grouped_forward; pre_a is
 * not read for LRMOE_ACT_NONE.  The residual's gradient is dy.  fw's T and
 * d_in are checked but not used.  workspace: NULL without dbias. */
lrmoe_status lrmoe_act_backward(const lrmoe_forward* fw, int32_t dz_dtype,
                                const int32_t* seg_offsets, const void* dy, const void* pre_a,
                                const void* pre_b, void* dz, float* dbias, void* workspace,
                                size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * 8-bit expert products.  Values in e4m3 (finite up to 448), one power-of-two
 * scale 2^(byte - 127) for each block of 128: the smallest one with the block's
 * largest magnitude at most 448 * scale, from 2^-126 on (1 for a block of zeros).
 * Rows have blocks of 1 x 128, weights of 128 x 128; the last block of a row, column or
 * weight may be smaller.  A row of scales has ceil(columns / 128) bytes, padded with 127
 * to a multiple of four:
 *   S(d) = 4 * ceil(ceil(d / 128) / 4)
 * Infinity and NaN become the NaN code and do not count in their block's scale.
 * Rows in 8 bits are whole 16-byte pieces: their lengths are multiples of 16.
 *
 * Gradients: dx of a product is the product of the quantised dz with the
 * transposed weights (qt, scale_t), through lrmoe_grouped_forward_quantized; dW is
 * lrmoe_grouped_backward on the unrounded rows.
 * ------------------------------------------------------------------------ */

/* Rows to 8 bits: x [T, D] of type dtype, q uint8 (e4m3) [T, D], scale uint8
 * [T, S(D)].  0 <= T < 2^31, D a multiple of 16. */
lrmoe_status lrmoe_quantize_rows(int32_t dtype, int64_t T, int32_t D, const void* x, uint8_t* q,
                                uint8_t* scale, void* stream);

/* Weights to 8 bits: W [E, d_out, d_in] of type dtype, q uint8 [E, d_out, d_in],
 * scale uint8 [E, ceil(d_out / 128), S(d_in)]; and, unless qt and scale_t are NULL
 * (both or neither), the same values and scales transposed: qt [E, d_in, d_out],
 * scale_t [E, ceil(d_in / 128), S(d_out)].  d_in a multiple of 16, d_out of 8
 * (with qt: of 16). */
lrmoe_status lrmoe_quantize_weights(int32_t dtype, int32_t E, int32_t d_out, int32_t d_in,
                                        const void* W, uint8_t* q, uint8_t* scale, uint8_t* qt,
                                        uint8_t* scale_t, void* stream);

/* lrmoe_grouped_forward with x and W in 8 bits: xq [T, d_in], x_scale [T, S(d_in)], Wq
 * [E, d_out, d_in], W_scale [E, ceil(d_out / 128), S(d_in)].  Everything else is as
 * there; fw->dtype, the type of bias, residual, y, pre_a and pre_b, is LRMOE_BF16
 * (else LRMOE_ERR_DTYPE), and d_in a multiple of 16.  float32 accumulation and
 * epilogue, one rounding; of each run of 8 products the matrix instruction drops what
 * lies below 2^-13 of the largest. */
lrmoe_status lrmoe_grouped_forward_quantized(const lrmoe_forward* fw, const int32_t* seg_offsets,
                                       const int32_t* row_index, const uint8_t* xq,
                                       const uint8_t* x_scale, const uint8_t* Wq,
                                       const uint8_t* W_scale, const void* bias,
                                       const void* residual, void* y, void* pre_a, void* pre_b,
                                       void* stream);

/* ------------------------------------------------------------------------
 * The norms around a block, with its gate and residual scale:
 *   b_t = y_t                              without branch_weight
 *         y_t * rms(y_t) * branch_weight   with it;  rms(v) = (mean(v^2) + eps)^-1/2
 *   s_t = scale * x_t + gate * b_t
 *   h_t = s_t * rms(s_t) * weight
 * s is the residual stream behind the block whose output is y, h the next
 * block's input.  float32 sums and statistics; h is computed from s before its
 * rounding; each output is rounded once.
 * ------------------------------------------------------------------------ */

/* columns of a row; the gradient of more than 8192 takes 3.5 to 4.3 times as long as its
 * bytes */
#define LRMOE_MAX_NORM_WIDTH 16384

typedef enum {
  LRMOE_BRANCH_GATE_NONE = 0,    /* 1                                        */
  LRMOE_BRANCH_GATE_CHANNEL = 1, /* one factor a column, [D] of type dtype   */
  LRMOE_BRANCH_GATE_TOKEN = 2    /* one factor a row, float32 [T]            */
} lrmoe_branch_gate;

typedef struct {
  int64_t T;      /* rows, 0 <= T < 2^31                                     */
  int32_t D;      /* columns, at most LRMOE_MAX_NORM_WIDTH, whole 16 bytes   */
  int32_t dtype;  /* of x, y, s, h, their gradients and the weights          */
  int32_t gate;   /* lrmoe_branch_gate                                       */
  float scale;    /* factor of the residual                                  */
  float eps;      /* at least 0                                              */
} lrmoe_norm;

/* x, y, s, h [T, D]; branch_weight, weight [D].  y NULL: no branch; then
 * branch_weight, gate and s have to be NULL, scale 1 (else LRMOE_ERR_INVALID), and
 * s_t is x_t.  weight and h go together (both or neither: LRMOE_ERR_NULL), and so do
 * gate and its kind; with y, s is needed. */
lrmoe_status lrmoe_residual_norm(const lrmoe_norm* nm, const void* x, const void* y,
                                 const void* branch_weight, const void* gate, const void* weight,
                                 void* s, void* h, void* stream);

/* Workspace bytes of lrmoe_residual_norm_backward. */
lrmoe_status lrmoe_residual_norm_backward_workspace(const lrmoe_norm* nm, size_t* bytes_out);

/* Gradient, at the stored s (x itself without a branch; not read without weight) and
 * y, from ds [T, D] (NULL: nothing arrives at s but through h) and dh [T, D] (with
 * weight and only then):
 *   dx [T, D], dy [T, D] (with y and only then)
 *   dweight, dbranch_weight float32 [D] (with the weights) or NULL: not computed
 *   dgate float32 [D] or [T] (with the gate) or NULL: not computed
 * Sums over rows do not depend on timing.  workspace: not read when only dx, dy and
 * a token's dgate are asked for (then NULL will do). */
lrmoe_status lrmoe_residual_norm_backward(const lrmoe_norm* nm, const void* ds, const void* dh,
                                          const void* s, const void* y, const void* branch_weight,
                                          const void* gate, const void* weight, void* dx, void* dy,
                                          float* dweight, float* dbranch_weight, float* dgate,
                                          void* workspace, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * AdamW over many tensors in one call (one launch for each 48 tensors of the
 * same types), in place:
 *   g' = grad_scale * g
 *   m  = beta1 m + (1 - beta1) g'         v = beta2 v + (1 - beta2) g'^2
 *   p  = (1 - lr * weight_decay) p
 *        - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * in float32.  The states are float32 [n], or 8-bit: e4m3 [n] with a scale byte
 * for each run of 128 elements (the blocks of the products above), m itself and,
 * in v's place, sqrt(v).  p is updated from the unrounded m and v.  8-bit states
 * and bfloat16 parameters are rounded stochastically: up with a probability of
 * the distance from the lower neighbour (in 65536ths), so that small changes are
 * not lost on average; a second moment that is not zero is not rounded to zero.
 * So m and the root keep their means, and v, the root's square, gains the rounding's
 * variance: it is 2.6 % (beta2 0.95) to 4.3 % (0.999) high on average where the root is
 * within 2^-14 of its block's largest, and nine in ten elements are between 0.65 and 1.6
 * times the exact v at any one step.  From 2^-16 to 2^-18 of the largest, v is 1.8 to 1.9
 * times the exact one, and a root further below is held at the smallest code, 2^-9 of the
 * scale: those elements take smaller steps.  Tensors whose neighbouring elements' gradients
 * differ by more than that want float32 states.
 * The random bits of element i of tensor k are a hash of (seed, step, k, i):
 *   mix(a): a ^= a >> 16; a *= 0x6A09E667; a ^= a >> 15; a *= 0xBB67AE85;
 *           a ^= a >> 16                                        (32 bits)
 *   key = mix(mix(seed + step * 0x9E3779B9) + (k + 1) * 0x3C6EF373)
 *   r   = mix((i mod 2^32) + key)
 * r's upper half rounds m, its lower half sqrt(v), the upper half of
 * mix(r + 0xA54FF53B) a bfloat16 p.
 * ------------------------------------------------------------------------ */

typedef struct {
  int64_t n;         /* elements, 0 <= n < 2^36 (0: skipped)                 */
  void* p;           /* parameter [n], updated                               */
  const void* g;     /* gradient [n]                                         */
  void* m;           /* first moment [n], updated                            */
  void* v;           /* second moment (8-bit: its root) [n], updated         */
  uint8_t* m_scale;  /* 8-bit states: [ceil(n / 128)], updated; else NULL    */
  uint8_t* v_scale;  /* with m_scale, both or neither                        */
  void* copy;        /* bfloat16 [n] or NULL: p rounded to nearest; p float32 */
  int32_t p_dtype;   /* lrmoe_dtype of p                                     */
  int32_t g_dtype;   /* lrmoe_dtype of g                                     */
} lrmoe_adamw_tensor;

typedef struct {
  double lr, beta1, beta2, eps, weight_decay; /* 0 <= beta < 1, the others >= 0 */
  int64_t step;            /* from 1 on                                      */
  uint32_t seed;           /* of the stochastic rounding                     */
  const float* lr_at;      /* device float32 or NULL: in lr's place          */
  const int64_t* step_at;  /* device int64 or NULL: in step's place (from 1 on) */
  const float* grad_scale; /* device float32 or NULL (1)                     */
  const float* skip;       /* device float32 or NULL: nothing is changed if not 0 */
} lrmoe_adamw;

/* tensors: host array of count descriptors (read before the call returns), k their
 * index in it; device pointers 16-byte aligned except the four scalars (their own
 * size).  A captured call replays with the descriptors and host scalars of its
 * capture: lr_at and step_at are for that.  No two buffers may overlap. */
lrmoe_status lrmoe_adamw_step(const lrmoe_adamw* cfg, const lrmoe_adamw_tensor* tensors,
                              int32_t count, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* LRMOE_H */
