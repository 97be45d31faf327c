/*
 * fa_gb300.h -- C ABI of the GB300 (sm_103a) attention forward library.
 *
 * The FlashAttention forward pass over packed variable-length sequences and a
 * paged KV cache, with per-row log-sum-exp output, its backward pass, and the
 * operators of a serving loop around the paged decode (shared prefixes, key
 * weights, eviction).  The forward:  For query row i of sequence b and head h:
 *
 *   out[i]  = sum_j softmax_j(s_ij) * v_j        over the keys j the mask allows
 *   lse[i]  = log sum_j exp(s_ij)                (natural log)
 *   s_ij    = scale * <q_i, k_j>, then soft-cap, then ALiBi
 *
 * The passages that define it:
 *  - tiled QK^T, online (running max / running sum) softmax, PV and the
 *    attention-domain LSE = M + log(L) over packed cu_seqlens tensors
 *    [total_tokens, H, D]: RL-Kernel PR #237 "SM90 TMA + mma.sync
 *    FlashAttention", commit texts and summary;
 *  - the LSE written also for fully masked rows, and the split-K combine
 *    m_max*ln2 + ln(den): FlyDSL PR #844 "Add forward LSE output", Changes;
 *  - paged KV addressed through block_table, FP8 e4m3 KV with scales,
 *    Q/K head dim 192 with V/O 128 at native BF16 width, bottom-right causal
 *    mask, offsets above 4 GiB: FlyDSL PR #1066 "Support paged FP8 Flash
 *    attention with asymmetric K/V head dim", overview, review and PR
 *    description;
 *  - per-token fp8 scale max|row|/448, ALiBi, SoftCap, SlidingWindow and
 *    128x128 block sparsity: fkl_python PR #7 "flash_attention: prologue
 *    fusion, mma tensor cores, fp8 KV cache, flex attention + block
 *    sparsity", commits and summary.
 *
 * Conventions for every entry point:
 *  - Pointers inside fa_tensor_t are DEVICE pointers on the current CUDA
 *    device, owned by the caller.  The library never frees them and keeps no
 *    reference after the call returns.
 *  - Calls are asynchronous: work is enqueued on `stream` (a cudaStream_t
 *    passed as void*, NULL = legacy default stream) and the call returns.
 *    The library performs no host<->device copy, no device synchronisation
 *    and no memory allocation inside fa_fwd_varlen / fa_combine.
 *  - All validation happens on the host before any launch, using the shapes
 *    in fa_tensor_t and the host scalars in fa_launch_t.  On any non-OK
 *    status nothing has been enqueued; fa_last_error() describes the cause.
 *  - Device-side waits are bounded.  A wait that runs out, or an index that
 *    the kernel finds out of range, records a code in a per-device error word
 *    read by fa_get_device_error(); the kernel then returns early.
 */
#ifndef FA_GB300_H
#define FA_GB300_H

#include <stddef.h>
#include <stdint.h>

/* Every entry point below is exported; the library is built with hidden
 * visibility for everything else (kernels, templates, helpers), so that two
 * copies loaded into one process do not bind to each other's internals. */
#if defined(__GNUC__)
#define FA_API __attribute__((visibility("default")))
#else
#define FA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FA_OK = 0,
    FA_ERR_INVALID_ARG = 1,    /* malformed shape, dtype, stride or pointer */
    FA_ERR_UNSUPPORTED = 2,    /* valid request outside the compiled variant set */
    FA_ERR_OVERFLOW = 3,       /* a size that does not fit the index types */
    FA_ERR_CUDA = 4,           /* a CUDA runtime/driver call failed */
    FA_ERR_DEVICE_TIMEOUT = 5, /* (device word) a bounded wait ran out */
    FA_ERR_DEVICE_BOUNDS = 6   /* (device word) an index was out of range */
} fa_status_t;

typedef enum { FA_BF16 = 0, FA_E4M3 = 1, FA_F32 = 2, FA_I32 = 3, FA_U8 = 4, FA_I8 = 5 } fa_dtype_t;

/* A strided device tensor.  Strides are in ELEMENTS; shape[ndim..4] unused. */
typedef struct {
    void *data;
    int32_t dtype;       /* fa_dtype_t */
    int32_t ndim;
    int64_t shape[5];
    int64_t stride[5];
} fa_tensor_t;

/* Score modifier (fkl_python PR #7, flex commit): kind 0 none, 1 ALiBi
 * (s -= alibi_slope * |i' - j|, i' = i + Sk - Sq), 2 soft-cap
 * (s = softcap * tanh(s / softcap), on the scaled score, before ALiBi). */
typedef struct {
    int32_t kind;
    float alibi_slope;
    float softcap;
} fa_score_mod_t;

/* Prologue (fkl_python PR #7, prologue-fusion commit: op chains fused onto
 * the Q/K/V reads, values passed at run time).  Each tensor has a chain of
 * up to FA_PROLOGUE_MAX_OPS scalar ops, applied in order to every element as
 * it is read: FA_OP_MUL (x * value), FA_OP_ADD (x + value), FA_OP_SUB
 * (x - value), FA_OP_DIV (x / value).  n_q, n_k, n_v give the chain lengths
 * (0 = no op on that tensor).
 *
 * The library composes each chain into one map x -> a * x + b (in double
 * precision, on the host) and folds the maps instead of rewriting the
 * operands, which is exact in real arithmetic.  With q' = a_q q + b_q and
 * k' = a_k k + b_k the score scale * <q'_i, k'_j> is
 *   scale a_q a_k <q_i, k_j>                 (the scale is multiplied)
 *   + scale (a_q b_k sum_d q_i[d] + b_q b_k Dk)   (one term per query row)
 *   + scale b_q a_k sum_d k_j[d]             (one term per key),
 * and with v' = a_v v + b_v the output is a_v out + b_v (softmax weights sum
 * to 1).  The row term cancels in the softmax and is added to the LSE, or,
 * under the soft-cap (not shift-invariant), enters the capped score.  The key
 * term (a Q add) is computed by a pre-pass over the keys into the caller's
 * workspace (fa_fwd_workspace_bytes() includes it) and added to each score.
 * Rows that see no key keep out = 0 and LSE = -inf.
 * Limits: FA_ERR_INVALID_ARG for an unknown op, a chain longer than
 * FA_PROLOGUE_MAX_OPS, a value that is not finite or a division by 0;
 * FA_ERR_UNSUPPORTED for b_q or b_k != 0 with e4m3 q.  NULL, or empty chains,
 * is no prologue. */
enum { FA_OP_MUL = 1, FA_OP_ADD = 2, FA_OP_SUB = 3, FA_OP_DIV = 4 };
#define FA_PROLOGUE_MAX_OPS 8
typedef struct {
    int32_t op;          /* FA_OP_* */
    float value;
} fa_prologue_op_t;
typedef struct {
    int32_t n_q, n_k, n_v;
    fa_prologue_op_t q[FA_PROLOGUE_MAX_OPS];
    fa_prologue_op_t k[FA_PROLOGUE_MAX_OPS];
    fa_prologue_op_t v[FA_PROLOGUE_MAX_OPS];
} fa_prologue_t;

/* 128x128 block-sparsity mask, uint8 [num_seqs * Hq][n_qblk][n_kblk],
 * contiguous; block (qb, kb) of sequence b, head h is active when
 * data[((b*Hq + h)*n_qblk + qb)*n_kblk + kb] != 0, with qb = i/128 and
 * kb = j/128 in sequence-local indices.  blk_q = blk_k = 128 only. */
typedef struct {
    const uint8_t *data;
    int32_t n_qblk, n_kblk, blk_q, blk_k;
} fa_block_mask_t;

/* Opt-in precision mode (fa_launch_t.flags): P * V on e4m3 operands
 * (FlyDSL PR #1066, Technical Details and Test Result: direct FP8 P x V at V
 * head dim 128, with its larger error).  Taken with e4m3 q and e4m3 K/V,
 * (Dk, Dv) in {(128, 128), (192, 128)}, token-major pages or packed K/V, no
 * prologue and a single pass (num_splits 0); FA_ERR_UNSUPPORTED otherwise.
 * The attention weights go to e4m3 as p * v_scale / 2^e, with 2^e above the
 * largest V scale of the sequence (a pre-pass over the V scales, writing one
 * fp32 per (sequence, kv head) into the workspace), and P * V runs on the
 * tensor core's e4m3 path with fp32 accumulation; the row sums and the LSE
 * stay fp32.  Each weight carries up to 2^-4 relative rounding, so outputs
 * differ from the exact attention by more than in the default mode (the
 * tests hold them to 4e-2; the LSE keeps its 1e-3). */
#define FA_FLAG_PV_E4M3 1

/* Host-side scalars, so that no length is read back from the device.
 * num_splits: 0 = single pass; > 0 = split-KV over that many key ranges
 * followed by the combine.  workspace: fa_fwd_workspace_bytes() bytes, needed
 * by split-KV with 2 or more splits, by a prologue with a Q add and by
 * FA_FLAG_PV_E4M3.  flags: 0, or FA_FLAG_PV_E4M3. */
typedef struct {
    int32_t num_seqs;
    int32_t max_seqlen_q;
    int32_t max_seqlen_k;
    int32_t num_splits;
    int64_t total_q;
    int64_t total_k;
    void *workspace;         /* device, 256-byte aligned, caller-owned */
    size_t workspace_bytes;
    int32_t flags;
} fa_launch_t;

/*
 * fa_fwd_varlen -- the attention forward pass.
 *
 *  q            bf16 [T_q, Hq, Dk], or e4m3 [T_q, Hq, Dk] with e4m3 caches,
 *               Dk 128 or 192 and Dv 128 (FlyDSL PR #1066 description: E4M3
 *               Q/K/V with scalar descales; the caller folds the Q descale
 *               into softmax_scale, and QK runs on the e4m3 bytes with the
 *               per-key scale applied to each score).  Last dim contiguous, the other
 *               strides multiples of 16 bytes.  Split-KV takes bf16 q only
 *               (Dk = Dv in {64, 128}); score mods, block masks and
 *               prologues apply to it as to the single pass.
 *  k_cache      paged: [N_pg, P_s, Hkv, Dk]; packed (block_table NULL):
 *               [T_k, Hkv, Dk].  bf16, e4m3 or int8.  Last three dims contiguous.
 *  v_cache      same layout and dtype with Dv (Dv may differ from Dk).
 *               Paged e4m3 and int8 caches may instead come in the
 *               vectorized 5-D layouts (FlyDSL PR #1066, Technical Details
 *               and review): K [N_pg, Hkv, Dk/16, P_s, 16] and V [N_pg, Hkv,
 *               P_s/16, Dv, 16], contiguous, 16 one-byte elements in the last
 *               dim, with pages of >= 16 keys and k_scale/v_scale
 *               [N_pg, P_s, Hkv]; results are bit-identical to the
 *               token-major pages.  Not with e4m3 q, a prologue add on q, or
 *               an add on k under the soft-cap (FA_ERR_UNSUPPORTED).
 *  block_table  int32 [num_seqs, max_pages], or NULL for packed K/V.  Entries
 *               for pages past a sequence's length are never read.
 *  cu_seqlens_q int32 [num_seqs + 1], prefix sums of query lengths.
 *  cu_seqlens_k int32 [num_seqs + 1], prefix sums of key lengths (row offsets
 *               into packed K/V; with a block table only their differences,
 *               the lengths, are used).
 *  k_scale      fp32 per token and kv head, [N_pg, P_s, Hkv] (paged) or
 *  v_scale      [T_k, Hkv] (packed); required for e4m3, must be NULL for bf16.
 *               The dequantised key is e4m3(k) * k_scale (same for v).
 *  out          bf16 [T_q, Hq, Dv], contiguous, caller-allocated; rows whose
 *               allowed key set is empty are written as 0.
 *  lse          fp32 [Hq, T_q] contiguous, or NULL to skip; -inf for rows
 *               with no allowed key.
 *  softmax_scale  multiplies <q, k>.
 *  causal       non-zero: key j visible iff j <= i + Sk - Sq (bottom-right).
 *  window       > 0: sliding window of `window` keys including the diagonal
 *               (causal: i' - j < window; otherwise |i' - j| < window).
 *  score_mod    NULL or fa_score_mod_t.
 *  block_mask   NULL or fa_block_mask_t.
 *  prologue     NULL or fa_prologue_t.
 *  page_size    tokens per page when paged: a power of two, 1 ... 1024.
 *               Pages of 16 or more keys are landed by TMA boxes; pages of
 *               1 ... 8 keys are gathered key row by key row (same results,
 *               bit for bit; slower).  e4m3 q needs pages of >= 16 keys.
 *  launch       host scalars (required).
 *  stream       cudaStream_t.
 *
 * e4m3 caches: K and V become f16 operands RN(e4m3 * scale) inside the
 * kernel, so |e4m3 value * scale| must stay below 65504 (scales below 146).
 *
 * Supported head dims: (Dk, Dv) in {(64,64), (128,128), (192,128)}.  Hq must
 * be a multiple of Hkv (query head h reads kv head h / (Hq/Hkv)).
 * Returns FA_OK or an error status; see fa_last_error().
 */
FA_API fa_status_t fa_fwd_varlen(const fa_tensor_t *q, const fa_tensor_t *k_cache,
                          const fa_tensor_t *v_cache, const fa_tensor_t *block_table,
                          const fa_tensor_t *cu_seqlens_q, const fa_tensor_t *cu_seqlens_k,
                          const fa_tensor_t *k_scale, const fa_tensor_t *v_scale,
                          fa_tensor_t *out, fa_tensor_t *lse, float softmax_scale,
                          int32_t causal, int32_t window, const fa_score_mod_t *score_mod,
                          const fa_block_mask_t *block_mask, const fa_prologue_t *prologue,
                          int32_t page_size, const fa_launch_t *launch, void *stream);

/*
 * Prepared calls.  fa_fwd_plan_create validates a forward call exactly like
 * fa_fwd_varlen (same arguments except the stream) and records the launches
 * it would make -- tensor maps, kernel parameters, grid -- without enqueuing
 * anything.  fa_fwd_plan_launch enqueues them on `stream`: the host work of a
 * call drops to the kernel launches, which matters for small problems issued
 * repeatedly (decode loops, serving).  The plan keeps the device addresses of
 * every tensor and of the workspace: they must stay allocated, unmoved and of
 * the same shape while the plan is used, and their contents are read at each
 * launch.  A plan runs on the device that was current at creation.  Launching
 * a plan on two streams at once is allowed only without a workspace (split-KV
 * partials would race).  fa_fwd_plan_destroy frees the host-side plan (NULL is
 * a no-op).  Status and error reporting as for fa_fwd_varlen.
 */
typedef struct fa_fwd_plan_s *fa_fwd_plan_t;

FA_API fa_status_t fa_fwd_plan_create(const fa_tensor_t *q, const fa_tensor_t *k_cache, const fa_tensor_t *v_cache,
                               const fa_tensor_t *block_table, const fa_tensor_t *cu_seqlens_q,
                               const fa_tensor_t *cu_seqlens_k, const fa_tensor_t *k_scale,
                               const fa_tensor_t *v_scale, fa_tensor_t *out, fa_tensor_t *lse,
                               float softmax_scale, int32_t causal, int32_t window,
                               const fa_score_mod_t *score_mod, const fa_block_mask_t *block_mask,
                               const fa_prologue_t *prologue, int32_t page_size, const fa_launch_t *launch,
                               fa_fwd_plan_t *plan);
FA_API fa_status_t fa_fwd_plan_launch(fa_fwd_plan_t plan, void *stream);
FA_API void fa_fwd_plan_destroy(fa_fwd_plan_t plan);

/*
 * Workspace size in bytes of a forward call with these host scalars, head
 * counts and prologue (NULL = none): for split-KV with launch->num_splits >= 2,
 * partial outputs fp32 [num_splits, T_q, Hq, Dv] and partial LSEs fp32
 * [num_splits, Hq, T_q]; for a prologue whose Q chain adds a constant (see
 * fa_prologue_t), the per-key score terms fp32 [num_seqs, Hkv,
 * ceil(max_seqlen_k / 128) * 128].  Each part is 256-byte aligned.  0 when
 * neither applies or launch is NULL.
 */
FA_API size_t fa_fwd_workspace_bytes(const fa_launch_t *launch, int32_t hq, int32_t hkv, int32_t dv,
                              const fa_prologue_t *prologue);

/*
 * Recommended split count for a problem (0 = single pass).  Split-KV applies
 * when few query rows share each kv head (decode: max_seqlen_q * Hq/Hkv <= 16)
 * and keys are long.  The key ranges are sized so that the non-empty CTAs make
 * about three waves at two CTAs per SM of the current device; total_k (the
 * sum of key lengths, 0 if unknown) refines the estimate of non-empty ranges.
 */
FA_API int32_t fa_fwd_default_splits(int32_t num_seqs, int32_t max_seqlen_q, int32_t max_seqlen_k,
                              int64_t total_k, int32_t hq, int32_t hkv, int32_t page_size);

/*
 * fa_combine -- merge of partial results over disjoint key ranges (the
 * split-KV combine; FlyDSL PR #844, Changes: m_max*ln2 + ln(den)):
 *   LSE = ln sum_s exp(LSE_s),  out = sum_s exp(LSE_s - LSE) * O_s,
 * partials with LSE_s = -inf are skipped; all -inf gives out 0, LSE -inf.
 *  o_part   fp32 [num_splits, n_rows, Hq, Dv] contiguous (n_rows = T_q)
 *  lse_part fp32 [num_splits, Hq, n_rows] contiguous
 *  out      bf16 [n_rows, Hq, Dv] contiguous;  lse fp32 [Hq, n_rows] or NULL.
 */
FA_API fa_status_t fa_combine(const float *o_part, const float *lse_part, int32_t num_splits,
                       int64_t n_rows, int32_t hq, int32_t dv, void *out_bf16, float *lse,
                       void *stream);

/*
 * fa_bwd_varlen -- the backward pass: gradients of L = sum(dout * out) with
 * respect to q, k and v, recomputed from the forward's saved LSE
 * (RL-Kernel PR #237, backward commit: a Delta preprocess, then dQ/dK/dV from
 * the saved LSE):
 *   Delta_i = <dout_i, out_i>,   P_ij = exp(softmax_scale * <q_i, k_j> - LSE_i)
 *   dP_ij = <dout_i, v_j>,   dS_ij = P_ij * (dP_ij - Delta_i)
 *   dv_j = sum_i P_ij dout_i,  dk_j = softmax_scale * sum_i dS_ij q_i,
 *   dq_i = softmax_scale * sum_j dS_ij k_j      (allowed (i, j) only)
 * With a score mod, P uses the modified score s_ij.  ALiBi leaves dS as
 * written; the soft-cap s = cap * tanh(u / cap), u = softmax_scale <q, k>,
 * multiplies dS_ij by ds/du = 1 - tanh^2(u_ij / cap).
 *
 *  q, out, dout, dq   bf16 [T_q, Hq, D];  k, v, dk, dv   bf16 [T_k, Hkv, D],
 *                     packed varlen (no block table).  D = 64 or 128 (Dk = Dv).
 *                     Last dim contiguous, other strides multiples of 8
 *                     elements, bases 16-byte aligned.  GQA: Hq % Hkv == 0;
 *                     dk, dv sum over the q heads of each kv head's group.
 *  lse                fp32 [Hq, T_q] contiguous, the forward's LSE for the
 *                     same (q, k, v, masks).
 *  cu_seqlens_q/k     int32 [num_seqs + 1] (row offsets of q and of k/v).
 *  softmax_scale      > 0;  causal, window, score_mod (NULL or kind 0, 1, 2)
 *                     and block_mask (NULL or 128 x 128 blocks) as in
 *                     fa_fwd_varlen: a skipped block adds nothing to any
 *                     gradient.
 *  launch             num_seqs, max_seqlen_q/k, total_q (= T_q) and a
 *                     workspace of fa_bwd_workspace_bytes(T_q, Hq) bytes,
 *                     256-byte aligned, for Delta (fp32 [Hq, T_q]).
 * Outputs are overwritten (rows of keys or queries that see nothing get 0)
 * and must not overlap any input or each other.  Three kernels are enqueued
 * on `stream` (Delta, dK/dV, dQ); no allocation, copy or synchronisation.
 * Errors as for fa_fwd_varlen: FA_ERR_INVALID_ARG for shapes, dtypes,
 * strides, alignment or a missing workspace, FA_ERR_UNSUPPORTED for other
 * head dims, FA_ERR_CUDA for launch failures.
 */
FA_API fa_status_t fa_bwd_varlen(const fa_tensor_t *q, const fa_tensor_t *k, const fa_tensor_t *v,
                          const fa_tensor_t *out, const fa_tensor_t *dout, const fa_tensor_t *lse,
                          const fa_tensor_t *cu_seqlens_q, const fa_tensor_t *cu_seqlens_k,
                          fa_tensor_t *dq, fa_tensor_t *dk, fa_tensor_t *dv, float softmax_scale,
                          int32_t causal, int32_t window, const fa_score_mod_t *score_mod,
                          const fa_block_mask_t *block_mask, const fa_launch_t *launch, void *stream);

/* Workspace bytes of fa_bwd_varlen: Delta, fp32 [Hq, T_q], rounded up to 256. */
FA_API size_t fa_bwd_workspace_bytes(int64_t total_q, int32_t hq);

/*
 * fa_fwd_varlen_noalloc -- the split-KV decode of fa_fwd_varlen for callers
 * that cannot allocate device memory.  (The pages have no counterpart: this
 * entry exists for deployment, not for the method.)
 *
 * Who needs it: custom ops and plugins that are handed only their input and
 * output buffers, serving loops whose device memory is fixed at start-up, and
 * request paths that must not call cudaMalloc because it may synchronise the
 * device or fail under memory pressure.  Instead of launch->workspace, the
 * per-split partials go to a static device array of FA_NOALLOC_SCRATCH_BYTES
 * owned by the library.  The array is part of the library's device code:
 * CUDA reserves it on a device when it loads the library's code there, which
 * under lazy module loading (the default since CUDA 12) happens at the first
 * use on that device -- possibly this entry's first call -- and it stays
 * reserved until the process exits.  Callers with no spare device memory
 * should therefore make one call per device at start-up.  The call itself
 * asks for no memory: no cudaMalloc, no allocating library routine.
 *
 * Arguments and layouts are those of fa_fwd_varlen; launch->workspace and
 * launch->workspace_bytes are ignored.  launch->num_splits <= 0 picks
 * fa_fwd_default_splits(); the problem must be a split-KV decode shape with
 * at least 2 splits, and fa_fwd_workspace_bytes() for it (with q.shape[0]
 * rows, which must equal launch->total_q) must not exceed
 * FA_NOALLOC_SCRATCH_BYTES, else FA_ERR_UNSUPPORTED is returned with nothing
 * enqueued.
 *
 * The first call on each device looks up the array's device address (with
 * that device current); make that first call before any stream capture.
 * Every call shares the one array and leaves its partials there: calls whose
 * work overlaps on the GPU (different streams, or the same stream from several
 * host threads without ordering) race on it.  No part of the array needs to
 * start at zero.
 */
#define FA_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
FA_API fa_status_t fa_fwd_varlen_noalloc(const fa_tensor_t *q, const fa_tensor_t *k_cache,
                                  const fa_tensor_t *v_cache, const fa_tensor_t *block_table,
                                  const fa_tensor_t *cu_seqlens_q, const fa_tensor_t *cu_seqlens_k,
                                  const fa_tensor_t *k_scale, const fa_tensor_t *v_scale,
                                  fa_tensor_t *out, fa_tensor_t *lse, float softmax_scale,
                                  int32_t causal, int32_t window, const fa_score_mod_t *score_mod,
                                  const fa_block_mask_t *block_mask, const fa_prologue_t *prologue,
                                  int32_t page_size, const fa_launch_t *launch, void *stream);

/*
 * Decode of a batch whose sequences share prefixes.
 *
 * fa_fwd_shared_prefix computes what fa_fwd_varlen computes -- same arguments,
 * layouts, masks and results -- for a paged batch of few query rows per
 * sequence, and reads the keys that a group of sequences shares once for the
 * whole group instead of once per sequence.
 *
 * The sequences come in groups, in order: group g holds the sequences
 * cu_groups[g] ... cu_groups[g + 1] - 1 (cu_groups[0] = 0 and
 * cu_groups[num_groups] = num_seqs; a violation records
 * FA_ERR_DEVICE_BOUNDS and the rows left out are undefined).  The sequences of
 * group g hold the same keys first: lens[g] of them, rounded down to whole
 * pages, in the same pages.  Their block-table rows repeat those pages; the
 * group's first row is read.  Lengths (cu_seqlens_k) count the shared keys.
 * Each row keeps its own causal limit, window and length, also inside the
 * prefix, and a group of one sequence or a prefix of 0 keys is fine.
 *
 * max_len and num_splits only size the work: max_len bounds lens[] (a longer
 * prefix is still attended in full), num_splits >= 1 cuts a prefix of max_len
 * keys into that many key ranges, and shorter ones into fewer of the same
 * length (fa_shared_prefix_default_splits).  launch->num_splits
 * >= 1 cuts the keys behind the prefix likewise, sized by max_seqlen_k -
 * max_len (fa_shared_prefix_default_own_splits).
 */
typedef struct {
    const int32_t *cu_groups;   /* device, int32 [num_groups + 1] */
    const int32_t *lens;        /* device, int32 [num_groups] */
    int32_t num_groups;
    int32_t max_len;
    int32_t num_splits;
} fa_shared_prefix_t;

/*
 *  q, out, lse   as fa_fwd_varlen; q bf16, Dk = Dv in {64, 128},
 *                max_seqlen_q * Hq/Hkv <= 16.
 *  k_cache, v_cache, k_scale, v_scale, block_table, page_size
 *                token-major pages [N_pg, P_s, Hkv, D] of 1 ... 1024 keys,
 *                bf16, e4m3 or int8 (per-token scales), as fa_fwd_varlen.
 *  causal, window, score_mod   as fa_fwd_varlen.
 *  launch        workspace of fa_shared_prefix_workspace_bytes() bytes,
 *                256-byte aligned, for the partials; flags 0.
 * Three kernels: the prefix pass, the sequences' own keys, the merge.
 * FA_ERR_UNSUPPORTED for packed K/V, the 5-D pages, other head dims or more
 * query rows; other errors as fa_fwd_varlen.  A page id outside the pool
 * counts as a page of zeros and records FA_ERR_DEVICE_BOUNDS.  A sequence whose
 * query rows (cu_seqlens_q) lie outside q records it too and has no result.
 */
FA_API fa_status_t fa_fwd_shared_prefix(const fa_tensor_t *q, const fa_tensor_t *k_cache, const fa_tensor_t *v_cache,
                                 const fa_tensor_t *block_table, const fa_tensor_t *cu_seqlens_q,
                                 const fa_tensor_t *cu_seqlens_k, const fa_tensor_t *k_scale,
                                 const fa_tensor_t *v_scale, fa_tensor_t *out, fa_tensor_t *lse, float softmax_scale,
                                 int32_t causal, int32_t window, const fa_score_mod_t *score_mod,
                                 const fa_shared_prefix_t *prefix, int32_t page_size, const fa_launch_t *launch,
                                 void *stream);

/* Prepared form (see fa_fwd_plan_create): launched by fa_fwd_plan_launch and
 * freed by fa_fwd_plan_destroy.  fa_fwd_plan_launch returns
 * FA_ERR_INVALID_ARG when another device is current than at creation. */
FA_API fa_status_t fa_shared_prefix_plan_create(const fa_tensor_t *q, const fa_tensor_t *k_cache,
                                         const fa_tensor_t *v_cache, const fa_tensor_t *block_table,
                                         const fa_tensor_t *cu_seqlens_q, const fa_tensor_t *cu_seqlens_k,
                                         const fa_tensor_t *k_scale, const fa_tensor_t *v_scale, fa_tensor_t *out,
                                         fa_tensor_t *lse, float softmax_scale, int32_t causal, int32_t window,
                                         const fa_score_mod_t *score_mod, const fa_shared_prefix_t *prefix,
                                         int32_t page_size, const fa_launch_t *launch, fa_fwd_plan_t *plan);

/* Workspace bytes of fa_fwd_shared_prefix: fp32 partials [splits, T_q, Hq, D]
 * and LSEs [splits, Hq, T_q], each 256-byte aligned, of prefix->num_splits +
 * launch->num_splits splits. */
FA_API size_t fa_shared_prefix_workspace_bytes(const fa_launch_t *launch, const fa_shared_prefix_t *prefix, int32_t hq,
                                        int32_t dv);

/* Recommended number of key ranges of the prefix pass, and of the pass over
 * the keys behind it (max_own_len: the longest sequence's such keys; total_own:
 * their sum over the sequences, 0 if unknown).  Both are >= 1. */
FA_API int32_t fa_shared_prefix_default_splits(int64_t total_q, int32_t num_groups, int32_t max_len, int32_t hq,
                                        int32_t hkv, int32_t kv_dtype);
FA_API int32_t fa_shared_prefix_default_own_splits(int32_t num_seqs, int32_t max_own_len, int64_t total_own, int32_t hkv);

/*
 * fa_key_weights -- the attention weight that each key received, summed over
 * query rows and over the heads that share a kv head, from the forward's LSE:
 *   out[b][hk][j] = beta * weights[b][hk][j]
 *                   + sum_{i, h in group(hk)} exp(s_ij - lse[h][i])
 * over the rows i of sequence b that see key j (s_ij, causal, window and
 * score_mod as in the fa_fwd_varlen call that wrote lse).  It is the score by
 * which fa_cache_evict chooses; accumulate over decode steps with beta = 1 (or
 * a decay below 1) and out = weights.
 *
 *  q            bf16 [T_q, Hq, Dk], Dk in {64, 128, 192}, Hq/Hkv <= 128.
 *  k_cache      as fa_fwd_varlen: packed or token-major pages of 1 ... 1024
 *               keys; bf16, or e4m3 / int8 with k_scale.
 *  lse          fp32 [Hq, T_q] contiguous, natural log; rows with -inf add
 *               nothing.
 *  weights      fp32 [num_seqs, Hkv, L], last dim contiguous, or NULL (as
 *               beta = 0: nothing is read).
 *  beta         finite; 0 reads nothing.
 *  out          fp32 [num_seqs, Hkv, L], last dim contiguous, rows apart from
 *               each other, L >= launch->max_seqlen_k; `weights` itself (same
 *               address and strides) or no overlap with it.  Entries j past a
 *               sequence's keys get beta * weights (0 without weights).
 *  launch       num_seqs, max_seqlen_q, max_seqlen_k, total_q (and total_k
 *               for packed K); no workspace.  max_seqlen_k and max_seqlen_q
 *               bound the lengths: a longer sequence records
 *               FA_ERR_DEVICE_BOUNDS and its excess is left out.  A page id
 *               outside the pool counts as keys of zeros and records it too,
 *               and a sequence whose query rows lie outside q adds nothing.
 * One kernel: for max_seqlen_q * Hq/Hkv <= 16 bound by reading K, otherwise
 * tensor-core tiles.  Sums are fp32 in a fixed order (the same bits each run).
 */
FA_API fa_status_t fa_key_weights(const fa_tensor_t *q, const fa_tensor_t *k_cache, const fa_tensor_t *block_table,
                           const fa_tensor_t *cu_seqlens_q, const fa_tensor_t *cu_seqlens_k, const fa_tensor_t *k_scale,
                           const fa_tensor_t *lse, const fa_tensor_t *weights, float beta, fa_tensor_t *out,
                           float softmax_scale, int32_t causal, int32_t window, const fa_score_mod_t *score_mod,
                           int32_t page_size, const fa_launch_t *launch, void *stream);

/* Prepared form, as fa_shared_prefix_plan_create. */
FA_API fa_status_t fa_key_weights_plan_create(const fa_tensor_t *q, const fa_tensor_t *k_cache,
                                       const fa_tensor_t *block_table, const fa_tensor_t *cu_seqlens_q,
                                       const fa_tensor_t *cu_seqlens_k, const fa_tensor_t *k_scale,
                                       const fa_tensor_t *lse, const fa_tensor_t *weights, float beta, fa_tensor_t *out,
                                       float softmax_scale, int32_t causal, int32_t window,
                                       const fa_score_mod_t *score_mod, int32_t page_size, const fa_launch_t *launch,
                                       fa_fwd_plan_t *plan);

/*
 * fa_cache_evict -- shortens the sequences of a paged cache to `budget` keys
 * per kv head, by accumulated attention weight (fa_key_weights).
 *
 * A sequence of at most `budget` keys keeps them all.  A longer one keeps, for
 * each kv head on its own, its first `sink` keys, its last `recent` keys and,
 * of the others, the budget - sink - recent with the largest weights (ties:
 * the lowest index; NaN ranks below every number).  The keys that stay keep
 * their order and become keys 0 ... n - 1: their K and V rows, scales and
 * weights move, everything else in the pages stays as it was.  All heads keep
 * the same number, so the new lengths serve every later call; positions that
 * were encoded into K beforehand stay with the keys.
 *
 *  weights           fp32 [num_seqs, Hkv, L], last dim contiguous, L >=
 *                    launch->max_seqlen_k.
 *  weights_out       NULL: weights themselves are updated; or fp32 [num_seqs,
 *                    Hkv, >= budget], last dim contiguous, no overlap with
 *                    weights.  Entries past the kept keys are set to 0, so that
 *                    appended keys start from 0.
 *  k_cache, v_cache  token-major pages [N_pg, P_s, Hkv, D], (Dk, Dv) and types
 *                    as fa_fwd_varlen; k_scale, v_scale [N_pg, P_s, Hkv] with
 *                    byte caches.
 *  block_table       int32 [num_seqs, max_pages].
 *  block_table_out   NULL: in place; or int32 [num_seqs, >= ceil(budget /
 *                    page_size)]: the kept keys are written to these pages of
 *                    the pool, which no block_table row may hold, and the old
 *                    pages stay as they were.
 *  cu_seqlens_k      int32 [num_seqs + 1];  cu_seqlens_k_out the same shape, the
 *                    prefix sums of the new lengths; no overlap.
 *  kept              int32 [num_seqs, Hkv, budget] contiguous: the old index of
 *                    each kept key, ascending; -1 past the kept keys.
 *  budget >= 1, sink >= 0, recent >= 0, sink + recent <= budget.
 *  launch            num_seqs, max_seqlen_k; no workspace.  A sequence longer
 *                    than max_seqlen_k, L or its table records
 *                    FA_ERR_DEVICE_BOUNDS and counts as that long.
 * In place, a page may stand in several block_table rows (or twice in one) only
 * within the first `sink` keys (those never move); in block_table_out once.  A page id outside the pool is skipped and records
 * FA_ERR_DEVICE_BOUNDS.
 */
FA_API fa_status_t fa_cache_evict(const fa_tensor_t *weights, fa_tensor_t *weights_out, const fa_tensor_t *k_cache,
                           const fa_tensor_t *v_cache, const fa_tensor_t *k_scale, const fa_tensor_t *v_scale,
                           const fa_tensor_t *block_table, const fa_tensor_t *block_table_out,
                           const fa_tensor_t *cu_seqlens_k, fa_tensor_t *cu_seqlens_k_out, fa_tensor_t *kept,
                           int32_t budget, int32_t sink, int32_t recent, int32_t page_size, const fa_launch_t *launch,
                           void *stream);

/* Message for the last non-OK status returned on this thread ("" if none). */
FA_API const char *fa_last_error(void);

/* Synchronises `stream`, then reads and clears the current device's error
 * word into *code (FA_OK when no kernel recorded a problem). */
FA_API fa_status_t fa_get_device_error(void *stream, int32_t *code);

/* Library version string. */
FA_API const char *fa_version(void);

#ifdef __cplusplus
}
#endif
#endif /* FA_GB300_H */
