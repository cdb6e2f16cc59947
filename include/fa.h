/*
 * fa.h — C ABI of the exact-attention library for one NVIDIA GB300 (sm_103a).
 *
 * The library computes exact scaled-dot-product attention
 *
 *     O = softmax(scale * Q K^T) V
 *
 * FlashAttention-2 style: an outer loop over 128-row query blocks and an inner
 * loop over key/value blocks (64 rows for D <= 64, 128 for D = 128 in the
 * forward pass) with an online softmax (running row
 * maximum m and running sum l), so the [S, S] score matrix never reaches
 * memory.  Only O and the per-row logsumexp L are written.  The backward pass
 * recomputes the probabilities from L.  Definitions followed:
 *   - forward recurrence and L: "从零训练语言模型（第二部分：FlashAttention 与设备内存）"
 *     §安全 / 在线 softmax and §使用 LSE 连接正向和反向传播;
 *     "T5 讲解：FlashAttention forward" §④ (online softmax update), §⑤ (causal
 *     block skipping), §⑥ (default scale 1/sqrt(D));
 *   - backward: the same "第二部分" page §反向传播 (P = exp(S - L), dV = P^T dO,
 *     dP = dO V^T, dS = P o (dP - D), dQ = dS K * scale, dK = dS^T Q * scale),
 *     and the CS336 Assignment 2 write-up, "4. Problem (flash_backward)"
 *     (recompute backward with the row vector D = rowsum(dO o O)).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Layout: every matrix argument (q, k, v, o, dout, dq, dk, dv) is a dense,
 *   contiguous row-major tensor [B, H, S, D] of 16-bit floats (fp16 or bf16,
 *   chosen by `dtype`), element strides (H*S*D, S*D, D, 1).  Query and key
 *   lengths are equal (S).  `lse` is fp32 [B, H, S]; it holds the NATURAL-log
 *   logsumexp of the scaled scores, L_i = ln sum_j exp(scale * q_i . k_j).
 * Causal: when `causal` is nonzero, query i attends to keys j <= i (top-left
 *   aligned mask).  Every query row then sees at least key 0.
 * Scale: any finite float; the usual value is 1/sqrt(D).
 * Supported: D in {16, 32, 64, 128}; S >= 0; B, H >= 0; B*H < 2^31;
 *   S < 2^31.  S == 0 or B*H == 0 is a valid empty call that launches nothing.
 * Pointers: DEVICE pointers of the current CUDA device, each 16-byte aligned
 *   (the tensor-memory-access engine requires it).  In an empty call they are
 *   not used and may be NULL.
 * Ownership: the caller owns every buffer and the stream.  The library
 *   allocates no memory, keeps no pointer after a call returns, and does not
 *   synchronise: results are ready when `stream` reaches the launched work.
 * Stream: a cudaStream_t passed as void* (NULL = the legacy default stream).
 * Errors: every entry point validates all arguments before launching anything
 *   and returns FA_OK or an fa_status code; nothing is launched on error.
 *   fa_last_error_detail() gives a one-line description of the last failure
 *   on the calling thread.  Kernels never trap: a device-side pipeline wait
 *   that exceeds its time limit (2 s by default, see fa_set_wait_limit_ns)
 *   ends the kernel and sets a device error word that fa_check_device_errors()
 *   reads.
 */
#ifndef FA_GB300_H
#define FA_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1, /* null pointer, negative size, non-finite scale, bad dtype */
  FA_ERR_UNSUPPORTED = 2, /* head dimension not in {16,32,64,128}, or sizes too large */
  FA_ERR_ALIGNMENT = 3,   /* a pointer is not 16-byte aligned */
  FA_ERR_WORKSPACE = 4,   /* workspace missing or smaller than fa_bwd_workspace_size() */
  FA_ERR_CUDA = 5,        /* a CUDA runtime/driver call or a kernel launch failed */
  FA_ERR_TIMEOUT = 6      /* a device pipeline wait exceeded its limit (see fa_check_device_errors) */
} fa_status;

typedef enum { FA_FP16 = 0, FA_BF16 = 1 } fa_dtype;

/*
 * Forward pass.
 *   q, k, v : [B, H, S, D] inputs (read only).
 *   o       : [B, H, S, D] output, same dtype; O = softmax(scale Q K^T (+mask)) V.
 *   lse     : [B, H, S] fp32 output, natural-log logsumexp per query row.
 * Per query block the kernel visits only key blocks that are not wholly above
 * the diagonal when causal ("T5 讲解" §⑤), masks element-wise only in the
 * diagonal block and in a ragged last key block, and writes O / l and
 * L = m + ln l in the epilogue.
 */
fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B, int64_t H,
                 int64_t S, int64_t D, int causal, float scale, fa_dtype dtype, void* stream);

/*
 * Forward pass with grouped K/V heads (multi-query / grouped-query attention,
 * "Inside FlashAttention" §6.1, the MQA / GQA interface: several query heads
 * share one K/V head, and K, V are passed with fewer heads instead of being
 * copied out to H heads).
 *   q, o    : [B, H, S, D];  lse : [B, H, S] fp32.
 *   k, v    : [B, H_kv, S, D].
 * H must be a positive multiple of H_kv (H_kv >= 1); query head h of batch b
 * reads K/V head h / (H / H_kv) of batch b, so each K/V head serves a run of
 * H / H_kv consecutive query heads.  H_kv = H is fa_fwd; H_kv = 1 is
 * multi-query attention.  A call with B*H == 0 (then H_kv == 0 is allowed
 * when H == 0) or S == 0 launches nothing.  Every other convention
 * (layout, alignment, ownership, errors) is fa_fwd's; a bad H_kv returns
 * FA_ERR_INVALID_ARG.
 */
fa_status fa_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B, int64_t H,
                     int64_t H_kv, int64_t S, int64_t D, int causal, float scale, fa_dtype dtype, void* stream);

/*
 * Bytes of device workspace fa_bwd needs for these sizes: the fp32 row vector
 * D_i = rowsum(dO o O) for every (b, h, i), rounded up to 256 bytes.
 */
size_t fa_bwd_workspace_size(int64_t B, int64_t H, int64_t S, int64_t D);

/*
 * Backward pass (recompute).  Given the forward inputs, its outputs o and lse,
 * and the loss gradient dout = dL/dO, writes dq, dk, dv ([B, H, S, D], same
 * dtype).  Three passes run in order on `stream`:
 *   1. D_i = rowsum(dO o O) into the workspace (fp32);
 *   2. per 128-key block: dV = sum_i P^T dO and dK = scale * sum_i dS^T Q over the
 *      query blocks that see it, P = exp(S - L) recomputed from lse;
 *   3. per 128-query block: dQ = scale * sum_j dS K over its visible key blocks.
 * At D <= 64 the dQ kernel computes D_i itself (and writes it to the
 * workspace): two kernels then run, the dQ pass first and the dK/dV pass after.
 * workspace: device buffer of at least fa_bwd_workspace_size() bytes, 256-byte
 * aligned, owned by the caller; its contents on entry do not matter.
 */
fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
                 const float* lse, void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t S, int64_t D,
                 int causal, float scale, fa_dtype dtype, void* workspace, size_t workspace_bytes,
                 void* stream);

/*
 * fa_bwd with timing marks.  Same arguments, same launches, same results;
 * in addition, each non-NULL entry of `marks` (a cudaEvent_t passed as void*,
 * owned by the caller) is recorded on `stream`, in this order: marks[0]
 * before the first kernel; marks[1] after the Delta kernel, or after the dQ
 * kernel where that computes Delta (fa_bwd, fa_bwd_gqa at D <= 64; the
 * window and packed-batch calls always run the Delta kernel); marks[2] after
 * the dK/dV kernel (and its partial-sum reduction); marks[3] after the dQ
 * kernel where it runs last, else right after marks[2].  Lets a caller time
 * each kernel with CUDA events on the stream that runs it.  `marks` itself
 * may be NULL.
 */
fa_status fa_bwd_marked(const void* q, const void* k, const void* v, const void* o, const void* dout,
                        const float* lse, void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t S,
                        int64_t D, int causal, float scale, fa_dtype dtype, void* workspace,
                        size_t workspace_bytes, void* stream, void* const* marks);

/*
 * Backward pass with grouped K/V heads: the gradient of fa_fwd_gqa.
 *   q, o, dout, dq : [B, H, S, D];  lse : [B, H, S] fp32.
 *   k, v, dk, dv   : [B, H_kv, S, D].
 * A K/V head's gradients sum the contributions of all H / H_kv query heads
 * that read it: dV_g = sum over the group's heads h of P_h^T dO_h, and dK_g
 * likewise with dS_h^T Q_h.  A dK/dV CTA owns one (K/V head, 128-key block)
 * and streams query heads of the group one after another through the same
 * accumulators.  When the K/V heads alone give too few CTAs to fill the GPU
 * (few K/V heads, short sequences), s CTAs share a (K/V head, key block),
 * each over G/s of the group's heads (s the smallest divisor of G that gives
 * 304 CTAs, else G); they write fp32 partial sums to the workspace and a
 * further kernel adds them in a fixed order.  No atomics either way: results
 * are deterministic.  Workspace: fa_bwd_gqa_workspace_size() bytes.  Other
 * conventions as fa_bwd; H_kv as in fa_fwd_gqa.
 */
fa_status fa_bwd_gqa(const void* q, const void* k, const void* v, const void* o, const void* dout,
                     const float* lse, void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t H_kv,
                     int64_t S, int64_t D, int causal, float scale, fa_dtype dtype, void* workspace,
                     size_t workspace_bytes, void* stream);

/*
 * Bytes of device workspace fa_bwd_gqa needs: the fp32 row vector D of every
 * query row (B*H*S floats, rounded up to 256 bytes), plus, when the dK/dV
 * pass splits the group (see fa_bwd_gqa), s * B*H_kv*S*2*D fp32 partial sums
 * (rounded up to 256 bytes).  Equals fa_bwd_workspace_size() when H_kv = H.
 * Returns 0 for an empty problem or an H_kv that does not divide H.
 */
size_t fa_bwd_gqa_workspace_size(int64_t B, int64_t H, int64_t H_kv, int64_t S, int64_t D);

/* fa_bwd_gqa with the timing marks of fa_bwd_marked (marks[2] is recorded
 * after the dK/dV kernel and, when it runs, the partial-sum kernel). */
fa_status fa_bwd_gqa_marked(const void* q, const void* k, const void* v, const void* o, const void* dout,
                            const float* lse, void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t H_kv,
                            int64_t S, int64_t D, int causal, float scale, fa_dtype dtype, void* workspace,
                            size_t workspace_bytes, void* stream, void* const* marks);

/*
 * Sliding-window (local) attention ("Inside FlashAttention" §6.1, window_size
 * = (left, right): only the key blocks inside the window are computed).  Key j
 * is visible to query i only if i - window_left <= j <= i + window_right; a
 * negative side is unlimited, and `causal` additionally hides j > i (so
 * causal with (left, 0) is the usual local causal window).  Layouts, grouped
 * heads (H_kv) and every other convention as fa_fwd_gqa / fa_bwd_gqa.  Each
 * 128-row query tile (or 128-key tile in the backward) visits only the key
 * (query) blocks that meet its band; blocks crossing either edge of the band
 * are masked element-wise, the others run unmasked.  Every query row sees at
 * least its own key, so no row is empty.  A window that covers the whole
 * sequence runs the ordinary kernels.  Workspace: fa_bwd_gqa_workspace_size().
 */
fa_status fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B, int64_t H,
                        int64_t H_kv, int64_t S, int64_t D, int causal, int64_t window_left, int64_t window_right,
                        float scale, fa_dtype dtype, void* stream);

fa_status fa_bwd_window(const void* q, const void* k, const void* v, const void* o, const void* dout,
                        const float* lse, void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t H_kv,
                        int64_t S, int64_t D, int causal, int64_t window_left, int64_t window_right, float scale,
                        fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/* fa_bwd_window with the timing marks of fa_bwd_marked. */
fa_status fa_bwd_window_marked(const void* q, const void* k, const void* v, const void* o, const void* dout,
                               const float* lse, void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t H_kv,
                               int64_t S, int64_t D, int causal, int64_t window_left, int64_t window_right,
                               float scale, fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream,
                               void* const* marks);

/*
 * Split-KV forward with a logsumexp merge ("T5 讲解" §⑥: the stored
 * L = m + log l is what lets shards be merged).  The keys are cut into shards
 * of ceil(S / num_splits) keys rounded up to a multiple of 128; one launch
 * computes, per (b, h, query tile, shard), the fp32 output normalised over the
 * shard's keys and its logsumexp into `workspace`, and a second kernel merges
 * the shards:  L = ln sum_s exp(L_s),  O = sum_s exp(L_s - L) O_s.  The result
 * equals fa_fwd_gqa's up to fp32 rounding; it pays off where B*H*ceil(S/512)
 * (ceil(S/256) for D = 128) query tiles alone cannot fill the GPU.  Layouts,
 * heads and causal as in fa_fwd_gqa.  num_splits >= 1 (1 is legal: one
 * shard); fa_splitkv_num_splits() proposes one.  workspace: at least
 * fa_fwd_splitkv_workspace_size() bytes, 256-byte aligned, owned by the caller.
 */
fa_status fa_fwd_splitkv(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B, int64_t H,
                         int64_t H_kv, int64_t S, int64_t D, int causal, int64_t num_splits, float scale,
                         fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace of fa_fwd_splitkv: shards * B*H*S * (D + 1) fp32 values, rounded up to 256 bytes. */
size_t fa_fwd_splitkv_workspace_size(int64_t B, int64_t H, int64_t S, int64_t D, int64_t num_splits);

/* A split count that gives a 152-SM GPU at least two CTAs per SM (1 when the
 * query tiles already do; at most one shard per 128 keys). */
int64_t fa_splitkv_num_splits(int64_t B, int64_t H, int64_t S, int64_t D);

/*
 * The merge on its own, for partials computed elsewhere (other GPUs' key
 * shards, a cache of earlier keys):
 *   o_part   : DEVICE fp32 [shards, rows, D], each shard's normalised output;
 *   lse_part : DEVICE fp32 [shards, rows], each shard's natural-log L_s
 *              (-inf for a row that sees no key of the shard; its O_s is ignored);
 *   o        : [rows, D] 16-bit output (dtype);  lse : [rows] fp32 output.
 * A row whose every L_s is -inf gets O = 0 and L = -inf.  D in {16,32,64,128}.
 */
fa_status fa_merge_lse(const float* o_part, const float* lse_part, void* o, float* lse, int64_t shards,
                       int64_t rows, int64_t D, fa_dtype dtype, void* stream);

/*
 * Packed variable-length batches ("Inside FlashAttention" §6.1, varlen: samples
 * of different lengths concatenated with no padding, a prefix-sum array
 * cu_seqlens marking their bounds, and no attention across samples).
 *   q, o           : [T, H, D]     (token-major; T = total tokens)
 *   k, v           : [T, H_kv, D]  (H a positive multiple of H_kv, as in fa_fwd_gqa)
 *   lse            : [H, T] fp32, natural-log logsumexp
 *   cu_seqlens     : DEVICE int32 [batch + 1]; cu[0] = 0, non-decreasing,
 *                    cu[batch] <= total; sample b is tokens cu[b] .. cu[b+1]-1
 *                    (empty samples allowed) and attends only to itself, with the
 *                    top-left causal mask inside the sample when causal.
 *   max_seqlen     : host bound on every sample length (sizes the grid).
 * The kernels read cu_seqlens themselves.  A sample longer than max_seqlen,
 * or one that runs past `total`, is not computed: the kernels record it and
 * fa_check_device_errors() then returns FA_ERR_INVALID_ARG.  Rows of tokens
 * that no sample covers are left unwritten.  Other conventions as fa_fwd
 * (cu_seqlens needs 4-byte alignment only).  batch, H, max_seqlen or total
 * equal to 0 is an empty call.
 */
fa_status fa_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                        const int32_t* cu_seqlens, int64_t batch, int64_t max_seqlen, int64_t total, int64_t H,
                        int64_t H_kv, int64_t D, int causal, float scale, fa_dtype dtype, void* stream);

/* Workspace bytes of fa_bwd_varlen: Delta for the T*H query rows, plus the
 * dK/dV partial sums when the grouped pass splits (as fa_bwd_gqa_workspace_size,
 * with batch entries of up to max_seqlen rows; T*H_kv K/V rows). */
size_t fa_bwd_varlen_workspace_size(int64_t batch, int64_t max_seqlen, int64_t total, int64_t H, int64_t H_kv,
                                    int64_t D);

/* Backward of fa_fwd_varlen: dq [T, H, D], dk, dv [T, H_kv, D]; the packed
 * layout and checks of fa_fwd_varlen, the rest as fa_bwd_gqa. */
fa_status fa_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const void* dout,
                        const float* lse, void* dq, void* dk, void* dv, const int32_t* cu_seqlens, int64_t batch,
                        int64_t max_seqlen, int64_t total, int64_t H, int64_t H_kv, int64_t D, int causal,
                        float scale, fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/* fa_bwd_varlen with the timing marks of fa_bwd_marked. */
fa_status fa_bwd_varlen_marked(const void* q, const void* k, const void* v, const void* o, const void* dout,
                               const float* lse, void* dq, void* dk, void* dv, const int32_t* cu_seqlens,
                               int64_t batch, int64_t max_seqlen, int64_t total, int64_t H, int64_t H_kv, int64_t D,
                               int causal, float scale, fa_dtype dtype, void* workspace, size_t workspace_bytes,
                               void* stream, void* const* marks);

/* ------------------------------------------------------------------------
 * Modified scores.  The score of query i and key j,
 *
 *     s_ij = cap * tanh(scale * q_i . k_j / cap) - slopes[h] * |i - j|
 *
 * stands in the place of scale * q_i . k_j; either part may be absent.  i and j
 * are positions within the sequence (sample).
 * ------------------------------------------------------------------------ */
typedef struct {
  float softcap;         /* cap > 0, from 1e-10 to 1e10; 0: scores are not capped */
  const float* slopes;   /* DEVICE fp32 [H], one finite slope per query head, any sign; NULL: no bias */
  const int32_t* prefix; /* DEVICE int32 [B] (packed: [batch]), or NULL: keys j < prefix[b] are visible to
                            every query of the sequence, as far as the window's left side allows */
} fa_scores;

/*
 * fa_fwd_window with modified scores: key j is visible to query i iff
 * i - window_left <= j and (j <= i + window_right or j < prefix[b]), a negative
 * side being unlimited and `causal` making the right side 0.  Prefix lengths may
 * lie outside [0, S]: they count as the nearer end.  scores == NULL, or all of
 * its parts absent, runs fa_fwd_window.  The window's sides and `causal` hide keys
 * whatever the scores there are.  tanh is evaluated in fp32: beside the product's
 * own error a score is off by at most 2^-20 of itself, or by 2^-21 of cap.
 * Slopes must be finite and slopes[h] * S far below fp32's largest number.  The
 * bias is off by at most 2^-21 of itself, and by up to 2^-15 max(1, slope) for
 * slopes up to 1.04.
 */
fa_status fa_fwd_scores(const void* q, const void* k, const void* v, void* o, float* lse, int64_t B, int64_t H,
                        int64_t H_kv, int64_t S, int64_t D, int causal, int64_t window_left, int64_t window_right,
                        const fa_scores* scores, float scale, fa_dtype dtype, void* stream);

/*
 * Its gradient: dq, dk, dv as fa_bwd_gqa, through the cap's derivative
 * 1 - tanh^2(scale q.k / cap).  Slopes and prefix lengths are constants of the
 * call and get no gradient.  The weights are exp(s - L) of the stored fp32 L: off
 * by up to 2^-20 |L| of themselves, which a negative slope can make much (|L| is
 * about |slopes[h]| * S there; keep it below some thousands).  Workspace: fa_bwd_gqa_workspace_size() bytes.
 */
fa_status fa_bwd_scores(const void* q, const void* k, const void* v, const void* o, const void* dout,
                        const float* lse, void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t H_kv, int64_t S,
                        int64_t D, int causal, int64_t window_left, int64_t window_right, const fa_scores* scores,
                        float scale, fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Both for packed batches (fa_fwd_varlen's layout and checks), with a window
 * inside each sample: documents of a training batch, each its own sequence, with
 * a prefix length each.  What tokens behind the last sample hold, NaN included,
 * has no say.  Workspace of the backward: fa_bwd_varlen_workspace_size() bytes.
 */
fa_status fa_fwd_scores_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                               const int32_t* cu_seqlens, int64_t batch, int64_t max_seqlen, int64_t total, int64_t H,
                               int64_t H_kv, int64_t D, int causal, int64_t window_left, int64_t window_right,
                               const fa_scores* scores, float scale, fa_dtype dtype, void* stream);

fa_status fa_bwd_scores_varlen(const void* q, const void* k, const void* v, const void* o, const void* dout,
                               const float* lse, void* dq, void* dk, void* dv, const int32_t* cu_seqlens,
                               int64_t batch, int64_t max_seqlen, int64_t total, int64_t H, int64_t H_kv, int64_t D,
                               int causal, int64_t window_left, int64_t window_right, const fa_scores* scores,
                               float scale, fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * fa_bwd without a workspace argument, for callers that cannot allocate
 * device memory when they run the backward pass (for example code inside a
 * custom allocator or a fully carved-up memory pool, or a framework that
 * forbids cudaMalloc on its hot path).  The pages describe no such variant:
 * it has no counterpart there.
 *
 * Same arguments and results as fa_bwd minus the workspace.  The scratch row
 * vector D lives in a fixed device array inside the library (8 MiB, held by
 * every GPU that loads the library until the process exits), so
 * B*H*S may not exceed 2^21 rows; larger calls return FA_ERR_UNSUPPORTED.
 * The call allocates nothing: no cudaMalloc, cudaFree or allocating library
 * routine.  Its first call on a device looks up the array's device address
 * (with that device current) and caches it; make that first call before any
 * stream capture.  All calls share the one array and it keeps the last
 * call's contents (each call overwrites the rows it uses before reading
 * them): calls whose work overlaps on the GPU, e.g. on two streams at once,
 * race on it and must be serialised by the caller.
 */
fa_status fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o, const void* dout,
                         const float* lse, void* dq, void* dk, void* dv, int64_t B, int64_t H, int64_t S,
                         int64_t D, int causal, float scale, fa_dtype dtype, void* stream);

/* ------------------------------------------------------------------------
 * Rotary positions and a paged key/value cache.
 *
 * The pages stop at attention itself ("Inside FlashAttention" §6.1 names the
 * packed and grouped interfaces); these calls are what a caller puts around
 * it: positions rotated into Q and K (with their gradient, for training), and,
 * for serving, new tokens appended to a cache of pages and attended to it.
 * Conventions as above unless stated; tokens are packed, [T, heads, D], and
 * cu_seqlens is fa_fwd_varlen's.
 * ------------------------------------------------------------------------ */

/* How inverse frequencies are scaled for contexts longer than `original_len`
 * (fa_rope_inv_freq):
 *   NONE    f_i = base^(-2 i / rot_dim)
 *   LINEAR  f_i / factor
 *   BASE    base * factor^(rot_dim / (rot_dim - 2)) in base's place
 *   PARTS   f_i for pairs that turn more than `fast_turns` times in original_len
 *           positions, f_i / factor for those that turn less than `slow_turns`
 *           times, a linear ramp over the pair index between; the magnitude is
 *           0.1 ln(factor) + 1 (1 for factor <= 1) */
typedef enum { FA_ROPE_NONE = 0, FA_ROPE_LINEAR = 1, FA_ROPE_BASE = 2, FA_ROPE_PARTS = 3 } fa_rope_scaling;

/*
 * HOST helper: the rot_dim / 2 inverse frequencies (radians per position) and
 * the factor on cos and sin.  rot_dim even, >= 2; base > 0; factor > 0 unless
 * scaling is NONE; original_len > 0 and fast_turns > slow_turns > 0 for PARTS.
 * inv_freq: HOST double [rot_dim / 2]; magnitude: HOST, may be NULL.
 */
fa_status fa_rope_inv_freq(int64_t rot_dim, double base, fa_rope_scaling scaling, double factor, double original_len,
                           double fast_turns, double slow_turns, double* inv_freq, float* magnitude);

/*
 * HOST helper: each finite inverse frequency as a phase step, inv_freq / 2 pi
 * turns in units of 2^-64 turns, modulo one turn.  A caller copies the n steps
 * to the device once.  position * step mod 2^64 is then the angle's fraction of
 * a turn without loss at any position.  inv_freq, steps: HOST arrays [n].
 */
fa_status fa_rope_steps(const double* inv_freq, int64_t n, uint64_t* steps);

/*
 * Rotates the first rot_dim columns of every row of q [T, H, D] and k
 * [T, H_kv, D] by its token's position.  Pair i of a row is columns
 * (i, rot_dim / 2 + i), or (2 i, 2 i + 1) when `interleaved`; with
 * t = positions[token] * inv_freq[i] it becomes
 *   (m (a cos t - b sin t), m (b cos t + a sin t)),  m = magnitude.
 * Columns from rot_dim on pass unchanged.  Arithmetic in fp32, rounded once.
 *   q_stride, ... : elements between tokens (heads and columns are dense), a
 *                   multiple of 8 and at least heads * D, so q and k may be
 *                   slices of one projection; H or H_kv may be 0 (its pointers
 *                   are then not used).
 *   q_out, k_out  : outputs; in place (q_out = q with the same stride) is
 *                   allowed, any other overlap of rows is not.
 *   positions     : DEVICE int32 [T], any sign;  steps: DEVICE uint64 [rot_dim / 2].
 * rot_dim even, 2 .. D.  T = 0 or H = H_kv = 0 is an empty call.
 */
fa_status fa_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, void* q_out,
                  int64_t q_out_stride, void* k_out, int64_t k_out_stride, const int32_t* positions,
                  const uint64_t* steps, int64_t total, int64_t H, int64_t H_kv, int64_t D, int64_t rot_dim,
                  int interleaved, float magnitude, fa_dtype dtype, void* stream);

/* Gradient of fa_rope: dq, dk [T, heads, D] from the gradients of its outputs.
 * The rotation is linear, so this is the rotation by -t, times m; the same
 * arguments otherwise (dq_out, dk_out are read; dq, dk are written). */
fa_status fa_rope_bwd(const void* dq_out, int64_t dq_out_stride, const void* dk_out, int64_t dk_out_stride, void* dq,
                      int64_t dq_stride, void* dk, int64_t dk_stride, const int32_t* positions,
                      const uint64_t* steps, int64_t total, int64_t H, int64_t H_kv, int64_t D, int64_t rot_dim,
                      int interleaved, float magnitude, fa_dtype dtype, void* stream);

/*
 * A paged key/value cache.  Key j of sequence b, head g is the D elements at
 *   k + block_table[b][j / page_size] * page_stride + (j % page_size) * row_stride + g * head_stride,
 * its value likewise from v.  page_size is a power of two, 16 or more; strides
 * are in elements, shared by k and v, multiples of 8, and leave rows apart
 * (pages, rows and heads in any order of nesting).
 *   block_table : DEVICE int32, rows of table_pages entries (0: table_stride
 *                 of them), table_stride entries apart, so it may be a slice of a
 *                 wider table; entries past a sequence's last page, and of
 *                 pages no query can see, are not used and may hold anything.
 *   kv_lens     : DEVICE int32 [batch], keys of each sequence INCLUDING the
 *                 call's new tokens, so token i of the n new ones is key
 *                 kv_lens[b] - n + i.
 * Lengths and entries are checked on the device: a length below 0, beyond the
 * call's bound or the block table's row, or (append) below n leaves that
 * sequence alone, an entry in use outside [0, num_pages) is read as zeros and
 * never written; both make fa_check_device_errors() return FA_ERR_INVALID_ARG.
 */
typedef struct {
  void* k;
  void* v;
  const int32_t* block_table;
  const int32_t* kv_lens;
  int64_t table_stride, table_pages;
  int64_t num_pages, page_size;
  int64_t page_stride, row_stride, head_stride;
} fa_paged_cache;

/*
 * Appends the new tokens' K and V rows to the cache (the slots above must be
 * there already), rotating K, and rotates Q on the way, in one launch:
 *   q, k, v     : [T, H, D], [T, H_kv, D] with token strides as in fa_rope;
 *   q_out       : rotated Q; H = 0 leaves Q alone (q, q_out not used);
 *   positions   : DEVICE int32 [T], or NULL: a token's position is its key index;
 *   steps       : DEVICE uint64 [rot_dim / 2]; rot_dim = 0 (steps not used)
 *                 appends K as it is and copies Q;
 *   max_seqlen  : host bound on the new tokens of a sequence; may be loose.
 * Two new tokens must not share a slot.  Where offsets decrease, other sequences
 * of the call may be left alone beside the one that is reported.  Other slots and rows of tokens that no
 * sequence covers are left as they were.
 */
fa_status fa_paged_append(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k,
                          int64_t k_stride, const void* v, int64_t v_stride, const fa_paged_cache* cache,
                          const int32_t* cu_seqlens, const int32_t* positions, const uint64_t* steps, int64_t batch,
                          int64_t max_seqlen, int64_t total, int64_t H, int64_t H_kv, int64_t D, int64_t rot_dim,
                          int interleaved, float magnitude, fa_dtype dtype, void* stream);

/*
 * Attention of each sequence's new tokens over its cache: one token
 * (decoding), a few, or a chunk of a prompt, mixed in one call.
 *   q, o        : [T, H, D];  lse : [H, T] fp32 (as fa_fwd_varlen).
 *   Query i of the n new tokens of sequence b stands at key position
 *   p = kv_lens[b] - n + i and sees keys j < kv_lens[b] with
 *   p - window_left <= j <= p + window_right (a negative side is unlimited;
 *   `causal` makes the right side 0): the causal diagonal ends at the last key.
 *   A row that sees no key gets O = 0, L = -inf.
 *   H is a positive multiple of H_kv, at most 128 query heads to a K/V head.
 *   max_seqlen_q, max_seqlen_k : host bounds on the new tokens and on kv_lens
 *   (at most 2^29).  They may be loose: `total` and the block table's row bound
 *   the lengths too.  Too large for the library (FA_ERR_UNSUPPORTED) is a call
 *   whose sequences, each as long as these bounds allow, have more than 2^30
 *   tiles of query rows or 2^37 blocks of keys over all tiles and heads; batch *
 *   min(max_seqlen_q, total) <= 2^30 and that times H_kv * (min(max_seqlen_k,
 *   the row's keys) / 64 + 2) <= 2^37 is always supported.
 *   workspace   : fa_fwd_paged_workspace_size() bytes, 256-byte aligned, for the
 *   partials of sequences that several CTAs share; its contents on entry do not
 *   matter, and calls that may overlap on the GPU need one each.
 * Cached keys no row sees (past the end, before the window) may hold anything,
 * NaN included.  A NaN in a query, or in a key that it sees, makes that row's
 * O and L NaN.  A NaN or infinity in V at a key some row sees reaches that
 * row, and may reach other rows of the call that share the K/V head.
 * Rounding: as in the other forward calls, the probabilities (relative to the
 * row's running maximum) are rounded to the inputs' type for the product with V,
 * and O once at the end; products, sums, maxima and partials are fp32.
 * The result depends on the lengths and bounds, not on timing: repeated calls
 * give the same bits.
 */
fa_status fa_fwd_paged(const void* q, void* o, float* lse, const fa_paged_cache* cache, const int32_t* cu_seqlens,
                       int64_t batch, int64_t max_seqlen_q, int64_t max_seqlen_k, int64_t total, int64_t H,
                       int64_t H_kv, int64_t D, int causal, int64_t window_left, int64_t window_right, float scale,
                       fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * fa_fwd_paged with modified scores (positions are the key positions); their
 * prefix must be NULL (a prefix's own chunk sees all of it with causal = 0).
 */
fa_status fa_fwd_paged_scores(const void* q, void* o, float* lse, const fa_paged_cache* cache,
                              const int32_t* cu_seqlens, int64_t batch, int64_t max_seqlen_q, int64_t max_seqlen_k,
                              int64_t total, int64_t H, int64_t H_kv, int64_t D, int causal, int64_t window_left,
                              int64_t window_right, const fa_scores* scores, float scale, fa_dtype dtype,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * Attention of drafted tokens that form a tree (several continuations of a
 * sequence, to be verified at once) over the cache.  The n new tokens of sequence
 * b, already in the cache, are keys f .. kv_lens[b] - 1, f = kv_lens[b] - n, in any
 * order that the caller's tree has.  New token i sees the keys j < f with
 * positions[i] - window_left <= j (negative: all), and of the new tokens those
 * whose bit is set in its row: new token j is bit j % 32 of word j / 32.  (Itself
 * and its ancestors, as a rule; no bit is implied.)  A row that sees no key gets
 * O = 0, L = -inf.
 *   positions   : DEVICE int32 [T], where each new token stands in its sequence
 *                 (f plus its depth, as a rule): the window's and the bias's i,
 *                 and the bias's j of a new token as a key.  Held to
 *                 [f, kv_lens[b] - 1].  (With kv_lens[b] < n the first new
 *                 tokens, which would stand before key 0, are no keys.)
 *   tree        : DEVICE uint32, the rows of the T new tokens, tree_stride words
 *                 apart; tree_words (at most tree_stride) words of a row are
 *                 used, 32 * tree_words >= min(max_seqlen_q, total).  Bits past a
 *                 sequence's new tokens are not used.
 *   scores      : as in fa_fwd_paged_scores, or NULL.
 * Everything else, the workspace too, is fa_fwd_paged's.
 */
fa_status fa_fwd_paged_tree(const void* q, void* o, float* lse, const fa_paged_cache* cache,
                            const int32_t* cu_seqlens, const int32_t* positions, const uint32_t* tree,
                            int64_t tree_stride, int64_t tree_words, int64_t batch, int64_t max_seqlen_q,
                            int64_t max_seqlen_k, int64_t total, int64_t H, int64_t H_kv, int64_t D,
                            int64_t window_left, const fa_scores* scores, float scale, fa_dtype dtype,
                            void* workspace, size_t workspace_bytes, void* stream);

/*
 * Keeps the accepted path of each sequence's drafted tree: of the n new tokens at
 * keys f .. kv_lens[b] - 1, f = kv_lens[b] - n, token path[b][i] (K and V rows of
 * all heads) moves to key f + i, i < path_lens[b].  The caller then shortens
 * kv_lens[b] to f + path_lens[b].  kv_lens and cu_seqlens are those that the trees
 * were attended to with.
 *   path       : DEVICE int32, rows of path_cols entries, path_stride apart; the
 *                first path_lens[b] of a row are used, increase strictly and lie
 *                in [0, n) (a parent precedes its children).
 *   path_lens  : DEVICE int32 [batch], 0 .. min(n, path_cols).
 *   max_seqlen : host bound on the new tokens of a sequence; may be loose.
 * A path that is longer, or does not increase within [0, n), leaves its sequence
 * alone, and so do lengths that contradict the call; a row of an entry that is no
 * page is read as zeros and never written; each makes fa_check_device_errors()
 * return FA_ERR_INVALID_ARG.  Slots from f + path_lens[b] on, and other sequences',
 * are left as they were.  Sequences must not share the pages of their new keys.
 */
fa_status fa_paged_keep(const fa_paged_cache* cache, const int32_t* cu_seqlens, const int32_t* path,
                        int64_t path_stride, int64_t path_cols, const int32_t* path_lens, int64_t batch,
                        int64_t max_seqlen, int64_t H_kv, int64_t D, fa_dtype dtype, void* stream);

/* Workspace bytes of fa_fwd_paged (0 for an empty call or one that no `total`
 * makes supported); never less for larger max_seqlen_q or max_seqlen_k. */
size_t fa_fwd_paged_workspace_size(int64_t batch, int64_t max_seqlen_q, int64_t max_seqlen_k, int64_t H,
                                   int64_t H_kv, int64_t D);

/* Static, human-readable name of a status code. */
const char* fa_status_string(fa_status status);

/* One-line description of the last failure on the calling thread ("" if none). */
const char* fa_last_error_detail(void);

/*
 * Synchronises `stream`, then reads and clears the device error word that the
 * kernels set when a pipeline wait times out, or a packed batch's cu_seqlens
 * or a paged cache's lengths or block table contradict the call.  Returns
 * FA_ERR_TIMEOUT or FA_ERR_INVALID_ARG (the latter for cu_seqlens and the
 * cache) if it was set, FA_ERR_CUDA if the synchronisation
 * failed, else FA_OK.  Meant for
 * tests and debugging; the compute entry points never synchronise.
 */
fa_status fa_check_device_errors(void* stream);

/*
 * Sets the time limit, in nanoseconds, of every pipeline wait in the kernels
 * launched after this call (a wait on a barrier that another warp of the same
 * CTA completes: operands landed, scores computed, a stage freed).  0 restores
 * the default of 2 s.  Returns the previous limit.  Process-wide, not tied to
 * a stream or device.  A wait that runs past its limit makes its CTA stop
 * early: it drains its own copies and MMAs (those waits keep the 2 s limit),
 * frees its tensor memory and exits, and fa_check_device_errors() returns
 * FA_ERR_TIMEOUT; the outputs of that call are then undefined.  A limit far
 * below the kernels' own latencies (nanoseconds) makes that happen on purpose,
 * which is how the tests exercise this path.  Not part of the pages' interface:
 * failure handling for callers that must not hang.
 */
uint64_t fa_set_wait_limit_ns(uint64_t ns);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_H */
