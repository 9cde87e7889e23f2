/*
 * rlk.h -- C-ABI of the layout-invariant selected-token logprob ("strict-path
 * linear logprob") for NVIDIA GB300 (sm_103a).
 *
 * What it computes.  For each token t of a batch, with bf16 hidden state
 * h[t, :] and bf16 output-head weights W[v, :] over the whole vocabulary,
 *
 *     lse[t]     = log sum_v exp(h[t] . W[v])
 *     logprob[t] = h[t] . W[target[t]] - lse[t]
 *
 * ("vLLM RL-Kernel v0.1.0: ROCm 上でのビット単位のトレーニング-ロールアウト一貫性",
 * strict-path boundary table, row "Linear logprob": actual vocabulary range,
 * target ownership, local reduction, cross-rank LSE merge; the blog on
 * bitwise consistency with RL-Kernel + vime on AMD, section 3.1: log_softmax
 * read at the target, whose max and sum reductions fix the last bits).
 *
 * The numeric contract "rlk-linlogp-v1" fixes every reduction, merge order,
 * precision, rounding point and primitive (the same page, section
 * 数値実行契約), so a token's two results are bit-identical whatever batch it
 * sits in (1-row decode or a packed batch), whatever its row position, and
 * however the vocabulary is split into tree-aligned shards:
 *
 *   - logits are fp32 tensor-core dot products of bf16 inputs, K ascending in
 *     steps of 16, one accumulator, never split over K, never rounded to bf16;
 *   - the vocabulary is cut into tiles of 128 columns; each tile gives
 *     (m, s) = (max logit, pairwise-tree sum of exp(logit - m)) for its real
 *     columns (a last, shorter tile simply has fewer columns);
 *   - tiles merge along one fixed tree (recursive bisection of the tile
 *     index range, lower half taking the extra tile) with
 *     merge(L, R) = (hi.m, fma(lo.s, exp(lo.m - hi.m), hi.s)), hi = the
 *     operand with the larger m, L on a tie;
 *   - n_shards (1, 2, 4 or 8) shards are the nodes of that tree at depth
 *     log2(n_shards), so shard records merged in shard order give the same
 *     bits as the unsharded call;
 *   - lse = RN(m + log(s)), logprob = RN(target logit - lse);
 *   - exp and log are the library's own (Cody-Waite + degree-7 Taylor; atanh
 *     series), not the CUDA math library's.
 *
 * Conventions for every call below.
 *   - Pointers named as device pointers must point to device memory of the
 *     current CUDA device; the caller owns every buffer.  The library keeps
 *     no per-call state and allocates no device memory.
 *   - A workspace serves one call at a time: calls that may overlap on the
 *     GPU (on unordered streams, or in graphs replayed side by side) need
 *     one each.  Outputs must not overlap inputs, other outputs or the
 *     workspace except where a call says so.
 *   - Calls are asynchronous and stream-ordered on `stream` (NULL = legacy
 *     default stream); outputs are valid once the stream reaches them.
 *   - Host-detectable errors are returned before anything is launched.
 *   - Device-detected errors are OR-ed into *dev_status (a device int32 the
 *     caller zeroes; may be NULL) as bit (1 << code): RLK_ERR_TARGET_RANGE
 *     for an active row whose target no shard owns (that row's outputs are
 *     NaN), RLK_ERR_TIMEOUT if a pipeline wait ran out (outputs undefined;
 *     the kernel returns instead of hanging), RLK_ERR_INVALID_ARG for
 *     sequence offsets that do not ascend within [0, T], RLK_ERR_NONFINITE
 *     for a gradient norm that is not finite.
 *   - T == 0 is a no-op returning RLK_OK (the losses and sums of the
 *     training-step calls still get their value for no tokens, 0); T < 0 or T > RLK_MAX_ROWS returns
 *     RLK_ERR_INVALID_ARG (kernels index rows in 32 bits and step past
 *     the last row by less than 2^20).
 *   - Inactive rows (active_mask[t] == 0) give out_logprob = out_lse = 0 and
 *     all-zero partial records; their hidden row and target are never used
 *     in any other row's result.  active_mask == NULL means all active.
 *   - Only sm_103 devices are supported; anything else returns
 *     RLK_ERR_UNSUPPORTED.  There is no fallback path.
 */
#ifndef RLK_H_
#define RLK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same handle type as cudaStream_t. */
struct CUstream_st;
typedef struct CUstream_st* rlk_stream_t;

typedef enum rlk_status {
    RLK_OK = 0,
    RLK_ERR_INVALID_ARG = 1,   /* null pointer, negative size, T > RLK_MAX_ROWS, bad shard index */
    RLK_ERR_UNSUPPORTED = 2,   /* device not sm_103; H % 64 != 0 or H > 2^20; V > 262144; n_shards not in {1,2,4,8} or > tiles */
    RLK_ERR_ALIGNMENT = 3,     /* hidden/W not 16-byte aligned, workspace not 256-byte aligned */
    RLK_ERR_WORKSPACE = 4,     /* workspace smaller than rlk_workspace_size() */
    RLK_ERR_CUDA = 5,          /* a CUDA runtime/driver call failed (launch, device query) */
    RLK_ERR_TARGET_RANGE = 6,  /* device-detected: active row whose target no shard owns */
    RLK_ERR_TIMEOUT = 7,       /* device-detected: a bounded pipeline wait gave up */
    RLK_ERR_NONFINITE = 8      /* device-detected: the gradient norm is infinite or NaN, or a row
                                * to draw a token from is no distribution */
} rlk_status_t;

/* Per-token record of one vocabulary shard (16 bytes). */
typedef struct rlk_partial {
    float m;          /* max logit over the shard's vocabulary range */
    float s;          /* sum of exp(logit - m) over the range, merged along the tile tree */
    float tgt;        /* the target's logit if this shard owns the target, else 0 */
    uint32_t owned;   /* 1 if target lies in [v_begin, v_end) of this shard, else 0 */
} rlk_partial_t;

#define RLK_VOCAB_TILE 128
#define RLK_MAX_SHARDS 8
#define RLK_MAX_VOCAB 262144          /* 2048 tiles */
#define RLK_K_BLOCK 64                /* H must be a multiple of this */
#define RLK_MAX_ROWS 2146435072       /* 2^31 - 2^20: the largest T (rows) any call takes */
#define RLK_DTYPE_F32 0               /* logits element types for the materialised-logits calls */
#define RLK_DTYPE_BF16 1
#define RLK_DTYPE_F16 2               /* gradients of rlk_grad_norm and rlk_grad_clip only */

/* "rlk-linlogp-v1": names the numeric contract above. */
const char* rlk_contract_id(void);

/* Build fingerprint: source revision, nvcc version, arch and contract flags. */
const char* rlk_build_fingerprint(void);

/* Human-readable name of a status code. */
const char* rlk_status_string(int status);

/*
 * Vocabulary range [*v_begin, *v_end) of shard `shard` of `n_shards`: the
 * shard-th node at depth log2(n_shards) of the tile tree, in vocabulary ids
 * (the strict-path table's "actual vocabulary range").  Host only.
 * Errors: RLK_ERR_INVALID_ARG (null outputs, V < 1, shard out of range),
 * RLK_ERR_UNSUPPORTED (bad n_shards, V > RLK_MAX_VOCAB).
 */
rlk_status_t rlk_shard_range(int64_t V, int n_shards, int shard, int64_t* v_begin, int64_t* v_end);

/*
 * Bytes of device workspace rlk_linear_logprob needs for (T, V, n_shards);
 * it also covers rlk_linear_logprob_shard for any shard of that split.
 * Layout (each part 256-byte aligned): per-tile (m, s) float pairs [T][tiles],
 * target logits float [T], shard records rlk_partial_t [n_shards][T].
 * Returns 0 for invalid arguments.
 */
size_t rlk_workspace_size(int64_t T, int64_t V, int n_shards);

/*
 * Full selected-token logprob of T tokens over V vocabulary entries,
 * vocabulary split into n_shards tree-aligned shards merged in shard order
 * on this device (the boundary table's local reduction + cross-rank LSE
 * merge, with the ranks emulated as shards).  The per-shard records are
 * left in the workspace's record area.
 *
 *   hidden       device, bf16 [T][H] row-major, 16-byte aligned
 *   W            device, bf16 [V][H] row-major (vocabulary rows), 16-byte aligned
 *   targets      device, int32 [T], global vocabulary ids
 *   active_mask  device, uint8 [T] (nonzero = active) or NULL
 *   H            multiple of 64, at most 2^20
 *   V            1 .. RLK_MAX_VOCAB
 *   n_shards     1, 2, 4 or 8, and at most ceil(V / 128)
 *   out_logprob  device, float [T];  out_lse  device, float [T]
 *   workspace    device, 256-byte aligned, >= rlk_workspace_size(T, V, n_shards) bytes
 *   dev_status   device int32 or NULL (see conventions)
 */
rlk_status_t rlk_linear_logprob(const void* hidden, const void* W, const int32_t* targets,
                                const uint8_t* active_mask, int64_t T, int64_t H, int64_t V,
                                int n_shards, float* out_logprob, float* out_lse,
                                void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                rlk_stream_t stream);

/*
 * The part one vocabulary shard (one emulated TP rank) computes: its record
 * (m, s, tgt, owned) per token from its own weight rows only.
 *
 *   W_shard      device, bf16 rows [v_begin, v_end) of the full W (see
 *                rlk_shard_range), [v_end - v_begin][H] row-major, 16-byte aligned
 *   targets      global vocabulary ids; ownership is target in [v_begin, v_end)
 *   V_total      the full vocabulary size (defines the tile tree)
 *   out_partial  device, rlk_partial_t [T]
 *   workspace    >= rlk_workspace_size(T, v_end - v_begin, 1) bytes
 * Other arguments as rlk_linear_logprob.
 */
rlk_status_t rlk_linear_logprob_shard(const void* hidden, const void* W_shard,
                                      const int32_t* targets, const uint8_t* active_mask,
                                      int64_t T, int64_t H, int64_t V_total, int n_shards,
                                      int shard, rlk_partial_t* out_partial, void* workspace,
                                      size_t workspace_bytes, int32_t* dev_status,
                                      rlk_stream_t stream);

/*
 * Cross-shard LSE merge in fixed shard order (the boundary table's
 * "cross-rank LSE merge" and the distributed-aggregation row's fixed rank
 * reduction order): records merge pairwise (0,1),(2,3),... then pairs of
 * those; the target logit comes from the one owning shard.
 *
 *   partials     HOST array of n_shards DEVICE pointers, each rlk_partial_t [T], shard order
 *   n_shards     1, 2, 4 or 8
 *   out_logprob, out_lse  device, float [T]
 * An active row with no owning shard, or with more than one, gets NaN and
 * sets RLK_ERR_TARGET_RANGE in *dev_status.
 * The records may come from other processes: with the vocabulary split over
 * n ranks (rank r holding shard r's W rows and calling
 * rlk_linear_logprob_shard), gathering every rank's records in rank order and
 * merging them here on each rank gives every rank the unsharded call's bits.
 */
rlk_status_t rlk_lse_merge(const rlk_partial_t* const* partials, int n_shards, int64_t T,
                           const uint8_t* active_mask, float* out_logprob, float* out_lse,
                           int32_t* dev_status, rlk_stream_t stream);

/*
 * The two stages of rlk_linear_logprob as separate calls (same kernels,
 * same bits), so a caller can time or overlap them:
 *   rlk_tile_partials: logits GEMM + fused per-tile (m, s) and target pick,
 *                      into the workspace;
 *   rlk_tile_merge:    tile tree, shard records, final lse/logprob.
 * Arguments mean what they mean for rlk_linear_logprob; the workspace must
 * be the same buffer for both calls.
 */
rlk_status_t rlk_tile_partials(const void* hidden, const void* W, const int32_t* targets,
                               const uint8_t* active_mask, int64_t T, int64_t H, int64_t V,
                               int n_shards, void* workspace, size_t workspace_bytes,
                               int32_t* dev_status, rlk_stream_t stream);
rlk_status_t rlk_tile_merge(const int32_t* targets, const uint8_t* active_mask, int64_t T,
                            int64_t V, int n_shards, float* out_logprob, float* out_lse,
                            void* workspace, size_t workspace_bytes, int32_t* dev_status,
                            rlk_stream_t stream);

/*
 * Diagnostic: the fp32 logits [T][V] exactly as the fused path sees them
 * (same kernel mainloop, the epilogue stores the accumulator instead of
 * reducing it).  out_logits: device, float [T][V] row-major.  Meant for
 * tests and for locating a divergence (the blog's advice to dump the
 * intermediate values, section 5.2).
 */
rlk_status_t rlk_debug_logits(const void* hidden, const void* W, int64_t T, int64_t H, int64_t V,
                              float* out_logits, int32_t* dev_status, rlk_stream_t stream);

/*
 * Diagnostic: evaluates one of the contract's primitives on the GPU over the
 * fp32 bit patterns [first, first + count) and writes
 *   sum_i (bits(f(x_i)) + 0x9E3779B9) * (2 i + 1)   (mod 2^64)
 * to *out_hash, so a caller can compare the device's primitive with another
 * implementation of the contract over a whole input range (any single
 * differing output changes the sum).  The primitives are the contract's
 * fixed exp, log and rsqrt ("vLLM RL-Kernel v0.1.0: ROCm 上でのビット単位の
 * トレーニング-ロールアウト一貫性", section 数値実行契約, item 6: the math
 * primitives are part of the contract); the check itself has no counterpart
 * in the pages.
 *   which     0: rlk_exp; 1: rlk_exp evaluated two values per instruction (the
 *             kernels' packed form; must equal 0); 2: rlk_log; 3: rlk_rsqrt
 *   first, count  first bit pattern and how many; first + count <= 2^32
 *   out_hash  device, one uint64_t, overwritten
 * Errors: RLK_ERR_INVALID_ARG for an unknown primitive, a range beyond 2^32
 * or a null out_hash; otherwise as the other calls.
 */
rlk_status_t rlk_debug_primitive_hash(int which, uint32_t first, uint64_t count,
                                      uint64_t* out_hash, rlk_stream_t stream);

/*
 * Selected-token logprob from logits that already exist in memory, under
 * the same contract (the blog's rl_kernel.log_softmax with a fixed reduction
 * tree, sections 4.2-4.3, read at the target).  Given the fp32 logits the
 * fused path computes (rlk_debug_logits), it returns the fused path's bits.
 *
 *   logits       device, [T][ld] row-major, elements RLK_DTYPE_F32 or RLK_DTYPE_BF16
 *                (bf16 widens exactly to fp32); only columns [0, V) are read
 *   ld           row stride in elements, >= V; logits aligned to their element
 *                size (when every row starts on a 16-byte boundary -- a 16-byte
 *                aligned base and ld * element size a multiple of 16 -- rows
 *                are copied in 16-byte pieces; the values and results are the
 *                same either way)
 *   workspace    >= rlk_workspace_size(T, V, n_shards) bytes, same layout as rlk_linear_logprob
 * Other arguments, outputs and errors as rlk_linear_logprob.
 */
rlk_status_t rlk_logits_logprob(const void* logits, int logits_dtype, int64_t ld,
                                const int32_t* targets, const uint8_t* active_mask, int64_t T,
                                int64_t V, int n_shards, float* out_logprob, float* out_lse,
                                void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                rlk_stream_t stream);

/*
 * Full log_softmax of materialised logits: out[t][v] = RN(l[t][v] - lse[t])
 * with lse from the contract's tile tree; out_lse[t] = lse[t].  Inactive rows
 * give zeros.  The same tree gives the same lse bits as rlk_linear_logprob.
 *
 *   out          device, float [T][V] row-major (dense, V columns)
 *   out_lse      device, float [T]
 *   workspace    >= rlk_workspace_size(T, V, 1) bytes
 * logits, logits_dtype, ld as rlk_logits_logprob.
 */
rlk_status_t rlk_log_softmax(const void* logits, int logits_dtype, int64_t ld,
                             const uint8_t* active_mask, int64_t T, int64_t V, float* out,
                             float* out_lse, void* workspace, size_t workspace_bytes,
                             int32_t* dev_status, rlk_stream_t stream);

/*
 * Backward of sum_t grad_logprob[t] * logprob[t] (the blog's requirement,
 * sections 3.3 and 4.2, that the kernel provide a backward with the same
 * numeric discipline as its forward):
 *
 *   G[t, v]        = bf16_RN(RN(g_t * d)), d = RN(1 - p) at the target, -p elsewhere,
 *                    p = rlk_exp(RN(logit[t, v] - lse[t])), from the same fp32 logits
 *   grad_hidden    = G · W   (fp32; the sum over v in 8 fixed ranges of ascending
 *                    vocabulary, each one accumulator, added pairwise in fixed order;
 *                    a token's row does not depend on the rest of the batch)
 *   grad_W         = Gᵀ · h  (fp32; the sum over t ascending in one accumulator)
 *
 *   lse           device, float [T]: the forward's out_lse for this batch
 *   grad_logprob  device, float [T]: dL/dlogprob
 *   grad_hidden   device, float [T][H], or NULL to skip
 *   grad_W        device, float [V][H], or NULL to skip (at least one is required)
 *   workspace     >= rlk_backward_workspace_size(T, H, V) bytes, 256-byte aligned
 *                 (holds G as bf16 [T][roundup(V, 8)] at offset 0)
 * Inactive rows contribute nothing (their G row is zero).  An active row
 * whose target lies outside [0, V) sets RLK_ERR_TARGET_RANGE and gets no
 * one-hot term.  Other arguments as rlk_linear_logprob.
 * When both gradients are asked for, grad_hidden's fixed-order split sum
 * runs beside the grad_W GEMM on a library stream, forked from `stream`
 * after grad_hidden's GEMM and joined back before the call's work on
 * `stream` ends (events; capturable in a CUDA graph).  The first such call
 * on a device creates that stream and its two events; they live for the
 * process.
 */
size_t rlk_backward_workspace_size(int64_t T, int64_t H, int64_t V);
rlk_status_t rlk_linear_logprob_backward(const void* hidden, const void* W,
                                         const int32_t* targets, const uint8_t* active_mask,
                                         const float* grad_logprob, const float* lse, int64_t T,
                                         int64_t H, int64_t V, float* grad_hidden, float* grad_W,
                                         void* workspace, size_t workspace_bytes,
                                         int32_t* dev_status, rlk_stream_t stream);

/*
 * Training pair that trades memory for the backward's second logits GEMM:
 * rlk_linear_logprob_save_logits is rlk_linear_logprob (same outputs, same
 * bits) that also stores every row's fp32 logits (the exact accumulator
 * values the epilogue reduces), and rlk_linear_logprob_backward_from_logits
 * forms G from those stored logits instead of recomputing them, then runs
 * the same two GEMMs: its grad_hidden and grad_W have the bits of
 * rlk_linear_logprob_backward on the same batch.  Same backward definition
 * as above (the blog's sections 3.3 and 4.2).
 *
 *   logits       device, float [T][ld_logits] row-major; written by the
 *                forward (columns [0, V) of every row below T, active or
 *                not), read by the backward; 16-byte aligned, ld_logits a
 *                multiple of 4 and >= V (else RLK_ERR_ALIGNMENT /
 *                RLK_ERR_INVALID_ARG); T * ld_logits * 4 bytes, owned by the
 *                caller (2.49 GB at T = 4096, V = 151936)
 * Forward: other arguments, outputs and errors as rlk_linear_logprob.
 * Backward: other arguments, outputs and errors as rlk_linear_logprob_backward
 * (hidden and W are still read: the GEMMs need them).
 */
rlk_status_t rlk_linear_logprob_save_logits(const void* hidden, const void* W,
                                           const int32_t* targets, const uint8_t* active_mask,
                                           int64_t T, int64_t H, int64_t V, int n_shards,
                                           float* out_logprob, float* out_lse, float* logits,
                                           int64_t ld_logits, void* workspace,
                                           size_t workspace_bytes, int32_t* dev_status,
                                           rlk_stream_t stream);
rlk_status_t rlk_linear_logprob_backward_from_logits(
    const float* logits, int64_t ld_logits, const void* hidden, const void* W,
    const int32_t* targets, const uint8_t* active_mask, const float* grad_logprob,
    const float* lse, int64_t T, int64_t H, int64_t V, float* grad_hidden, float* grad_W,
    void* workspace, size_t workspace_bytes, int32_t* dev_status, rlk_stream_t stream);

/*
 * Strict RMSNorm producing the hidden states the head consumes (the
 * strict-path table's "RMSNorm" row: reduction domain, epsilon, residual
 * add, output boundary).  Per row:
 *   x'   = bf16_RN(RN(x + residual))          (x itself when residual is NULL)
 *   s    = pairwise tree over nextpow2(H) feature slots of x'_i^2 (fp32)
 *   rstd = rlk_rsqrt(RN(RN(s / H) + eps))      (the library's own rsqrt)
 *   out  = bf16_RN(RN(RN(x'_i * rstd) * gamma_i))
 * A row's result does not depend on the batch around it.
 *
 *   x, residual  device, bf16 [T][H] (residual may be NULL), 16-byte aligned
 *   gamma        device, bf16 [H]
 *   eps          > 0
 *   out          device, bf16 [T][H]
 *   residual_out device, bf16 [T][H] receiving x' (the next residual stream), or NULL;
 *                requires residual
 * out may be x and residual_out may be residual (updated in place): every
 * element is read before it is written.  No other overlap is allowed.
 *   H            multiple of 64, at most 8192
 */
rlk_status_t rlk_rmsnorm(const void* x, const void* residual, const void* gamma, float eps,
                         int64_t T, int64_t H, void* out, void* residual_out, rlk_stream_t stream);

/*
 * Backward of rlk_rmsnorm: with x the row that was normalised (rlk_rmsnorm's
 * residual_out where it added a residual, its x where it did not) and rstd the
 * forward's own (same tree, same rsqrt, same bits), per row
 *   up_i    = grad_out_i * gamma_i
 *   c       = rstd^2 / H * sum_i up_i * x_i           (fp32, chains of 8, then a tree)
 *   grad_x_i = rstd * (up_i - x_i * c) + grad_residual_i
 *   grad_gamma_i = sum over the rows of grad_out_i * x_i * rstd
 * in fp32, each grad_x element rounded once to its type.  grad_residual is
 * the gradient that reached residual_out from further on (NULL where there
 * is none); grad_x is then the gradient of both x and residual.  A row's
 * grad_x does not depend on the batch around it; grad_gamma is summed over
 * ranges of consecutive rows, in chains of 64 rows, and then over the ranges,
 * in an order that T, H and the types fix.
 * (The blog's sections 3.3 and 4.2 ask for a backward with the forward's
 * numeric discipline; the strict-path table's "RMSNorm" row.)
 *
 *   grad_out       device, [T][H] of grad_out_dtype (RLK_DTYPE_F32 -- rlk_linear_logprob_backward's
 *                  grad_hidden -- or RLK_DTYPE_BF16)
 *   x, gamma       device, bf16 [T][H] and [H]
 *   eps            as in the forward, and a normal number (2^-126 or more)
 *   grad_residual  device, [T][H] of grad_x_dtype, or NULL
 *   grad_x         device, [T][H] of grad_x_dtype (RLK_DTYPE_F32 or RLK_DTYPE_BF16); may be
 *                  grad_residual, or grad_out where the types are the same
 *   grad_gamma     device, float [H], or NULL to skip; all zeros when T == 0
 *   workspace      >= rlk_rmsnorm_backward_workspace_size(T, H) bytes, 256-byte aligned; that
 *                  is 0 for T <= 16, and nothing is needed when grad_gamma is NULL
 *   H              multiple of 64, at most 8192; every pointer 16-byte aligned
 */
size_t rlk_rmsnorm_backward_workspace_size(int64_t T, int64_t H);
rlk_status_t rlk_rmsnorm_backward(const void* grad_out, int grad_out_dtype, const void* x,
                                  const void* gamma, float eps, const void* grad_residual,
                                  int64_t T, int64_t H, void* grad_x, int grad_x_dtype,
                                  float* grad_gamma, void* workspace, size_t workspace_bytes,
                                  rlk_stream_t stream);

/*
 * Clipped policy loss with a KL term, and its gradient with respect to the
 * new log-probabilities, over packed sequences (the reinforcement-learning
 * step that the pages' strict path serves: vime's trainer compares the
 * rollout's logprobs with the training side's).  Per active token, with
 * d = logprob - old_logprob, r = e^d and A its advantage:
 *   s = min(r A, clamp(r, 1 - clip_low, 1 + clip_high) A)
 *   s = max(s, dual_clip A)                    where dual_clip > 0 and A < 0
 *   k = d' (k1), d'^2 / 2 (k2) or e^-d' - 1 + d' (k3), d' = logprob - ref_logprob
 *   loss   = scale * sum_t w_t (-s_t + kl_coef k_t)
 *   grad_t = scale * w_t (-(r A where s follows r, else 0) + kl_coef dk/dlogprob)
 * with w_t = 1 (RLK_REDUCE_SUM), 1 / (active tokens) (RLK_REDUCE_TOKEN_MEAN)
 * or 1 / (n_seqs * active tokens of t's sequence) (RLK_REDUCE_SEQ_MEAN; a
 * sequence without active tokens adds 0 and still counts).  Whether a token
 * is clipped is decided on the exact d, not on a rounded ratio.
 *
 * A token takes part if its mask is nonzero and it lies in
 * [seq_offsets[0], seq_offsets[n_seqs]); any other token's inputs are not
 * used (they may be NaN) and its grad is 0; a NaN of a token that takes part
 * goes into the loss and its own grad, an infinity counts as the formulas say
 * (a clipped ratio may be infinite; infinity times an advantage of 0 is NaN).
 * Per-token terms are fp32; their sums run over fixed ranges of 1024 tokens in
 * fp32 and then as pairs of floats, so the results are the same bits on every
 * run.  T == 0 gives loss and stats 0.
 *
 *   logprob, old_logprob  device, float [T]
 *   ref_logprob   device, float [T], or NULL (then kl_coef must be 0)
 *   advantages    device, float [T], or [n_seqs] with advantages_per_seq
 *   active_mask   device, uint8 [T] or NULL
 *   seq_offsets   device, int32 [n_seqs + 1], ascending within [0, T], or NULL for one sequence
 *                 of all T tokens (n_seqs must be 1); offsets that are not ascending set
 *                 RLK_ERR_INVALID_ARG in *dev_status and make loss and stats NaN
 *   clip_low, clip_high  >= 0;  dual_clip  0 (off) or > 1;  kl_kind  RLK_KL_K1 .. RLK_KL_K3;
 *                 all finite (a large one clips nothing);  |kl_coef| and |scale| at most the
 *                 largest fp32 number
 *   out_loss      device, float [1]
 *   kl_coef       with 0 the KL term is only reported in out_stats
 *   out_stats     device, float [4]: sums (with weights w_t, without scale) of -s, of k, of the
 *                 clipped tokens and of old_logprob - logprob
 *   grad_logprob  device, float [T], or NULL for the loss alone
 *   workspace     >= rlk_policy_loss_workspace_size(T, n_seqs) bytes, 256-byte aligned; that is 0
 *                 for small batches (up to 32768 tokens and 1024 sequences), then NULL is allowed
 */
#define RLK_KL_K1 1
#define RLK_KL_K2 2
#define RLK_KL_K3 3
#define RLK_REDUCE_SUM 0
#define RLK_REDUCE_TOKEN_MEAN 1
#define RLK_REDUCE_SEQ_MEAN 2
size_t rlk_policy_loss_workspace_size(int64_t T, int64_t n_seqs);
rlk_status_t rlk_policy_loss(const float* logprob, const float* old_logprob,
                             const float* ref_logprob, const float* advantages,
                             int advantages_per_seq, const uint8_t* active_mask,
                             const int32_t* seq_offsets, int64_t n_seqs, int64_t T,
                             double clip_low, double clip_high, double dual_clip, int kl_kind,
                             double kl_coef, int reduction, double scale, float* out_loss,
                             float* out_stats, float* grad_logprob, void* workspace,
                             size_t workspace_bytes, int32_t* dev_status, rlk_stream_t stream);

/*
 * Preference loss on paired log ratios, and its gradient with respect to the
 * log-probabilities, over 2 * n_pairs packed sequences.  With m_q the sum of
 * logprob - ref_logprob over sequence q's active tokens (their mean with
 * length_normalize; 0 where there are none), h = m_chosen - m_rejected and
 * z = beta h - margin, per pair
 *   RLK_PREF_SIGMOID  l = -(1 - label_smoothing) log sig(z) - label_smoothing log sig(-z)
 *   RLK_PREF_HINGE    l = max(0, 1 - z)
 *   RLK_PREF_IPO      l = (h - 1 / (2 beta))^2
 * and loss = scale * (mean of l over the pairs; 0 when n_pairs == 0).  Pair i
 * is sequences (2i, 2i + 1) with RLK_PAIRS_ADJACENT and (i, n_pairs + i) with
 * RLK_PAIRS_HALVES, the chosen one first.  A pair's loss, rewards and
 * gradients do not depend on where its sequences lie in the batch.
 *
 *   ref_logprob   device, float [T], or NULL (no reference: its terms are 0)
 *   seq_offsets   device, int32 [2 * n_pairs + 1], ascending within [0, T], else
 *                 RLK_ERR_INVALID_ARG in *dev_status and loss NaN
 *   beta          > 0;  label_smoothing in [0, 1], 0 unless SIGMOID;  margin 0 with IPO;  beta,
 *                 |margin| and |scale| at most the largest fp32 number
 *   out_loss      device, float [1];  out_pair_loss  device, float [n_pairs]
 *   out_rewards   device, float [2 * n_pairs]: beta m_q, in sequence order
 *   grad_logprob  device, float [T], or NULL; 0 for inactive tokens and those of no sequence
 *   n_pairs       at most 2^30
 *   workspace     >= rlk_preference_loss_workspace_size(T, n_pairs) bytes, 256-byte aligned; that
 *                 is 0, and NULL allowed, for all but few pairs of many tokens
 */
#define RLK_PREF_SIGMOID 0
#define RLK_PREF_HINGE 1
#define RLK_PREF_IPO 2
#define RLK_PAIRS_ADJACENT 0
#define RLK_PAIRS_HALVES 1
size_t rlk_preference_loss_workspace_size(int64_t T, int64_t n_pairs);
rlk_status_t rlk_preference_loss(const float* logprob, const float* ref_logprob,
                                 const uint8_t* active_mask, const int32_t* seq_offsets,
                                 int64_t n_pairs, int64_t T, int layout, int kind, double beta,
                                 double label_smoothing, double margin, int length_normalize,
                                 double scale, float* out_loss, float* out_pair_loss,
                                 float* out_rewards, float* grad_logprob, void* workspace,
                                 size_t workspace_bytes, int32_t* dev_status,
                                 rlk_stream_t stream);

/*
 * Global gradient norm over many tensors, and clipping by it:
 *   norm  = sqrt(sum of g^2 over all elements of all tensors)
 *   scale = max_norm / norm where norm is finite and above max_norm, else 1
 *   out   = RN(g * scale), rounded once to the tensor's type
 * Squares are summed in fp32 by each thread, and those sums added by a fixed
 * tree, at last as pairs of floats (a norm above 1.8e19 becomes infinite and
 * |g| below 1e-23 counts as 0); the order depends on the tensors' sizes,
 * types and places within 16 bytes alone.  A norm that is not finite leaves scale at 1 (the
 * gradients keep their values) and sets RLK_ERR_NONFINITE in *dev_status.
 *
 *   grads, outs   HOST arrays of n_tensors DEVICE pointers, each aligned to its element size.
 *                 outs[i] may be grads[i] (in place: nothing is written when scale is 1); any
 *                 other overlap of an output with an input or output is RLK_ERR_INVALID_ARG
 *   numels        HOST, elements per tensor (0 allowed; at most 2^38 in all)
 *   dtypes        HOST, RLK_DTYPE_F32, RLK_DTYPE_BF16 or RLK_DTYPE_F16 per tensor
 *   max_norm      >= 0 (infinity allowed)
 *   out_norm, out_scale  device, float [1] each
 *   workspace     >= rlk_grad_norm_workspace_size() bytes, 256-byte aligned; that
 *                 is 0 for small sets (about 1.5 MB in 64 tensors), then NULL is allowed
 * The host arrays are read before the call returns.
 */
size_t rlk_grad_norm_workspace_size(const int64_t* numels, const int32_t* dtypes,
                                    int64_t n_tensors);
rlk_status_t rlk_grad_norm(const void* const* grads, const int64_t* numels,
                           const int32_t* dtypes, int64_t n_tensors, float* out_norm,
                           void* workspace, size_t workspace_bytes, int32_t* dev_status,
                           rlk_stream_t stream);
rlk_status_t rlk_grad_clip(const void* const* grads, void* const* outs, const int64_t* numels,
                           const int32_t* dtypes, int64_t n_tensors, double max_norm,
                           float* out_norm, float* out_scale, void* workspace,
                           size_t workspace_bytes, int32_t* dev_status, rlk_stream_t stream);

/*
 * Activation checkpoints in 8 bits.  A row's features lie in blocks of 32 that
 * share a power of two, kept as one byte; with b the block's byte and c a
 * feature's code, the feature is
 *   RLK_SAVED_INT8   c * 2^(b - 133), c in -127 .. 127
 *   RLK_SAVED_E4M3   c * 2^(b - 127), c an e4m3 number (4 exponent, 3 mantissa bits, no infinities)
 * (the shared-exponent blocks of the OCP microscaling formats).  Every value that
 * rlk_act_quantize writes is a bf16 number, so restoring its checkpoints rounds nothing.
 * rlk_act_quantize takes, with e the exponent of the block's largest
 * magnitude m = f 2^e, b = e + 127 (INT8) and b = e + 119, one more where f >
 * 1.75 (E4M3; not below 0), and rounds each feature to the nearest code, ties
 * to the even one: within half a step, that is 2^-7 of 2^e (INT8), and 2^-4 of
 * the feature or 2^-10 of 2^(b - 127) (E4M3).  At e = 127 magnitudes above 1.75 * 2^127 become that
 * (E4M3).  A block with an infinity or NaN gets b = 255 and comes back as NaN throughout.
 *
 *   x, out       device, bf16 [T][H], 16-byte aligned
 *   format       RLK_SAVED_INT8 or RLK_SAVED_E4M3
 *   codes        device, one byte a feature [T][H], 16-byte aligned
 *   scales       device, uint8 [T][H / 32]
 *   H            multiple of 64, at most 2^20
 * Of codes that the quantiser does not write, INT8 -128 and E4M3 0x7F and 0xFF are taken as -128 and
 * +-480; E4M3 codes that under the bytes 0, 1 and 2 are no multiple of 2^-133, bf16's smallest step,
 * are restored to the nearest bf16 number, ties to even; from 2^128 on, and with b = 255, values are
 * infinite.
 */
#define RLK_SAVED_BF16 0              /* not a checkpoint: the bf16 tensor itself */
#define RLK_SAVED_INT8 1
#define RLK_SAVED_E4M3 2
rlk_status_t rlk_act_quantize(const void* x, int format, int64_t T, int64_t H, void* codes,
                              uint8_t* scales, rlk_stream_t stream);
rlk_status_t rlk_act_dequantize(const void* codes, const uint8_t* scales, int format, int64_t T,
                                int64_t H, void* out, rlk_stream_t stream);

/*
 * The norms before and after a block of the trunk, with the block's gate and
 * the residual stream's scales, in one pass (the strict-path table's
 * "RMSNorm" row with its residual add, for trunks that norm a block's output
 * too or scale and gate it).  Per row, in fp32:
 *   n   = block * rstd(block) * gamma_post       (block itself where gamma_post is NULL)
 *   x'  = bf16_RN(fma(residual_scale, residual, block_scale * (n * gate(g))))
 *   out = rlk_rmsnorm of x' with gamma_pre, the same bits
 * with rstd as in rlk_rmsnorm and gate(g) = 1, g or 1 / (1 + e^-g), where g below -87 counts as
 * -87 (a gate of 2^-125) and e^-g counts as 0 for g above 86.  Without
 * gamma_post and gate, and with both scales 1, x' too has rlk_rmsnorm's bits.
 * A row's result does not depend on the batch around it.
 *
 * With saved_format RLK_SAVED_INT8 or RLK_SAVED_E4M3 the pass also stores
 * checkpoints (rlk_act_quantize's, the same bits) of what the backward needs:
 * x', and where codes and scales are given, block and gate.
 *
 *   block, residual  device, bf16 [T][H];  gate  device, bf16 [T][H], or NULL
 *   gate_kind        RLK_GATE_IDENTITY or RLK_GATE_SIGMOID (of no effect without a gate)
 *   gamma_post       device, bf16 [H], or NULL;  gamma_pre  device, bf16 [H]
 *   residual_scale, block_scale  finite;  eps  > 0, of both norms
 *   out, residual_out  device, bf16 [T][H]: the normed rows and x'
 *   saved_x          {codes, scales} of x';  saved_block, saved_gate  of block and gate, both
 *                    NULL where not wanted;  none of them with RLK_SAVED_BF16
 *   H                multiple of 64, at most 8192; every pointer but scales 16-byte aligned
 * residual_out may be residual, and out may be block (in place); no other overlap is allowed.
 */
#define RLK_GATE_IDENTITY 1
#define RLK_GATE_SIGMOID 2
rlk_status_t rlk_block_norm(const void* block, const void* gamma_post, const void* gate,
                            int gate_kind, const void* residual, float residual_scale,
                            float block_scale, const void* gamma_pre, float eps, int64_t T,
                            int64_t H, void* out, void* residual_out, int saved_format,
                            void* saved_x, uint8_t* saved_x_scales, void* saved_block,
                            uint8_t* saved_block_scales, void* saved_gate,
                            uint8_t* saved_gate_scales, rlk_stream_t stream);

/*
 * Backward of rlk_block_norm.  With dx the gradient of x',
 *   dx            = rlk_rmsnorm_backward(grad_out; x', gamma_pre) + grad_residual_out
 *   grad_residual = residual_scale * dx
 *   dn            = block_scale * dx
 *   grad_gate     = dn * n * gate'(g)
 *   grad_block    = rmsnorm_backward(dn * gate(g); block, gamma_post), or dn * gate(g) itself
 *                   where gamma_post is NULL
 * and both norms' grad_gamma, in fp32, each gradient of the batch rounded once to
 * its type.  x, block and gate are bf16 tensors (saved_format RLK_SAVED_BF16, scales
 * NULL) or checkpoints, all three alike; from a checkpoint of rlk_act_quantize or rlk_block_norm the
 * call has the bits that it has from the restored tensor.  (Other codes may stand for values that a bf16
 * tensor would round; the call takes them as they are.)  A row's gradients do not depend on the batch around it; the grad_gammas are
 * summed over ranges of consecutive rows, in chains of 64 rows, and then over the ranges, in an
 * order that T and H fix.
 *
 *   grad_out       device, [T][H] of grad_out_dtype (RLK_DTYPE_F32 or RLK_DTYPE_BF16)
 *   grad_residual_out  device, [T][H] of grad_dtype: the gradient that reached x' from further
 *                  on, or NULL
 *   x              x' as the forward stored it
 *   block, gate    as in the forward; block is not read, and may be NULL, where gamma_post and
 *                  gate are NULL
 *   grad_residual, grad_block, grad_gate  device, [T][H] of grad_dtype (RLK_DTYPE_F32 or
 *                  RLK_DTYPE_BF16), each NULL where not wanted (grad_gate where there is no gate)
 *   grad_gamma_pre, grad_gamma_post  device, float [H], or NULL; all zeros when T == 0
 *   eps            as in the forward, and a normal number (2^-126 or more)
 *   workspace      >= rlk_block_norm_backward_workspace_size(T, H) bytes, 256-byte aligned;
 *                  nothing is needed when both grad_gammas are NULL
 *   H              multiple of 64, at most 8192; every pointer but scales 16-byte aligned
 * grad_residual may be grad_residual_out, or one of the three gradients grad_out where the types
 * are the same; no other overlap is allowed.
 */
size_t rlk_block_norm_backward_workspace_size(int64_t T, int64_t H);
rlk_status_t rlk_block_norm_backward(
    const void* grad_out, int grad_out_dtype, const void* grad_residual_out, int saved_format,
    const void* x, const uint8_t* x_scales, const void* block, const uint8_t* block_scales,
    const void* gate, const uint8_t* gate_scales, int gate_kind, const void* gamma_post,
    const void* gamma_pre, float residual_scale, float block_scale, float eps, int64_t T,
    int64_t H, void* grad_residual, void* grad_block, void* grad_gate, int grad_dtype,
    float* grad_gamma_pre, float* grad_gamma_post, void* workspace, size_t workspace_bytes,
    rlk_stream_t stream);

/*
 * rlk_rmsnorm_backward from an 8-bit checkpoint of x, rlk_act_quantize's or rlk_block_norm's:
 * grad_x has the bits of that call on the restored tensor; grad_gamma is its sum in this call's order
 * (as rlk_block_norm_backward's).
 *   format, codes, scales  rlk_act_quantize's
 *   workspace      >= rlk_block_norm_backward_workspace_size(T, H) bytes, 256-byte aligned;
 *                  nothing is needed when grad_gamma is NULL
 * Other arguments as rlk_rmsnorm_backward.
 */
rlk_status_t rlk_rmsnorm_backward_q8(const void* grad_out, int grad_out_dtype, int format,
                                     const void* codes, const uint8_t* scales, const void* gamma,
                                     float eps, const void* grad_residual, int64_t T, int64_t H,
                                     void* grad_x, int grad_x_dtype, float* grad_gamma,
                                     void* workspace, size_t workspace_bytes,
                                     rlk_stream_t stream);

/*
 * Verification of drafted tokens against the target's probabilities, from
 * given random numbers, with the strict logprob of every token it emits (the
 * rollout's side of the logprobs that training recomputes).  Sequence s has
 * n_s = draft_offsets[s + 1] - draft_offsets[s] drafted tokens, which may be
 * none, and n_s + 1 rows of target logits, from row draft_offsets[s] + s on: row i of them is
 * the target's distribution for the token at place i.  With p_i = softmax of that row and q_i the
 * draft's distribution, e^(draft_logits - draft_lse),
 *   the i-th drafted token x_i is accepted where all before it were and u_i q_i(x_i) < p_i(x_i);
 *   at the first one that is not (place i), the token is argmax_v max(p_i(v) - q_i(v), 0) / e(v);
 *   behind the last accepted draft (i = n_s), it is argmax_v p_i(v) / e(v)
 * with u the call's uniform numbers and e the sequence's noise.  With u uniform in
 * [0, 1) and e exponentially distributed the emitted tokens are distributed as the
 * target's own.  Without draft_logits the draft is certain of its tokens: q_i(x_i) = 1, 0 elsewhere.
 * Ties go to the lowest token; where p_i exceeds q_i nowhere the token is drawn from p_i.  A token whose
 * q_i is NaN (its draft logit or its row's draft_lse is) is never drawn, nor is one whose noise is NaN or
 * negative.
 * p is formed from the contract's (m, s) pair of the row and decisions do not depend on the batch;
 * a token's logprob has the bits that rlk_logits_logprob gives for that row and token.
 *
 *   target_logits  device, [n_draft + n_seqs][ld_target] of target_dtype (RLK_DTYPE_F32 or
 *                  RLK_DTYPE_BF16), aligned to its element size; columns [0, V) are read
 *   draft_logits   device, [n_draft][ld_draft] of draft_dtype, or NULL (certain drafts)
 *   draft_lse      device, float [n_draft] (rlk_logits_logprob's out_lse of the drafting step),
 *                  or NULL: draft_logits are log-probabilities (rlk_log_softmax's out)
 *   draft_tokens   device, int32 [n_draft];  uniforms  device, float [n_draft]
 *   noise          device, float [n_seqs][ld_noise], positive; columns [0, V) are read
 *   draft_offsets  device, int32 [n_seqs + 1], ascending within [0, n_draft]
 *   active_mask    device, uint8 [n_seqs] (nonzero = active), or NULL; an inactive sequence
 *                  gets out_accepted 0, tokens -1 and logprobs 0, whatever its rows, drafts and noise
 *                  hold.  (Its target rows are read all the same: an inactive sequence saves its draw,
 *                  not the sums over its rows, which are the larger part of a large batch.)
 *   out_accepted   device, int32 [n_seqs]: how many drafts were accepted
 *   out_tokens     device, int32 [n_draft + n_seqs], rows as target_logits: the accepted drafts,
 *                  the drawn token, then -1
 *   out_logprob    device, float [n_draft + n_seqs]: of those tokens, 0 behind the drawn one
 *   workspace      >= rlk_draft_verify_workspace_size(n_draft, n_seqs, V) bytes, 256-byte aligned
 * A drafted token outside [0, V) is not accepted, and reports RLK_ERR_TARGET_RANGE where it is
 * the first one refused.  A row that has to be drawn from and whose sum is not a number
 * (a NaN or +infinity in it, or nothing but -infinity) or that has no positive weight gives token -1, logprob NaN and
 * RLK_ERR_NONFINITE.  A sequence whose offsets descend or leave [0, n_draft] gets
 * out_accepted -1 and reports RLK_ERR_INVALID_ARG; its tokens are not written (and no row of the outputs
 * that belongs to no sequence is).  n_seqs == 0, with n_draft == 0, is a no-op.  No output may overlap
 * an input or another output.
 */
size_t rlk_draft_verify_workspace_size(int64_t n_draft, int64_t n_seqs, int64_t V);
rlk_status_t rlk_draft_verify(const void* target_logits, int target_dtype, int64_t ld_target,
                              const int32_t* draft_tokens, const void* draft_logits,
                              int draft_dtype, int64_t ld_draft, const float* draft_lse,
                              const float* uniforms, const float* noise, int64_t ld_noise,
                              const int32_t* draft_offsets, const uint8_t* active_mask,
                              int64_t n_draft, int64_t n_seqs, int64_t V, int32_t* out_accepted,
                              int32_t* out_tokens, float* out_logprob, void* workspace,
                              size_t workspace_bytes, int32_t* dev_status, rlk_stream_t stream);

/*
 * Same result as rlk_linear_logprob (same kernels, same bits), for callers
 * that cannot allocate device memory when they call: e.g. a rollout engine
 * that reserved almost all GPU memory for its KV cache at start-up, or a
 * decode loop that cannot afford the device-wide synchronisation cudaFree
 * performs.  Instead of a caller workspace it uses a scratch array of
 * RLK_STATIC_WS_BYTES compiled into the library (one copy per GPU that
 * loads the library, held until the process exits).  The pages have no
 * counterpart to this call; it is a deployment convenience.
 *
 *   - Allocates nothing and calls no allocating routine.
 *   - Batches whose workspace (rlk_workspace_size(T, V, n_shards)) exceeds
 *     RLK_STATIC_WS_BYTES are refused with RLK_ERR_WORKSPACE; at V = 151936
 *     that is about 1700 tokens per call with 4 shards.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current).  Under CUDA's
 *     default lazy module loading that lookup also loads the array itself,
 *     so the first call on a device is the one that still needs 16 MiB of
 *     free device memory: make it at start-up, before reserving the rest of
 *     the memory (a KV cache), and before any stream capture.  Later calls
 *     need no free memory at all.
 *   - The looked-up address belongs to the device's primary context: do not
 *     reset the device (cudaDeviceReset) or call from another context
 *     between calls.
 *   - All calls on a device share the array: calls that overlap on the GPU
 *     (e.g. on two unordered streams) race; order them.  Nothing in the
 *     array needs to start at zero.
 * Other arguments and errors (and the order in which they are checked) as
 * rlk_linear_logprob; RLK_ERR_CUDA also if the address lookup fails.
 */
#define RLK_STATIC_WS_BYTES (16u << 20)
rlk_status_t rlk_linear_logprob_static_ws(const void* hidden, const void* W,
                                          const int32_t* targets, const uint8_t* active_mask,
                                          int64_t T, int64_t H, int64_t V, int n_shards,
                                          float* out_logprob, float* out_lse, int32_t* dev_status,
                                          rlk_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RLK_H_ */
