/*
 * pstat.h -- C ABI of libpstat.so: batch-invariant per-token policy
 * statistics over a wide vocabulary on one GB300 (sm_103a).
 *
 * What the library computes is defined in torchtitan PR #4685, "[RL] Avoid
 * full-vocab gather for TP policy statistics":
 *   - Summary / Why: per-token sampled-token logprob and exact entropy from
 *     shard-local sufficient statistics (global maximum, softmax
 *     denominator, target contribution, entropy-weighted sum); entropy is a
 *     no-grad metric.
 *   - Review diff of loss.py: logprobs = -cross_entropy(logits, labels).
 *   - Correctness and compatibility: even/uneven vocabulary shards, FP32 and
 *     BF16 logits, ignored labels, partially masked (-inf) logits, and
 *     non-uniformly weighted gradients compared with the full vocabulary.
 * The fused lm_head entry points follow the chunked lm_head of TRL PR #6949
 * "ZeroSyncGRPOTrainer" (the vocabulary projection is multiplied chunk by
 * chunk; backward GEMMs run in bf16 and accumulate in fp32).
 *
 * Per row t with logits z_t[0..V), label y_t and weight w_t:
 *   M_t       = max_v z_tv,   S_t = sum_v exp(z_tv - M_t)
 *   logprob_t = z_{t,y_t} - M_t - ln S_t          (+0.0 if y_t == ignore_index)
 *   entropy_t = ln S_t - U_t / S_t,  U_t = sum_v exp(z_tv - M_t)(z_tv - M_t)
 *               (computed for ignored rows too: it does not depend on y_t)
 *   dlogits_tv = w_t (1[v = y_t] - exp(z_tv - M_t - ln S_t))
 *               (an all +0.0 row when y_t == ignore_index or w_t == 0)
 *
 * Numerics and batch invariance.  Each row is cut into fixed chunks that
 * restart at every shard start: chunk k of shard s covers columns
 * [b_s + k C, min(b_s + (k+1) C, b_{s+1})), C = PSTAT_CHUNK_BF16 or
 * PSTAT_CHUNK_F32 elements.  Per chunk the kernel forms (m, s, u) with a
 * reduction tree fixed at compile time; within a shard the chunks are folded
 * by a fixed tree (32 lane-strided ascending partial sums, then an xor
 * butterfly) and shards in ascending order within the row.  A row's
 * results therefore depend only on its own values, V, the shard bounds and
 * the dtype: they are bit-identical whatever batch the row sits in, at
 * whatever position, and from call to call.  Sharded and unsharded results
 * agree to rounding, not bitwise (the page's point that a partial sum then a
 * SUM reduction differs in the low bits from one contiguous sum).
 *
 * Conventions for every entry point:
 *   - All pointers except `shard_bounds` are DEVICE pointers owned by the
 *     caller (typically torch tensors).  `shard_bounds` is a HOST array.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream).  The library allocates no memory; scratch lives in the
 *     caller's `workspace`, sized by the matching *_workspace_size call.
 *   - Errors a host can see (null pointers, shapes, shard bounds, dtype,
 *     alignment, workspace size) are returned before anything is launched.
 *     A launch failure returns PSTAT_ERR_CUDA (from cudaGetLastError).
 *   - Errors only the device can see are OR-ed into `*dev_error` (a device
 *     int, may be NULL) with atomics, and the affected row's outputs become
 *     NaN; no kernel traps or asserts.  Read the flag when you need it.
 *   - Labels are int64, weights float32, statistics and logprob/entropy
 *     float32.  Logits/dlogits are row-major with a row stride `ld` (in
 *     elements, >= V).
 */
#ifndef PSTAT_H
#define PSTAT_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PSTAT_API __attribute__((visibility("default")))
#else
#define PSTAT_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Opaque CUDA stream handle; identical to cudaStream_t. */
typedef struct CUstream_st* pstat_stream_t;

typedef enum { PSTAT_F32 = 0, PSTAT_BF16 = 1 } pstat_dtype;

/* Return codes. */
enum {
    PSTAT_OK = 0,
    PSTAT_ERR_NULLPTR = -1,     /* a required pointer is NULL */
    PSTAT_ERR_SHAPE = -2,       /* T < 0, V < 1, ld < V, d not a multiple of 64, ... */
    PSTAT_ERR_SHARDS = -3,      /* bounds not strictly increasing from 0 to V, or too many */
    PSTAT_ERR_DTYPE = -4,       /* unknown dtype or unsupported combination */
    PSTAT_ERR_ALIGN = -5,       /* a pointer lacks the alignment stated for it */
    PSTAT_ERR_WORKSPACE = -6,   /* workspace NULL or smaller than required */
    PSTAT_ERR_CUDA = -7,        /* a CUDA runtime call or launch failed */
    PSTAT_ERR_UNSUPPORTED = -8, /* the current device is not sm_103 (GB300) */
    PSTAT_ERR_PARAM = -9        /* a numeric parameter is out of range, or outputs overlap */
};

/* Bits OR-ed into *dev_error by the kernels. */
#define PSTAT_DEV_BAD_LABEL 0x1 /* label outside [0, V) and != ignore_index */
#define PSTAT_DEV_EMPTY_ROW 0x2 /* every logit of a row is -inf: softmax undefined */
#define PSTAT_DEV_TIMEOUT 0x4   /* a bounded wait on an asynchronous copy gave up */
#define PSTAT_DEV_RANGE 0x8     /* lm_head backward: a value exceeds the fp16 range (65504) */
#define PSTAT_DEV_BAD_PARAM 0x10 /* a temperature, top_p, min_p, uniform, parent, rate or step is out of range */
#define PSTAT_DEV_NONFINITE 0x20 /* the gradient norm, or an element to be quantised, is infinite or NaN */

#define PSTAT_MAX_SHARDS 64
#define PSTAT_CHUNK_BF16 4096 /* chunk length in elements for bf16 logits */
#define PSTAT_CHUNK_F32 2048  /* chunk length in elements for fp32 logits */

/* Human-readable text for a return code; never NULL. */
PSTAT_API const char* pstat_status_string(int code);

/* Version of this ABI (major * 10000 + minor * 100 + patch). */
PSTAT_API int pstat_version(void);

/*
 * Workspace bytes for pstat_forward / pstat_backward on T rows of V logits
 * of dtype `dt` split by `shard_bounds` (host, n_shards + 1 entries; NULL and
 * n_shards = 1 mean one shard {0, V}).  The workspace holds one 16-byte
 * (m, s, u) record per row and chunk, and the (M, ln S) pair per row that
 * pstat_backward needs when it is not given `rowstats`.
 */
PSTAT_API int pstat_workspace_size(int64_t T, int64_t V, pstat_dtype dt, const int64_t* shard_bounds,
                         int n_shards, size_t* bytes);

/*
 * Forward statistics: per-chunk statistics combined in a fixed order.  Plans
 * of at most 256 chunks per row run as one kernel with the records in shared
 * memory (no workspace needed: it may be NULL and is not touched); larger
 * plans run the chunk-statistics kernel into the workspace, then the combine.
 * Both give the same bits.
 *   logits        [T, ld] dtype `dt`; element (t, v) at logits + t*ld + v.
 *                 Any alignment works; 16-byte aligned rows and chunk starts
 *                 take the bulk-copy path, others a slower path with the same
 *                 numerics.
 *   labels        [T] int64 (NULL: every row ignored).
 *   shard_bounds  host int64[n_shards + 1], 0 = b_0 < b_1 < ... < b_S = V,
 *                 n_shards <= PSTAT_MAX_SHARDS; NULL means {0, V}.
 *   out_logprob   [T] float (may be NULL), out_entropy [T] float (may be
 *                 NULL), out_rowstats [T, 2] float (M, ln S) (may be NULL).
 *   workspace     >= pstat_workspace_size(...) bytes, 16-byte aligned;
 *                 required only for plans of more than 256 chunks per row
 *                 (PSTAT_ERR_WORKSPACE when it is missing there).
 *   dev_error     device int or NULL; bits PSTAT_DEV_*.
 * T = 0 is a no-op returning PSTAT_OK.
 */
PSTAT_API int pstat_forward(const void* logits, pstat_dtype dt, int64_t T, int64_t V, int64_t ld,
                  const int64_t* labels, int64_t ignore_index, const int64_t* shard_bounds,
                  int n_shards, float* out_logprob, float* out_entropy, float* out_rowstats,
                  void* workspace, size_t ws_bytes, int* dev_error, pstat_stream_t stream);

/* Bytes of the fixed device scratch used by pstat_forward_noalloc (8 MiB). */
#define PSTAT_NOALLOC_SCRATCH_BYTES (8u << 20)

/* PSTAT_NOALLOC_SCRATCH_BYTES as built into this library, for bindings that
 * cannot read the header. */
PSTAT_API size_t pstat_noalloc_scratch_bytes(void);

/*
 * pstat_forward for callers that cannot allocate device memory.  The pages
 * have no counterpart to this entry point; it exists for this library's
 * users.  Some callers must not call cudaMalloc where they compute these
 * statistics: allocation synchronises the device, a host runtime or
 * framework may own all device memory through its own pool, or a plain C
 * caller may have no allocator at all.  This variant takes no workspace and
 * allocates nothing: its per-chunk scratch is a fixed array of
 * PSTAT_NOALLOC_SCRATCH_BYTES inside the library, present on every GPU that
 * loads the library until the process exits.  The caller still passes the
 * inputs and outputs, with the same meaning, layout and results as
 * pstat_forward.
 *   Limit: T * n_chunks * 16 bytes must fit the scratch (n_chunks as in
 *   pstat_workspace_size; e.g. T <= 13,797 rows at V = 151,936 in bf16),
 *   else PSTAT_ERR_WORKSPACE is returned before anything is launched.
 *   The first call on each device looks up the scratch's device address
 *   (cudaGetSymbolAddress) with that device current; make that first call
 *   before any stream capture.  The address is cached per CUDA context
 *   (cuCtxGetId): after cudaDeviceReset, the first call in the new context
 *   looks it up again, so that call too belongs before any capture.
 *   Every call on a device shares the one scratch array, which keeps the last
 *   call's contents.  Nothing in it needs clearing (each call writes every
 *   record it reads), but calls whose kernels overlap on the GPU (different
 *   streams, or host threads issuing concurrently) race on it: serialise
 *   them, e.g. on one stream.
 */
PSTAT_API int pstat_forward_noalloc(const void* logits, pstat_dtype dt, int64_t T, int64_t V,
                                    int64_t ld, const int64_t* labels, int64_t ignore_index,
                                    const int64_t* shard_bounds, int n_shards, float* out_logprob,
                                    float* out_entropy, float* out_rowstats, int* dev_error,
                                    pstat_stream_t stream);

/*
 * Weighted backward dlogits = w (onehot(y) - softmax(z)) (fused elementwise
 * kernel).
 *   weights       [T] float (NULL: all ones).
 *   rowstats      [T, 2] float (M, ln S) from pstat_forward on the same
 *                 logits and shard bounds; NULL recomputes them first through
 *                 the forward kernels (needs the workspace).
 *   out_dlogits   [T, ld_out] of `out_dt` (PSTAT_BF16 rounds to nearest even;
 *                 PSTAT_F32 needs dt == PSTAT_F32).  Every element of the
 *                 T x V block is written.
 *   workspace     needed only when rowstats is NULL (else may be NULL / 0).
 */
PSTAT_API int pstat_backward(const void* logits, pstat_dtype dt, int64_t T, int64_t V, int64_t ld,
                   const int64_t* labels, int64_t ignore_index, const float* weights,
                   const float* rowstats, const int64_t* shard_bounds, int n_shards,
                   void* out_dlogits, pstat_dtype out_dt, int64_t ld_out, void* workspace,
                   size_t ws_bytes, int* dev_error, pstat_stream_t stream);

/*
 * pstat_forward followed by pstat_backward in one pass over the logits
 * (the pages' forward+backward unit, reusing cross-entropy forward and
 * backward together; here as one kernel).  Results are bit-identical to the
 * two calls with the same arguments; the logits are read from HBM once (each
 * CTA re-reads a row's chunks from L2 for the gradient), so a bf16 token
 * moves 4V bytes instead of 6V.  No workspace: a row's chunk records live in
 * shared memory.
 *   Arguments as in pstat_forward / pstat_backward; out_dlogits [T, ld_out]
 *   is required, out_logprob / out_entropy / out_rowstats may be NULL.
 *   The shard plan may have at most 256 chunks per row (PSTAT_ERR_SHAPE).
 */
PSTAT_API int pstat_forward_backward(const void* logits, pstat_dtype dt, int64_t T, int64_t V,
                                     int64_t ld, const int64_t* labels, int64_t ignore_index,
                                     const float* weights, const int64_t* shard_bounds,
                                     int n_shards, float* out_logprob, float* out_entropy,
                                     float* out_rowstats, void* out_dlogits, pstat_dtype out_dt,
                                     int64_t ld_out, int* dev_error, pstat_stream_t stream);

/*
 * Vocabulary-parallel use: each rank holds the logits of one vocabulary shard
 * [b_s, b_{s+1}) of every row (torchtitan PR #4685, Summary and the review
 * thread's batch-invariance answer: shard-local maximum, sum of exponentials,
 * entropy-weighted sum and target logit, reduced across ranks).  Here the
 * ranks exchange the [T, 4] statistics with an all-gather instead of MAX/SUM
 * all-reduces, and every rank folds them in ascending shard order with
 * pstat_combine_shards, so all ranks hold the same bits and the result does
 * not depend on the collective's reduction order.
 *
 * pstat_shard_stats on every shard followed by pstat_combine_shards equals
 * pstat_forward with those shard_bounds bit for bit; pstat_backward_shard
 * equals the shard's columns of pstat_backward.
 */

/*
 * Per-row statistics of one vocabulary shard.
 *   logits        [T, ld] dtype `dt`: this shard's V columns (chunks are laid
 *                 from its first column).  V may hold at most 256 chunks
 *                 (PSTAT_ERR_SHAPE otherwise).
 *   labels        [T] int64 in the whole vocabulary's numbering, or NULL.
 *   vocab_start   the shard's first column in that numbering (b_s).
 *   out_stats     [T, 4] float, 16-byte aligned: (M_s, S_s, U_s, z_y) with
 *                 S_s = sum exp(z - M_s), U_s = sum exp(z - M_s)(z - M_s) over
 *                 the shard, and z_y the label's logit when vocab_start <= y <
 *                 vocab_start + V, else 0.  A fully masked shard gives
 *                 (-inf, 0, 0, .).  Label range errors are reported by
 *                 pstat_combine_shards.
 */
PSTAT_API int pstat_shard_stats(const void* logits, pstat_dtype dt, int64_t T, int64_t V,
                                int64_t ld, const int64_t* labels, int64_t ignore_index,
                                int64_t vocab_start, float* out_stats, int* dev_error,
                                pstat_stream_t stream);

/*
 * Fixed-order combine of gathered shard statistics into the row outputs.
 *   stats         [T, n_shards, 4] float (device, 16-byte aligned): row t,
 *                 shard s at stats + (t n_shards + s) 4, shards in ascending
 *                 vocabulary order.
 *   shard_bounds  host int64[n_shards + 1], 0 = b_0 < ... < b_S = V_total.
 *   Outputs, labels and dev_error as pstat_forward (bad labels: bit 1, NaN;
 *   fully masked rows: bit 2, NaN).
 */
PSTAT_API int pstat_combine_shards(const float* stats, int64_t T, int n_shards,
                                   const int64_t* shard_bounds, const int64_t* labels,
                                   int64_t ignore_index, float* out_logprob, float* out_entropy,
                                   float* out_rowstats, int* dev_error, pstat_stream_t stream);

/*
 * Weighted backward of one vocabulary shard's columns.
 *   As pstat_backward on the shard's V columns, with rowstats [T, 2] the
 *   global (M, ln S) (required) and labels in the whole vocabulary's
 *   numbering: the one-hot term lands in this shard only when vocab_start <=
 *   y < vocab_start + V; labels outside [0, vocab_total) give NaN rows and
 *   dev_error bit 1.  vocab_start + V <= vocab_total.
 */
PSTAT_API int pstat_backward_shard(const void* logits, pstat_dtype dt, int64_t T, int64_t V,
                                   int64_t ld, const int64_t* labels, int64_t ignore_index,
                                   const float* weights, const float* rowstats,
                                   int64_t vocab_start, int64_t vocab_total, void* out_dlogits,
                                   pstat_dtype out_dt, int64_t ld_out, int* dev_error,
                                   pstat_stream_t stream);

/*
 * The full log-softmax log p_tv = z_tv - M_t - ln S_t as a [T, V] tensor, in
 * one read and one write pass over the logits, from the same row statistics
 * as the other entry points (so it is batch-invariant too: a row's output
 * bits do not depend on the batch).  The BI log_softmax of the batch-
 * invariant GDN README's kernel list, for callers that need every column.
 *   rowstats  [T, 2] (M, ln S) from pstat_forward with the same shard bounds,
 *             or NULL to compute them first (needs the workspace).
 *   out       [T, ld_out] of out_dt (bf16 rounds to nearest even); -inf
 *             logits give -inf, rows with no finite logit give NaN and set
 *             PSTAT_DEV_EMPTY_ROW.
 */
PSTAT_API int pstat_log_softmax(const void* logits, pstat_dtype dt, int64_t T, int64_t V,
                                int64_t ld, const float* rowstats, const int64_t* shard_bounds,
                                int n_shards, void* out, pstat_dtype out_dt, int64_t ld_out,
                                void* workspace, size_t ws_bytes, int* dev_error,
                                pstat_stream_t stream);

/*
 * Trainer/rollout logprob mismatch metrics, as the torchtitan batch-invariant
 * GDN README logs them ("Code map": bit_wise/logprob_diff/{mean,abs_mean,max}
 * and bit_wise/ratio_tokens_different/mean).  Over the tokens whose label is
 * not ignore_index (all tokens when labels is NULL), d_t = logprob_t -
 * rollout_logprob_t:
 *   out_metrics[0] = mean d,  [1] = mean |d|,  [2] = max |d|,
 *   [3] = fraction of tokens whose float32 bit patterns differ.
 * With no token counted: [0], [1], [3] are NaN and [2] is 0.  One fixed-order
 * reduction on the device (double-precision sums): repeated calls give the
 * same bits.  logprob, rollout_logprob [T] float; out_metrics device float[4].
 */
PSTAT_API int pstat_logprob_diff_metrics(const float* logprob, const float* rollout_logprob,
                                         const int64_t* labels, int64_t ignore_index, int64_t T,
                                         float* out_metrics, pstat_stream_t stream);

/*
 * Clipped-ratio policy surrogate (the DAPO recipes of the same README use
 * eps_low = 0.2, eps_high = 0.28), per token, with r_t = exp(logprob_t -
 * old_logprob_t):
 *   out_loss_t   = -scale min(r_t A_t, clip(r_t, 1 - eps_low, 1 + eps_high) A_t)
 *   out_weight_t = d out_loss_t / d logprob_t
 *                = -scale A_t r_t if the unclipped term is the minimum (or
 *                  ties), else 0 (the clipped term does not depend on logprob).
 * Ignored tokens get loss 0 and weight 0.  out_weight is what pstat_backward
 * and pstat_forward_backward take as `weights` to give the loss's gradient
 * with respect to the logits.  All arrays [T] float (out_loss may be NULL);
 * 0 <= eps_low < 1, eps_high >= 0.
 */
PSTAT_API int pstat_clipped_surrogate(const float* logprob, const float* old_logprob,
                                      const float* advantages, const int64_t* labels,
                                      int64_t ignore_index, int64_t T, float eps_low,
                                      float eps_high, float scale, float* out_loss,
                                      float* out_weight, pstat_stream_t stream);

/*
 * Workspace bytes for the fused lm_head entry points (T tokens, V vocab
 * rows, hidden size d).
 */
PSTAT_API int pstat_lmhead_workspace_size(int64_t T, int64_t V, int64_t d, size_t* bytes);

/*
 * Fused lm_head forward: logits z = hidden W^T are formed tile by tile on
 * the tensor cores (bf16 operands, fp32 accumulation in tensor memory) and
 * folded straight into the chunk statistics; logits are never written to
 * memory.  Outputs as pstat_forward.
 *   hidden  [T, d] bf16 row-major, W [V, d] bf16 row-major; both 16-byte
 *           aligned, d a multiple of 64 (PSTAT_ERR_SHAPE otherwise).
 */
PSTAT_API int pstat_lmhead_fused(const void* hidden, const void* W, int64_t T, int64_t V, int64_t d,
                       const int64_t* labels, int64_t ignore_index, float* out_logprob,
                       float* out_entropy, float* out_rowstats, void* workspace,
                       size_t ws_bytes, int* dev_error, pstat_stream_t stream);

/*
 * Fused lm_head backward through z = hidden W^T of the weighted gradient
 * g = w (onehot(y) - softmax(z)):
 *   dhidden [T, d] float  += g W
 *   dW      [V, d] float  += g^T hidden
 * Both are ACCUMULATED into (zero them first for a plain gradient), so calls
 * over token or vocabulary chunks compose.  rowstats [T, 2] from
 * pstat_lmhead_fused is required.  g is formed on chip from recomputed
 * logits and staged only per vocabulary chunk in the workspace.
 */
PSTAT_API int pstat_lmhead_backward(const void* hidden, const void* W, int64_t T, int64_t V, int64_t d,
                          const int64_t* labels, int64_t ignore_index, const float* weights,
                          const float* rowstats, float* dhidden, float* dW, void* workspace,
                          size_t ws_bytes, int* dev_error, pstat_stream_t stream);

/*
 * Tempered, truncated distributions: drawing a token from a row, and the
 * policy statistics of a given label under the distribution that draws come
 * from (the ratio pi/mu of an RL step compares two policies under one
 * distribution, so its trainer side needs the rollout's temperature and
 * truncation).
 *
 * Row z[0..V), temperature t, M = max z, x_v = (z_v - M)/t, e_v = e^(x_v).
 * Tokens are ordered by (logit descending, index ascending); -inf logits are
 * masked and never kept.  Each filter keeps a prefix of that order:
 *   top_k  the first top_k tokens (top_k <= 0 or >= V: all);
 *   top_p  the shortest prefix whose mass reaches top_p times the mass that
 *          top_k left (top_p = 1: all);
 *   min_p  the tokens with e_v >= min_p (min_p = 0: all).
 * The kept set is the shortest of the three.  Its last token is the cut
 * (tau, i): v is kept when z_v > tau, or z_v == tau and v <= i.  With no
 * filter the cut is (-inf, V - 1).
 * Which tokens are kept and drawn is decided by fixed-point weights, each within
 * 2^-45 + 2^-44.5 |x_v| of its e_v (relative), and exact integer sums of them;
 * ties by the lowest index.
 * The results of a row depend on its own values and settings only: they are
 * bit-identical in any batch.
 * A row with a NaN or +inf logit, or without a finite one, has no
 * distribution: PSTAT_DEV_EMPTY_ROW, NaN outputs, token and cut index -1.
 */

#define PSTAT_FILTER_MAX_V (1 << 20) /* largest vocabulary of these entry points */
#define PSTAT_FILTER_MAX_T (1 << 24) /* most rows of one call */

/* Settings of a call: one value for every row, or a device array [T] that
 * replaces it where the pointer is not NULL.  A row whose array value is out of
 * range gets PSTAT_DEV_BAD_PARAM, NaN outputs, token and cut index -1; a value
 * of the struct itself out of range is PSTAT_ERR_PARAM. */
typedef struct {
    float temperature;         /* in [2^-20, 2^20]; sampling also takes 0: the first maximum */
    float top_p;               /* in (0, 1] */
    float min_p;               /* in [0, 1] */
    int64_t top_k;
    const float* temperatures; /* device [T] or NULL */
    const int32_t* top_ks;
    const float* top_ps;
    const float* min_ps;
} pstat_filters;

/*
 * Workspace bytes of pstat_sample and pstat_filtered_forward on T rows of V
 * logits (V <= PSTAT_FILTER_MAX_V, T <= PSTAT_FILTER_MAX_T).
 */
PSTAT_API int pstat_filter_workspace_size(int64_t T, int64_t V, pstat_dtype dt, size_t* bytes);

/*
 * Draws one token per row: the first v in index order whose kept mass
 * sum_{w <= v, kept} e_w exceeds uniform times the whole kept mass.
 *   uniform      [T] float in [0, 1).
 *   out_token    [T] int64.
 *   out_logprob  [T] float: x_v - ln sum_{kept} e (0 at temperature 0).
 *   Logits, dev_error and stream as pstat_forward; workspace 16-byte aligned,
 *   at least pstat_filter_workspace_size(...) bytes.
 */
PSTAT_API int pstat_sample(const void* logits, pstat_dtype dt, int64_t T, int64_t V, int64_t ld,
                           const float* uniform, const pstat_filters* filters, int64_t* out_token,
                           float* out_logprob, void* workspace, size_t ws_bytes, int* dev_error,
                           pstat_stream_t stream);

/*
 * Policy statistics of labels under the tempered, truncated distribution.
 *   labels         [T] int64 (NULL: every row ignored).
 *   out_logprob    [T] float: x_y - ln S, S the kept mass; -inf where y is not
 *                  kept, +0 where it is ignore_index.
 *   out_entropy    [T] float: ln S - (1/S) sum_{kept} e x.
 *   out_rowstats   [T, 2] float (M, ln S).
 *   out_cut_logit  [T] float and out_cut_index [T] int64: the cut.
 *   All outputs are required.  Labels outside [0, V): PSTAT_DEV_BAD_LABEL,
 *   logprob and entropy NaN.  Workspace as pstat_sample.
 */
PSTAT_API int pstat_filtered_forward(const void* logits, pstat_dtype dt, int64_t T, int64_t V,
                                     int64_t ld, const int64_t* labels, int64_t ignore_index,
                                     const pstat_filters* filters, float* out_logprob,
                                     float* out_entropy, float* out_rowstats,
                                     float* out_cut_logit, int64_t* out_cut_index,
                                     void* workspace, size_t ws_bytes, int* dev_error,
                                     pstat_stream_t stream);

/*
 * Weighted backward of that logprob:
 *   dlogits_v = (w/t) (1[v = y] - kept_v e_v / S),
 * an all +0.0 row where y is ignored, w = 0 or y is not kept.  The kept set is
 * held fixed, as the truncation is piecewise constant in the logits.
 *   rowstats, cut_logit, cut_index  from pstat_filtered_forward on the same
 *                  logits and settings.
 *   temperature    for every row, or `temperatures` [T] where not NULL.
 *   weights, out_dlogits, out_dt, ld_out as pstat_backward; out_dlogits may not
 *   overlap the logits (PSTAT_ERR_PARAM).
 */
PSTAT_API int pstat_filtered_backward(const void* logits, pstat_dtype dt, int64_t T, int64_t V,
                                      int64_t ld, const int64_t* labels, int64_t ignore_index,
                                      const float* weights, const float* rowstats,
                                      const float* cut_logit, const int64_t* cut_index,
                                      float temperature, const float* temperatures,
                                      void* out_dlogits, pstat_dtype out_dt, int64_t ld_out,
                                      int* dev_error, pstat_stream_t stream);

/*
 * The global L2 norm of a list of gradients, and clipping by it.
 *   norm = sqrt(sum over all elements of all tensors of g^2)
 *   out  = g * min(1, max_norm / norm)
 * The list is a HOST array; each entry names `n` contiguous elements on the
 * device.  Tensors may differ in type and size, be empty, and start at any
 * element; at most PSTAT_GRAD_MAX_ELEMENTS each.  Squares are summed without
 * overflow or underflow, in an order fixed by the sizes and types and by the
 * device's number of SMs: the same values give the same bits, wherever the
 * tensors lie.  The norm is within 10 x 2^-24 of the exact one.  An empty list
 * has norm 0.
 */
#define PSTAT_GRAD_MAX_ELEMENTS ((int64_t)1 << 40)
typedef struct {
    const void* data;
    void* out; /* clipping: where the scaled tensor goes, same type; may equal data */
    int64_t n;
    int32_t dtype; /* PSTAT_F32 or PSTAT_BF16 */
} pstat_tensor;

PSTAT_API int pstat_grad_workspace_size(const pstat_tensor* tensors, int64_t n_tensors,
                                        size_t* bytes);

/* out_norm: device float.  An infinite or NaN norm sets PSTAT_DEV_NONFINITE.
 * Workspace 8-byte aligned, at least pstat_grad_workspace_size(...) bytes. */
PSTAT_API int pstat_grad_norm(const pstat_tensor* tensors, int64_t n_tensors, float* out_norm,
                              void* workspace, size_t ws_bytes, int* dev_error,
                              pstat_stream_t stream);

/* The norm before clipping goes to out_norm.  max_norm >= 0.  When the norm is
 * infinite or NaN the tensors are passed on unscaled (and the bit is set), so
 * that the caller can drop the step.  An `out` that overlaps another `out`, or
 * a `data` that is not its own, is PSTAT_ERR_PARAM. */
PSTAT_API int pstat_clip_grad_norm(const pstat_tensor* tensors, int64_t n_tensors, float max_norm,
                                   float* out_norm, void* workspace, size_t ws_bytes,
                                   int* dev_error, pstat_stream_t stream);

/*
 * An AdamW step over a list of tensors:
 *   g' = f g,  f = min(1, max_norm / norm) (1 where norm is NULL)
 *   m  = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
 *   p  = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
 * in fp32, with m and v as products and sums that are each rounded once (no fused
 * multiply-add).  A norm that is infinite or NaN sets PSTAT_DEV_NONFINITE, and
 * nothing is changed.
 *
 * Moments of 32 bits are float[n].  Moments of 8 bits are uint8[n + ceil(n / 128)]:
 * n codes, then one byte for each block of 128 of them, the exponent field E of the
 * block's largest magnitude as an fp32 number.  With base = max(8 (E - d), 0), code c
 * > 0 stands for the fp32 number whose bits are (c + base) << 20 (three bits of
 * mantissa), 0 for zero; m has d = 14, codes to 126, NaN 127, and the sign in bit 7;
 * v has d = 30, codes to 254 and NaN 255.  All zeros is a fresh state.
 * What is held in fewer than 32 bits (8-bit moments, bf16 parameters) is rounded
 * up with the probability of its distance from the number below, by a hash of
 * (seed, place of the tensor in the list, element), where `random` is set: the
 * same call gives the same bits.  Otherwise it is rounded to nearest (8-bit moments:
 * halves away from zero); then an 8-bit v follows only gradients that move it by
 * a sixteenth.  An 8-bit v above zero stays above zero.
 *   param, exp_avg, exp_avg_sq  read and written; they may overlap nothing else of
 *                   the call (PSTAT_ERR_PARAM).
 *   lr_at, step_at, seed_at     device values that take the place of lr, step and
 *                   seed where not NULL, so that a captured step can be replayed.
 *                   step >= 1 (t above).  A rate on the device that is negative, infinite
 *                   or NaN, and a step below 1, set PSTAT_DEV_BAD_PARAM, and nothing is
 *                   changed.
 */
#define PSTAT_ADAMW_MAX_TENSORS ((int64_t)1 << 28)
typedef struct {
    void* param;
    const void* grad;
    void* exp_avg;
    void* exp_avg_sq;
    int64_t n;
    int32_t param_dtype; /* PSTAT_F32 or PSTAT_BF16, each on its own */
    int32_t grad_dtype;
    int32_t bits; /* of the moments: 32 or 8 */
    int32_t reserved;
} pstat_adamw_tensor;
typedef struct {
    double lr, beta1, beta2, eps, weight_decay; /* lr, eps, wd >= 0; 0 <= beta < 1 */
    int64_t step;
    const float* lr_at;
    const int64_t* step_at;
    const int64_t* seed_at;
    const float* norm; /* device, as pstat_grad_norm leaves it, or NULL */
    uint64_t seed;
    float max_norm; /* >= 0, used with norm */
    int32_t random;
} pstat_adamw_options;

PSTAT_API int pstat_adamw_step(const pstat_adamw_tensor* tensors, int64_t n_tensors,
                               const pstat_adamw_options* options, int* dev_error,
                               pstat_stream_t stream);

/* The values that 8-bit moments stand for, as float[n] each. */
typedef struct {
    const void* exp_avg;
    const void* exp_avg_sq;
    float* out_avg;
    float* out_avg_sq;
    int64_t n;
} pstat_adamw_moment;
PSTAT_API int pstat_adamw_moments(const pstat_adamw_moment* list, int64_t n, pstat_stream_t stream);

/*
 * Matrices in 8-bit floating point (e4m3: 4 bits of exponent, 3 of mantissa, largest
 * 448, no infinity) with one scale for each run of 128 columns, of one row or
 * of 128 rows.
 *   scale = the least power of two s with max|x| <= 448 s over the block (at least
 *           2^-126; 1 for a block of zeros),  q = x / s, rounded to nearest even.
 * The division is exact, so q s is off by one rounding of 2^-4 relative.  A block
 * with an infinity or NaN gets scale NaN and codes 0 (PSTAT_DEV_NONFINITE).
 *   x        [T, ld] dtype `dt`, any alignment of its elements.
 *   rows     rows that share a scale: 1 or 128.
 *   out_q    [T, K] e4m3, rows of K bytes.
 *   out_scale  float, that of row block i and column block j at
 *            out_scale[i * scale_row + j * scale_col]; ceil(T / rows) by
 *            ceil(K / 128), each in a place of its own (PSTAT_ERR_SHAPE).
 * Outputs that overlap one another or x are refused (PSTAT_ERR_PARAM).
 */
PSTAT_API int pstat_fp8_quantize(const void* x, pstat_dtype dt, int64_t T, int64_t K, int64_t ld,
                                 int rows, void* out_q, float* out_scale, int64_t scale_row,
                                 int64_t scale_col, int* dev_error, pstat_stream_t stream);

/*
 * Logits of an 8-bit head: out[t, v] = sum_j S[v / 128, j] s[t, j] (sum over column
 * block j of q[t, k] W[v, k]).  The inner sums run on the tensor cores with fp32
 * accumulators, the outer one in fp32, blocks in ascending order: a row's results
 * depend on its own codes and scales only, they are bit-identical in any batch.
 *   q        [T, K] e4m3 with scales s as pstat_fp8_quantize lays them out (rows 1);
 *            scale_row 1 is the quick order.
 *   W        [V, K] e4m3, W_scale [ceil(V / 128), ceil(K / 128)] row-major: any
 *            scales, powers of two or not.
 *   q and W 16-byte aligned, K a multiple of 16.
 *   out      [T, ld_out] of out_dt; one that overlaps an input is refused (PSTAT_ERR_PARAM).
 */
PSTAT_API int pstat_fp8_logits(const void* q, const float* q_scale, int64_t scale_row,
                               int64_t scale_col, const void* W, const float* W_scale, int64_t T,
                               int64_t V, int64_t K, void* out, pstat_dtype out_dt, int64_t ld_out,
                               int* dev_error, pstat_stream_t stream);

/*
 * Beam search: the best n continuations of each of B searches with `beams` beams.
 * Beam k of search b has the row z = logits[b beams + k] and the score s = scores[b,
 * k]; its continuation by token v scores s + z_v - M - ln S.  Of the beams x V
 * continuations the n best, in descending order; equal ones by the lowest (k, v).
 * Scores are compared as they are in exact arithmetic, to 2^-38 of the largest of
 * |s|, |score| and 1; what comes out is within 6e-6 + 2^-24 |score| of the score.  A score of
 * -inf, and a row whose logits are all -inf, is a beam without continuations; a token
 * whose z_v - M or score lies below the range of fp32 is none either.  Places that
 * none is left for get score -inf, parent and token -1.  A score of NaN or +inf, or
 * a row with a NaN or +inf logit (of a beam with a finite score), leaves its search
 * undefined: PSTAT_DEV_EMPTY_ROW, scores NaN, parents and tokens -1.
 *   logits      [B beams, ld] of dtype `dt`, V <= PSTAT_FILTER_MAX_V; ld 0: one row for
 *               all beams.
 *   scores      [B, beams] float.
 *   n           at most PSTAT_BEAM_MAX_N; beams at most PSTAT_BEAM_MAX.
 *   out_score   [B, n] float, out_parent (k) and out_token (v) [B, n] int64.
 *   workspace   16-byte aligned, at least pstat_beam_workspace_size(...) bytes.
 * Outputs and workspace may overlap nothing else of the call (PSTAT_ERR_PARAM) but, for
 * n == beams, out_score == scores.
 */
#define PSTAT_BEAM_MAX 64
#define PSTAT_BEAM_MAX_N 128
PSTAT_API int pstat_beam_workspace_size(int64_t B, int64_t beams, int64_t V, pstat_dtype dt,
                                        size_t* bytes);
PSTAT_API int pstat_beam_select(const void* logits, pstat_dtype dt, int64_t B, int64_t beams,
                                int64_t V, int64_t ld, const float* scores, int64_t n,
                                float* out_score, int64_t* out_parent, int64_t* out_token,
                                void* workspace, size_t ws_bytes, int* dev_error,
                                pstat_stream_t stream);

/*
 * Reordering of the beams' states: row b out_beams + i of every output becomes row
 * b beams + parents[b, i] of its input.  A row consists of `segments` runs of
 * seg_bytes bytes; all strides are in bytes.  In place (out == data for all states,
 * equal strides, beams == out_beams) rows of beams that are their own parent are not
 * touched.  An output may overlap nothing else of the call but, in place, its own
 * input (PSTAT_ERR_PARAM).  A row moves by vectors of 16, 8, 4, 2 or 1 bytes, as its
 * addresses, strides and runs allow, of which it may have 2^32 - 257 (PSTAT_ERR_SHAPE).
 * A parent of -1 leaves its row as it was, and so does one outside [0, beams), which sets
 * PSTAT_DEV_BAD_PARAM.
 */
typedef struct {
    const void* data;
    void* out;
    int64_t row_stride, out_row_stride;
    int64_t segments, seg_stride, out_seg_stride, seg_bytes;
} pstat_beam_state;
PSTAT_API int pstat_beam_reorder(const pstat_beam_state* states, int64_t n_states,
                                 const int64_t* parents, int64_t B, int64_t beams,
                                 int64_t out_beams, int* dev_error, pstat_stream_t stream);
/* The same into outputs that hold nothing yet: rows without a parent, -1 or outside
 * [0, beams), become zeros.  Not in place (PSTAT_ERR_PARAM). */
PSTAT_API int pstat_beam_gather(const pstat_beam_state* states, int64_t n_states,
                                const int64_t* parents, int64_t B, int64_t beams,
                                int64_t out_beams, int* dev_error, pstat_stream_t stream);

/*
 * Self-test of the bounded waits.  Every kernel of this library waits on its
 * mbarriers for at most a fixed time (2 s); a wait that runs out sets
 * PSTAT_DEV_TIMEOUT in *dev_error and the kernel winds down instead of
 * hanging the GPU.  This entry point runs one such wait, limited to
 * `limit_ns` nanoseconds (at most 1e9, else PSTAT_ERR_SHAPE), on a barrier
 * that nothing arrives at, with no copy in flight: afterwards *dev_error
 * (a device int, required) has PSTAT_DEV_TIMEOUT set and the context is
 * usable as before.  The pages have no counterpart; it exists to test the
 * library's failure path without faulting or hanging a GPU.
 */
PSTAT_API int pstat_selftest_wait_timeout(uint64_t limit_ns, int* dev_error,
                                          pstat_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PSTAT_H */
