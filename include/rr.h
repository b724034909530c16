/*
 * rr.h -- C ABI of librr.so: single-pass fused row reductions for GB300 (sm_103a).
 *
 * Operations (definitions from "Engineering a CUDA Machine Learning Framework
 * from Scratch", sec. 3.1 "Online FlashSoftmax", sec. 3.2 "Welford
 * Single-Pass Normalization", sec. 2.1 (loss gradients fused into registers)
 * and sec. 2.2 (pre-derived analytic backward); cross-entropy as in the
 * "gpu-ml-learning" README, Module 3):
 *   rr_softmax_fwd           y = softmax(x) per row
 *   rr_softmax_xent_fwd_bwd  per-row cross-entropy loss and dlogits = softmax - onehot
 *   rr_layernorm_fwd         y = (x - mean) * rstd * gamma + beta, saving mean / rstd
 *   rr_layernorm_bwd         dx, dgamma, dbeta from the saved mean / rstd
 * and, built on the same machinery:
 *   rr_log_softmax_fwd, rr_softmax_bwd, rr_log_softmax_bwd   the softmax pair
 *   rr_rmsnorm_fwd, rr_rmsnorm_bwd                           RMSNorm
 *   rr_attention_fwd         causal scaled dot-product attention on the online softmax
 *   rr_distill_fwd_bwd       distillation loss and dlogits from a teacher's top entries
 *   rr_attention_tree_fwd    attention of a tree of new tokens over a paged cache
 *   rr_draft_verify          acceptance of drafted tokens against the target
 *   rr_qk_norm_rope_fwd, rr_qk_norm_rope_bwd    norms of queries and keys with the rotation
 *   rr_attention_packed_fwd, rr_attention_packed_bwd   causal attention, packed sequences
 *   rr_token_logprob_fwd, rr_token_logprob_bwd  log probabilities of given tokens
 *   rr_layernorm_bwd_noalloc the LayerNorm backward without a caller workspace
 *   rr_selftest_bounded_wait, rr_read_device_error   the bounded device waits
 *
 * Common conventions
 *   - Every tensor is dense, row-major [rows x cols] with row stride = cols
 *     (per-column vectors are [cols], per-row vectors are [rows]), but where an
 *     argument named *_stride says how many elements lie between rows.
 *   - Every pointer is a DEVICE pointer on the current CUDA device, allocated
 *     and owned by the caller; the library allocates nothing and keeps no state
 *     beyond a per-device cache of attributes (and the fixed scratch array of
 *     rr_layernorm_bwd_noalloc).  Any alignment is accepted;
 *     16-byte aligned bases and rows whose byte length is a multiple of 16 take
 *     the vectorised path.
 *   - `dtype` (RR_F32 or RR_BF16) is the storage type of x, y, logits, dlogits,
 *     gamma, beta, dy, dx, dgamma and dbeta.  mean, rstd and loss are always
 *     float32 and labels int32.  Arithmetic is float32 on the GPU.
 *   - Calls are asynchronous on `stream` (0 = legacy default stream).
 *     Argument errors are returned synchronously and nothing is launched;
 *     launch errors are returned as RR_ERR_CUDA (detail string from
 *     rr_last_error_detail()); faults during execution surface at the caller's
 *     next synchronisation.  No C++ exception crosses this ABI.
 *   - rows == 0 is a no-op returning RR_OK.  cols must be >= 1.
 *   - Per-device state (attributes, the device addresses of the library's
 *     error word and scratch array) is resolved on the first call on a device
 *     and kept for the life of the process: it assumes the device's primary
 *     context lives that long.  After cudaDeviceReset of a device, do not call
 *     the library on that device again in the same process.
 *   - Waits inside the kernels are bounded; a wait that gives up records
 *     RR_ERR_DEVICE_TIMEOUT in a per-device error word read by
 *     rr_read_device_error(), and the kernel returns instead of hanging.
 *   - The kernel tier is chosen per call from the row's byte length, the
 *     pointers' alignment and the device.  The environment variable
 *     RR_FORCE_TIER (read at every call; for tests and tuning) forces one:
 *     0 spans of short rows through shared memory, 1 a row in registers,
 *     2 staged rows (one per CTA, bulk copies to shared memory), 3 rows split
 *     over a thread-block cluster.  A shape the forced tier cannot hold returns
 *     RR_ERR_INVALID_ARG; so does a value other than 0..3 (or T0..T3).
 *   - Rows of at least 8 KB whose row tensors share their address modulo 16
 *     run on kernels that group the rows by their start offset within a
 *     16-byte block (every chunk then an aligned 16-byte block), where measured
 *     faster.  RR_SMX=0 (softmax family) and RR_LNX=0 (LayerNorm / RMSNorm)
 *     turn them off, RR_LNP=0/1 and RR_SMB=1 choose among their variants (tests
 *     and tuning; read at every call).  LayerNorm / RMSNorm rows of at least
 *     64 KB (LayerNorm backward: 8 KB) with no forced tier run on column-block
 *     kernels (row statistics in one launch, the outputs in the next; the
 *     forward keeps its per-block statistics in y until it writes y, so it
 *     takes them only when y does not overlap x); RR_LNC=0 turns those off and
 *     RR_LNC_MIN (bytes) sets their threshold.  Rows of one column with no
 *     forced tier run on elementwise kernels (a one-element row is its own
 *     maximum, sum and moments); RR_ONE=0 turns those off.  Results agree
 *     within the tolerances of the operation whichever kernel runs; they are
 *     not bit-identical across kernels.
 *   - Softmax family range: the exponentials are taken as
 *     2^(x log2 e - fl(m log2 e)) times 2^(-r), r the rounding residual of
 *     fl(m log2 e) (m the row maximum).  For |m| >= 2^30 that residual can
 *     leave the float32 exponent range, and the row's outputs can then be NaN;
 *     finite logits below 2^30 in magnitude are always in range.
 *     rr_distill_fwd_bwd and rr_draft_verify take 2^((x - m) log2 e / T): any
 *     finite logits are in range.
 */
#ifndef RR_H
#define RR_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { RR_F32 = 0, RR_BF16 = 1 } rr_dtype;

typedef enum {
    RR_OK = 0,
    RR_ERR_INVALID_ARG = 1,         /* null pointer, negative size, cols == 0, bad eps */
    RR_ERR_UNSUPPORTED_DTYPE = 2,
    RR_ERR_ALIASING = 3,            /* partial overlap of an input and an output */
    RR_ERR_WORKSPACE_TOO_SMALL = 4,
    RR_ERR_CUDA = 5,                /* a CUDA runtime call failed */
    RR_ERR_DEVICE_TIMEOUT = 6       /* a bounded device-side wait gave up */
} rr_status;

/* Static, human-readable name of a status. */
const char *rr_status_string(rr_status status);

/* Detail of the last error returned on the calling host thread ("" if none). */
const char *rr_last_error_detail(void);

/*
 * Softmax forward ("Online FlashSoftmax", sec. 3.1): for each row,
 *   y_j = exp(x_j - m) / d,  m = max_j x_j,  d = sum_j exp(x_j - m),
 * with (m, d) computed in one pass over global memory by the online
 * normaliser and merged across threads with its pairwise rule.
 *   x, y : [rows x cols] dtype.  y == x (in place) is allowed; any other
 *          overlap returns RR_ERR_ALIASING.
 * A row whose maximum is -inf (fully masked) produces y = 0.
 */
rr_status rr_softmax_fwd(const void *x, void *y, int64_t rows, int64_t cols,
                         rr_dtype dtype, cudaStream_t stream);

/*
 * Log-softmax forward of each row: z_j = (x_j - m) - ln d with m = max_j x_j
 * and d = sum_j exp(x_j - m), from the same one-pass online normaliser as
 * rr_softmax_fwd (sec. 3.1).  x, z : [rows x cols] dtype (z == x allowed).
 * A fully masked row (maximum -inf) gives z = 0; a -inf entry of a live row
 * gives -inf.
 */
rr_status rr_log_softmax_fwd(const void *x, void *z, int64_t rows, int64_t cols,
                             rr_dtype dtype, cudaStream_t stream);

/*
 * Softmax backward, the vector-Jacobian product of y = softmax(x) (the
 * Softmax layer of the "NexusGrad" README's layer stack):
 *   dx_j = y_j * (dy_j - sum_k y_k dy_k).
 *   y : the forward's output, dy : upstream gradient, dx : [rows x cols] dtype.
 * dx may equal y or dy exactly (partial overlap is RR_ERR_ALIASING).  A fully
 * masked row (y = 0) gets dx = 0.
 */
rr_status rr_softmax_bwd(const void *y, const void *dy, void *dx, int64_t rows,
                         int64_t cols, rr_dtype dtype, cudaStream_t stream);

/*
 * Log-softmax backward, the vector-Jacobian product of z = log_softmax(x):
 *   dx_j = dz_j - exp(z_j) * sum_k dz_k.
 *   z : the forward's output, dz : upstream gradient, dx : [rows x cols] dtype.
 * dx may equal z or dz exactly.  The formula is applied to every row (a row
 * the forward masked to z = 0 has no derivative of its own).
 */
rr_status rr_log_softmax_bwd(const void *z, const void *dz, void *dx, int64_t rows,
                             int64_t cols, rr_dtype dtype, cudaStream_t stream);

/*
 * Fused softmax cross-entropy, forward and backward in one pass (sec. 2.1
 * and sec. 3.1; cross-entropy as in Module 3 of "gpu-ml-learning"):
 *   loss_r      = m + log d - logits[r, label_r]           (float32, [rows])
 *   dlogits_r,j = softmax(logits_r)_j - [j == label_r]     ([rows x cols] dtype)
 *   logits  : [rows x cols] dtype.   labels : [rows] int32.
 *   dlogits : may equal logits (written in place); other overlap is an error.
 *   ignore_index : a row whose label equals it gets loss 0 and dlogits 0 and
 *           its logits are not read (PyTorch's default is -100).
 *   bad_label_count : nullable device int32; each row whose label is outside
 *           [0, cols) and is not ignore_index adds 1.  Such a row gets loss NaN
 *           and dlogits equal to the plain softmax.  There is no trap.
 * A fully masked row (max = -inf) gets loss 0 and dlogits 0.
 * dlogits is not divided by the number of rows (loss is per row).
 */
rr_status rr_softmax_xent_fwd_bwd(const void *logits, const int32_t *labels,
                                  float *loss, void *dlogits, int64_t rows,
                                  int64_t cols, int32_t ignore_index,
                                  int32_t *bad_label_count, rr_dtype dtype,
                                  cudaStream_t stream);

/*
 * LayerNorm forward ("Welford Single-Pass Normalization", sec. 3.2): per row,
 *   mean = (1/C) sum_j x_j,  var = (1/C) sum_j (x_j - mean)^2 (biased),
 *   rstd = 1 / sqrt(var + eps),  y_j = (x_j - mean) * rstd * gamma_j + beta_j,
 * the moments from one pass over global memory: with the row (or its slice)
 * held on chip, an exact mean from a compensated sum and then the squared
 * deviations about it (row groups, clusters of them, spans); the staged
 * engine kernels, left for rows no row group or cluster of them takes, merge
 * per-thread moments with the Chan/Welford update.
 *   x, y : [rows x cols] dtype (y == x allowed).  gamma, beta : [cols] dtype.
 *   mean, rstd : [rows] float32 outputs, saved for rr_layernorm_bwd.
 *   eps : >= 0 and finite.
 * A row holding a non-finite value is masked: y = 0, mean = 0, rstd = 0.
 */
rr_status rr_layernorm_fwd(const void *x, const void *gamma, const void *beta,
                           void *y, float *mean, float *rstd, int64_t rows,
                           int64_t cols, float eps, rr_dtype dtype,
                           cudaStream_t stream);

/* Bytes of device workspace rr_layernorm_bwd needs for (rows, cols, dtype);
 * 0 if the arguments are invalid.  Depends on the current device. */
size_t rr_layernorm_bwd_workspace_size(int64_t rows, int64_t cols, rr_dtype dtype);

/*
 * LayerNorm backward (analytic derivative, sec. 2.2): with
 * xhat = (x - mean) * rstd and g = dy * gamma,
 *   dx_j     = rstd * (g_j - mean_j(g) - xhat_j * mean_j(g * xhat)),
 *   dgamma_j = sum_r dy_rj * xhat_rj,   dbeta_j = sum_r dy_rj.
 *   dy, x, dx : [rows x cols] dtype (dx may equal dy or x).  gamma, dgamma,
 *   dbeta : [cols] dtype.  mean, rstd : [rows] float32 from rr_layernorm_fwd.
 *   workspace : device scratch of workspace_bytes >= the size query's answer
 *   (16-byte aligned), owned by the caller; its contents on entry are ignored.
 * A row with rstd == 0 (masked by the forward) gets dx = 0 and adds nothing to
 * dgamma / dbeta.  dgamma / dbeta are summed over rows in a fixed order, so the
 * result is deterministic for a given device and shape.
 */
rr_status rr_layernorm_bwd(const void *dy, const void *x, const float *mean,
                           const float *rstd, const void *gamma, void *dx,
                           void *dgamma, void *dbeta, void *workspace,
                           size_t workspace_bytes, int64_t rows, int64_t cols,
                           rr_dtype dtype, cudaStream_t stream);

/*
 * RMSNorm forward ("NexusGrad" README, "Core Capabilities", which lists
 * RMSNorm among its transformer components without a formula; this library
 * takes the standard definition):
 *   ms = (1/C) sum_j x_j^2,  rstd = 1 / sqrt(ms + eps),  y_j = x_j * rstd * gamma_j.
 *   x, y : [rows x cols] dtype (y == x allowed).  gamma : [cols] dtype.
 *   rstd : [rows] float32 output, saved for rr_rmsnorm_bwd.  eps : >= 0, finite.
 * A row whose mean square is not finite is masked: y = 0, rstd = 0.  Rows of
 * any length run where x and y share their address modulo 16 and do not
 * overlap (the column-block kernels); otherwise rows must fit one row group of
 * threads or a thread-block cluster of up to 8 row groups (at least 65537
 * columns for fp32 and bf16, in every alignment), and longer rows return
 * RR_ERR_INVALID_ARG.
 */
rr_status rr_rmsnorm_fwd(const void *x, const void *gamma, void *y, float *rstd,
                         int64_t rows, int64_t cols, float eps, rr_dtype dtype,
                         cudaStream_t stream);

/* Bytes of device workspace rr_rmsnorm_bwd needs for (rows, cols, dtype); 0 if
 * the arguments are invalid or no kernel holds the rows.  Depends on the
 * current device. */
size_t rr_rmsnorm_bwd_workspace_size(int64_t rows, int64_t cols, rr_dtype dtype);

/*
 * RMSNorm backward (analytic derivative of rr_rmsnorm_fwd): with
 * xhat = x * rstd and g = dy * gamma,
 *   dx_j = rstd * (g_j - xhat_j * mean_j(g * xhat)),  dgamma_j = sum_r dy_rj * xhat_rj.
 *   dy, x, dx : [rows x cols] dtype (dx may equal dy or x).  gamma, dgamma : [cols]
 *   dtype.  rstd : [rows] float32 from rr_rmsnorm_fwd.
 *   workspace : device scratch of workspace_bytes >= the size query's answer
 *   (16-byte aligned), owned by the caller; its contents on entry are ignored.
 * A row with rstd == 0 gets dx = 0 and adds nothing to dgamma, which is summed
 * over rows in a fixed order (deterministic for a given device and shape).
 * Rows of any length run where dy, x and dx share their address modulo 16
 * (the column-block kernels); otherwise rows must fit one row group (at least
 * 8192 columns) or, with 16-byte aligned gamma, a thread-block cluster of up
 * to 8 row groups (beyond 65536 columns for fp32 and bf16), and longer rows
 * return RR_ERR_INVALID_ARG (the size query returns 0 when no kernel holds
 * them).
 */
rr_status rr_rmsnorm_bwd(const void *dy, const void *x, const float *rstd,
                         const void *gamma, void *dx, void *dgamma, void *workspace,
                         size_t workspace_bytes, int64_t rows, int64_t cols,
                         rr_dtype dtype, cudaStream_t stream);

/*
 * LayerNorm backward without a caller-provided workspace (this entry point has
 * no counterpart in the pages; it is a convenience of this library).
 * For callers that cannot allocate device memory at call time -- code under a
 * framework's memory planner that owns every allocation, plugin interfaces
 * that receive only input and output buffers, latency-critical paths where an
 * allocation is not allowed.  Same arguments, results and error behaviour as
 * rr_layernorm_bwd, minus the workspace: the column partials go to a scratch
 * array of 8 MiB inside the library, held on every GPU that loads the library
 * until the process exits.  This entry point allocates nothing (no cudaMalloc,
 * cudaFree or allocating library routine).
 *   - The launch is planned with no more column partials (2 * cols fp32 each)
 *     than 8 MiB holds, so shapes whose rr_layernorm_bwd plan would need more
 *     run with fewer row groups.  Rows too long for even one partial
 *     (cols > 1048576) return RR_ERR_WORKSPACE_TOO_SMALL.
 *   - Arguments are checked on the host first, with the same statuses as
 *     rr_layernorm_bwd; only then is the device touched.
 *   - The first call on each device resolves the scratch's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.
 *   - Every call on a device shares the one scratch array, which keeps the last
 *     call's contents.  Calls that overlap on the GPU (e.g. on two streams
 *     without ordering between them) race on it and give wrong dgamma / dbeta.
 */
rr_status rr_layernorm_bwd_noalloc(const void *dy, const void *x, const float *mean,
                                   const float *rstd, const void *gamma, void *dx,
                                   void *dgamma, void *dbeta, int64_t rows, int64_t cols,
                                   rr_dtype dtype, cudaStream_t stream);

/*
 * Scaled dot-product attention forward, causal or not, built on the online
 * softmax: the extension the source names for it ("Engineering a CUDA Machine
 * Learning Framework from Scratch", sec. 6.4, FlashAttention-style fusion of
 * the sec. 3.1 online normaliser; attention as defined by Vaswani et al.
 * 2017).  For each head b and query row i:
 *   s_j = scale * q_i . k_j over the keys j it may see (j <= i when causal),
 *   o_i = sum_j softmax(s)_j v_j,   lse_i = log sum_j exp(s_j).
 *   q, k, v, o : [bh x seq x head_dim] bf16 (dtype must be RR_BF16), 16-byte
 *   aligned, o must not overlap q, k or v.  lse : [bh x seq] float32, or NULL.
 *   head_dim : 64 or 128;  seq : a multiple of 64;  scale > 0 (usually
 *   1 / sqrt(head_dim)).
 * Products on the tensor cores (bf16 in, fp32 accumulate), softmax in fp32,
 * P rounded to bf16 for P V.  Other shapes or dtypes return
 * RR_ERR_INVALID_ARG / RR_ERR_UNSUPPORTED_DTYPE; bh == 0 or seq == 0 is a no-op.
 */
rr_status rr_attention_fwd(const void *q, const void *k, const void *v, void *o, float *lse,
                           int64_t bh, int64_t seq, int64_t head_dim, float scale, int causal,
                           rr_dtype dtype, cudaStream_t stream);

/*
 * Distillation from a teacher's top entries, forward and backward in one call
 * (the cross-entropy's counterpart for soft labels given as a short list).
 * With T = temperature, s = softmax(x / T) over the row's columns and the
 * teacher's list (i_k, v_k), k < K:
 *   tail = 0: t = softmax(v / T) over the list (v logits or log-probabilities);
 *     loss = T^2 sum_k t_k (ln t_k - ln s_{i_k});
 *   tail != 0: t_k = exp(v_k) (v log-probabilities at this temperature), and
 *     the mass outside the list, tt = max(0, 1 - sum_k t_k), is matched with
 *     the student's, st = the sum of s over the unlisted columns:
 *     loss = T^2 [sum_k t_k (ln t_k - ln s_{i_k}) + tt (ln tt - ln st)];
 *   dlogits_j = grad T [M s_j - sum_{k: i_k = j} t_k - (j unlisted) tt s_j / st],
 *     M = sum_k t_k + tt (1 without a tail).
 *   logits : [rows x cols] dtype.  top_index : [rows x k] int32, top_value :
 *           [rows x k] float32, 0 <= k <= 1024 (k == 0: both may be NULL).
 *   grad    : [rows] float32, the upstream gradient of the row's loss, or NULL (1).
 *   loss    : [rows] float32.  dlogits : [rows x cols] dtype, may equal logits
 *           (written in place); other overlap is an error.  NULL: loss only.
 *   temperature : 2^-120 to 2^120.
 *   bad_index_count : nullable device int32; each entry with index >= cols adds 1.
 * An entry with a negative index, or one >= cols, is absent.  An entry listed
 * twice counts with both values.  A value of -inf has weight 0 (with a tail its
 * column still counts as listed).  A row with no entry present (without a tail:
 * none of finite weight), or fully masked logits, gets loss 0 and dlogits 0.
 * A NaN or +inf logit, or a NaN value, makes the loss and dlogits of a row with an
 * entry present NaN.  The tail term is left out of a row whose unlisted columns hold
 * none of the student's mass (all below 2^-126 of its largest probability).
 */
rr_status rr_distill_fwd_bwd(const void *logits, const int32_t *top_index,
                             const float *top_value, const float *grad, float *loss,
                             void *dlogits, int64_t rows, int64_t cols, int64_t k,
                             float temperature, int tail, int32_t *bad_index_count,
                             rr_dtype dtype, cudaStream_t stream);

/* Bytes of device workspace rr_attention_tree_fwd needs for these sizes; 0 if
 * none, or if the arguments are invalid.  Depends on the current device. */
size_t rr_attention_tree_workspace_size(int64_t batch, int64_t nodes, int64_t heads,
                                        int64_t kv_heads, int64_t head_dim);

/*
 * Attention of new tokens over a paged cache: `nodes` tokens a sequence that
 * form a tree (drafted tokens), a chain (a chunk of a prompt) or are one (plain
 * decoding), with grouped heads.  The caller has written the keys and values of
 * the new tokens to the cache: node j of sequence b is at position
 * context_len[b] + j, and position p is row p % page_size of page
 * page_table[b, p / page_size].  For node i and head h (key head
 * h / (heads / kv_heads)), over the keys it sees -- every position below
 * context_len[b], and of the nodes itself and its ancestors --
 *   o = sum_j softmax(scale q . k)_j v_j,   lse = log sum_j exp(scale q . k_j).
 *   q, o : [batch x nodes x heads x head_dim] bf16 (dtype must be RR_BF16).
 *   k_cache, v_cache : [pages x page_size x kv_heads x head_dim] bf16, any
 *           page_size >= 1; all four 16-byte aligned; a page size that is a
 *           multiple of 16 takes the tensor-core path.
 *   page_table : [batch x table_width] int32; only entries that cover
 *           context_len[b] + nodes positions are read.  context_len : [batch]
 *           int32 (negative counts as 0).
 *   parents : [batch x nodes] int32, the node that each follows, -1 for the
 *           root, a parent before its children; at most 256 nodes.  NULL: a chain
 *           (node i follows i - 1).  A node whose chain of parents does not end
 *           at -1 (an entry below -1, or not below the node) is absent: it sees
 *           nothing.
 *   lse : [batch x nodes x heads] float32, or NULL.
 *   head_dim 64 or 128; heads a multiple of kv_heads; scale > 0 and finite.
 *   At most 65536 sequences, 2^20 nodes, 2^30 rows (batch x nodes x heads) and 2^30
 *   positions in a row of the table; batch x kv_heads x ceil(nodes x heads / kv_heads
 *   / 128) x (ceil(table positions / 64) + 1) at most 2^30.
 *   workspace : device scratch of workspace_bytes >= the size query's answer
 *           (16-byte aligned), owned by the caller; its contents on entry are
 *           ignored.  Calls that may overlap on the GPU need one each.
 * A row that sees nothing gets o = 0 and lse = -inf.  Positions beyond the
 * table, or on a page outside [0, pages), are not seen.  What stands at unseen
 * positions (NaN or infinities too) changes nothing.  Products on the tensor cores
 * (bf16 in, fp32 accumulate), softmax in fp32, its weights rounded to bf16 for their
 * product with V (page sizes that are no multiple of 16: kept in fp32).  The scores
 * scale q . k are below 2^30 in magnitude.
 */
rr_status rr_attention_tree_fwd(const void *q, const void *k_cache, const void *v_cache,
                                const int32_t *page_table, const int32_t *context_len,
                                const int32_t *parents, void *o, float *lse, void *workspace,
                                size_t workspace_bytes, int64_t batch, int64_t nodes,
                                int64_t heads, int64_t kv_heads, int64_t head_dim,
                                int64_t pages, int64_t page_size, int64_t table_width,
                                float scale, rr_dtype dtype, cudaStream_t stream);

/*
 * Verification of drafted tokens against the target's probabilities, from
 * given random numbers (speculative sampling, over a chain or a tree).  From
 * the root, at the node reached so far (row 0 for the root, row i + 1 for node
 * i): p = softmax(target row / T), q = softmax(draft row / T), from which the
 * node's children were drawn.  The children are tried in the order of their
 * index; with c = 0, W = 1 at first, child i with token x is accepted iff
 *   uniform_i * W * q_x < p_x - c q_x;
 * else c += W and W = sum_j max(p_j - c q_j, 0) (the residual distribution is
 * max(p - c q, 0) / W).  An accepted child is the next node.  When none is
 * accepted the walk ends with the token argmax_j max(p_j - c q_j, 0) / race_j,
 * the lowest j at a tie (over p itself where W = 0): with exponential noise a
 * draw from the residual.
 *   target_logits : [batch x (nodes + 1) x cols] dtype.
 *   draft_logits : [batch x nodes x cols] dtype; row r holds the distribution the
 *           children of node r - 1 were drawn from.  nodes == 0: may be NULL, as
 *           may tokens and uniform.
 *   tokens : [batch x nodes] int32; a token outside [0, cols) marks an absent
 *           node (never accepted, its siblings are tried as if it were not there).
 *   parents : [batch x nodes] int32 as for rr_attention_tree_fwd, or NULL (a chain).
 *   uniform : [batch x nodes] float32 in [0, 1).  race : [batch x cols] float32,
 *           2^-126 to 2^126.
 *   temperature : [batch] float32, or NULL (1).  <= 0: greedy, p and q are all on
 *           their row's largest logit (the lowest index at a tie).  So the first
 *           child tried is accepted iff it is the target's largest, a later one iff
 *           it is and the draft's largest is another; the last token is the
 *           target's largest.  So list a greedy tree's siblings by the draft's logit,
 *           the largest first: then no child that is the target's choice is refused.
 *           Otherwise finite and >= 2^-120.
 *   out_tokens : [batch x (nodes + 1)] int32, the accepted tokens, the last
 *           token, then -1.  out_nodes : [batch x (nodes + 1)] int32, the nodes
 *           of the accepted tokens, then -1.  out_count : [batch] int32, how many
 *           were accepted.
 *   At most 65535 nodes; cols < 2^31.
 * Rows of nodes that are not reached change nothing.  A target row without a
 * finite logit, or with a NaN or +inf one where it is softmaxed, ends the walk
 * with the last token -1.  A draft row with a NaN or +inf one has no child accepted,
 * and the last token is drawn from p.  Probabilities and quotients are float32: where
 * two sides of a test, or two scores, are equal within their rounding (some 1e-6,
 * relative), either answer may come, and another for rows that another kernel takes.
 */
rr_status rr_draft_verify(const void *target_logits, const void *draft_logits,
                          const int32_t *tokens, const int32_t *parents, const float *uniform,
                          const float *race, const float *temperature, int32_t *out_tokens,
                          int32_t *out_nodes, int32_t *out_count, int64_t batch, int64_t nodes,
                          int64_t cols, rr_dtype dtype, cudaStream_t stream);

/*
 * Norms of queries and keys, head by head, and the position rotation, in one pass
 * (RMSNorm of rr_rmsnorm_fwd over each head; rotary position embedding, Su et al.
 * 2021).  For each token and head, with x its head_dim values and w the weight:
 *   u = x w / sqrt(mean(x^2) + eps),
 *   y_a = cos u_a - sin u_b,  y_b = sin u_a + cos u_b  for the pairs p < rot_dim / 2,
 *   (a, b) = (p, p + rot_dim / 2), or (2p, 2p + 1) if interleaved; the elements from
 *   rot_dim on are not rotated (y = u).
 *   q, q_out : [tokens x heads x head_dim] dtype; k, k_out : [tokens x kv_heads x
 *           head_dim]; a token's heads are dense, tokens *_stride elements apart (views
 *           of a fused projection).  An output may be its input (written in place);
 *           other overlap is an error.  kv_heads == 0: k, k_out may be NULL.
 *   q_weight, k_weight : [head_dim] dtype, or NULL (1).
 *   cos, sin : [max_positions x rot_dim / 2] float32.
 *   positions : [tokens] int32 row of the table, or NULL (the token's index).
 *   bad_position_count : nullable device int32; each token with a position >=
 *           max_positions adds 1, and its rotated elements are NaN.
 *   head_dim even, at most 256; rot_dim even, 2 .. head_dim; at most 65535 heads; tokens
 *   below 2^31, strides at most 2^28 elements; eps >= 0 and finite.
 * A token with a negative position (padding) gets zeros, and so does a head whose mean
 * square is not finite, or zero with eps == 0.
 */
rr_status rr_qk_norm_rope_fwd(const void *q, const void *k, const void *q_weight,
                              const void *k_weight, const float *cos, const float *sin,
                              const int32_t *positions, void *q_out, void *k_out,
                              int64_t tokens, int64_t heads, int64_t kv_heads, int64_t head_dim,
                              int64_t rot_dim, int64_t max_positions, int64_t q_stride,
                              int64_t k_stride, int64_t q_out_stride, int64_t k_out_stride,
                              float eps, int interleaved, int32_t *bad_position_count,
                              rr_dtype dtype, cudaStream_t stream);

/* Bytes of device workspace rr_qk_norm_rope_bwd needs for these sizes; 0 if none,
 * or if the arguments are invalid.  Depends on the current device. */
size_t rr_qk_norm_rope_bwd_workspace_size(int64_t tokens, int64_t heads, int64_t kv_heads,
                                          int64_t head_dim);

/*
 * Gradient of rr_qk_norm_rope_fwd (its arguments have the same meaning and limits).
 * With g the gradient of a head's output turned back by the token's angles, r the
 * head's 1 / sqrt(mean(x^2) + eps) (computed again from q, k) and xh = x r:
 *   dx = r (g w - xh mean(g w xh)),   dw = sum over tokens and heads of g xh.
 *   dq_out, dk_out : gradients of q_out, k_out.  dq, dk : gradients of q, k; each may be
 *           the gradient it comes from, or q / k (written in place); other overlap is
 *           an error.
 *   dq_weight, dk_weight : [head_dim] dtype, or both NULL (not computed).
 *   workspace : device scratch of workspace_bytes >= the size query's answer (16-byte
 *           aligned), owned by the caller; its contents on entry are ignored.  Calls
 *           that may overlap on the GPU need one each.  Without weight gradients: NULL.
 * Heads that the forward set to zero get dx = 0 and add nothing to dw, which is summed
 * in a fixed order (the same bits at every run).  Positions beyond the table: NaN.
 */
rr_status rr_qk_norm_rope_bwd(const void *dq_out, const void *dk_out, const void *q, const void *k,
                              const void *q_weight, const void *k_weight, const float *cos,
                              const float *sin, const int32_t *positions, void *dq, void *dk,
                              void *dq_weight, void *dk_weight, void *workspace,
                              size_t workspace_bytes, int64_t tokens, int64_t heads,
                              int64_t kv_heads, int64_t head_dim, int64_t rot_dim,
                              int64_t max_positions, int64_t dq_out_stride, int64_t dk_out_stride,
                              int64_t q_stride, int64_t k_stride, int64_t dq_stride,
                              int64_t dk_stride, float eps, int interleaved,
                              int32_t *bad_position_count, rr_dtype dtype, cudaStream_t stream);

/*
 * Causal attention over packed sequences of differing lengths, with grouped heads: the
 * attention of whole prompts and of training (rr_attention_tree_fwd has the form for
 * single new tokens over a cache).  Sequence b is the tokens cu_seqlens[b] ..
 * cu_seqlens[b + 1] - 1; for its token i and head h (key head h / (heads / kv_heads)),
 * over the tokens j <= i of the sequence,
 *   o = sum_j softmax(scale q_i . k_j)_j v_j,   lse = log sum_j exp(scale q_i . k_j).
 *   q, o : [tokens x heads x head_dim] dtype; k, v : [tokens x kv_heads x head_dim]; a
 *           token's heads are dense, tokens *_stride elements apart.  16-byte aligned
 *           tensors whose strides and rows (head_dim) are whole 16-byte chunks.  o must
 *           not overlap another tensor.
 *   cu_seqlens : [batch + 1] int32, not decreasing, within 0 .. tokens (bounds outside
 *           are taken as the nearest; of decreasing bounds the results are not
 *           specified).  Sequences may be empty.  Rows of o and lse outside every
 *           sequence are left as they were.
 *   lse : [heads x tokens] float32, or NULL.
 *   head_dim at most 256; heads a multiple of kv_heads, at most 65535; batch at most
 *   2^20, tokens below 2^31 - 4096, tokens x heads at most 2^32, (tokens / 128 + batch) x
 *   heads at most 2^31, strides at most 2^28 elements; scale > 0 and finite.
 *   |scale q . k| below 2^30, and the sum of a sequence's |v| within float32.
 * bf16 with head_dim 64 or 128 runs on the tensor cores (fp32 accumulate; weights rounded
 * to bf16 for their product with v); other head dimensions and float32 on plain kernels.
 * What stands at unseen tokens (NaN or infinities too) changes nothing; a NaN or infinity that
 * a token sees makes its output's element such.  Neither costs time in rows of no sequence; a
 * NaN in a sequence costs its tiles' reading again, and up to 127 tokens before it are computed
 * again by the slower arithmetic of the plain kernels.
 */
rr_status rr_attention_packed_fwd(const void *q, const void *k, const void *v,
                                  const int32_t *cu_seqlens, void *o, float *lse, int64_t tokens,
                                  int64_t batch, int64_t heads, int64_t kv_heads,
                                  int64_t head_dim, int64_t q_stride, int64_t k_stride,
                                  int64_t v_stride, int64_t o_stride, float scale, rr_dtype dtype,
                                  cudaStream_t stream);

/* Bytes of device workspace rr_attention_packed_bwd needs for these sizes; 0 if
 * none, or if the arguments are invalid. */
size_t rr_attention_packed_bwd_workspace_size(int64_t tokens, int64_t heads);

/*
 * Gradient of rr_attention_packed_fwd (arguments of the same names have the same
 * meaning and limits).  With p = exp(scale q . k - lse), delta = dout . o and
 * ds = p (dout . v - delta):
 *   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij dout_i,
 * dk and dv over the tokens i of the sequence that see j and all heads of the key head.
 *   dout : gradient of o.  o, lse : what the forward gave for these q, k, v, scale.
 *   dq, dk, dv : gradients, of the shapes of q, k, v; they must not overlap another
 *           tensor (three views of one fused buffer, side by side, do not).
 *   workspace : device scratch of workspace_bytes >= the size query's answer (16-byte
 *           aligned), owned by the caller; its contents on entry are ignored.  Calls
 *           that may overlap on the GPU need one each.
 * Rows outside every sequence are left as they were, and nothing there or in another
 * sequence changes a sequence's gradients.  Every sum has a fixed order (the same bits at
 * every run).  On the tensor cores p and ds are rounded to bf16 for their products, and delta
 * of a sequence's first 128 tokens is sum_j p (dout . v_j), the same number without o's
 * rounding.  A NaN or infinity in a sequence may reach any gradient of that sequence.
 */
rr_status rr_attention_packed_bwd(const void *dout, const void *q, const void *k, const void *v,
                                  const void *o, const float *lse, const int32_t *cu_seqlens,
                                  void *dq, void *dk, void *dv, void *workspace,
                                  size_t workspace_bytes, int64_t tokens, int64_t batch,
                                  int64_t heads, int64_t kv_heads, int64_t head_dim,
                                  int64_t dout_stride, int64_t q_stride, int64_t k_stride,
                                  int64_t v_stride, int64_t o_stride, int64_t dq_stride,
                                  int64_t dk_stride, int64_t dv_stride, float scale,
                                  rr_dtype dtype, cudaStream_t stream);

/*
 * Log probabilities of given tokens, with what a sampler or a policy's loss wants beside
 * them, from one pass over each row.  With z = logits / temperature, t the row's token:
 *   logprob  = z_t - log sum_j exp z_j,
 *   entropy  = -sum_j p_j ln p_j,  p = softmax(z),
 *   row_max  = max_j logits_j,  log_sum = ln sum_j exp(z_j - row_max / temperature)
 *              (both kept for rr_token_logprob_bwd; their sum, row_max / temperature +
 *              log_sum, is the row's log-sum-exp),
 *   rank     = how many columns are before t by (logit descending, column ascending),
 *   top_index, top_logprob = the first k columns in that order, and their log
 *              probabilities.
 *   logits : [rows x cols] dtype, rows logits_stride >= cols elements apart.
 *   tokens : [rows] int32.  A row whose token is ignore_index is not read: it gets 0 (rank
 *           and top_index -1).
 *   logprob : [rows] float32; entropy, row_max, log_sum ([rows] float32) and rank ([rows]
 *           int32) may be NULL.  top_index, top_logprob : [rows x k] int32 and float32,
 *           0 <= k <= 128 (k == 0: NULL).
 *   temperature : 2^-120 to 2^120.
 *   bad_token_count : nullable device int32; each token outside [0, cols) (and not
 *           ignored) adds 1; such a row gets logprob NaN and rank -1.
 * Columns of -inf are not listed; places of the list that are left get index -1 and
 * -inf.  A row of nothing but -inf gets logprob, entropy and log_sum 0, row_max -inf and an
 * empty list.  A row with a NaN or +inf gets NaN, rank -1 and top_index -1.  A row whose list
 * ends among hundreds of equal columns (a vocabulary masked with a finite value that leaves
 * fewer than k columns) takes k more passes over it: mask with -inf.
 */
rr_status rr_token_logprob_fwd(const void *logits, const int32_t *tokens, float *logprob,
                               float *entropy, float *row_max, float *log_sum, int32_t *rank,
                               int32_t *top_index, float *top_logprob, int64_t rows, int64_t cols,
                               int64_t logits_stride, int64_t k, float temperature,
                               int32_t ignore_index, int32_t *bad_token_count, rr_dtype dtype,
                               cudaStream_t stream);

/*
 * Gradient of rr_token_logprob_fwd's logprob and entropy:
 *   dlogits_j = [g (1_{j=t} - p_j) - h p_j (ln p_j + entropy)] / temperature.
 *   row_max, log_sum, entropy : [rows] float32 from the forward (same temperature).
 *   grad_logprob (g), grad_entropy (h) : [rows] float32, or NULL (0); entropy may be NULL
 *           where grad_entropy is.
 *   dlogits : [rows x cols] dtype, rows dlogits_stride apart; may be logits, with the
 *           same stride (written in place); other overlap is an error.
 * A row whose token is ignore_index, or of nothing but -inf, gets 0.  A token outside
 * [0, cols) adds no 1_{j=t}.  rows x ceil(a row's bytes / 16384) below 2^31.
 */
rr_status rr_token_logprob_bwd(const void *logits, const int32_t *tokens, const float *row_max,
                               const float *log_sum, const float *entropy,
                               const float *grad_logprob, const float *grad_entropy, void *dlogits,
                               int64_t rows, int64_t cols, int64_t logits_stride,
                               int64_t dlogits_stride, float temperature, int32_t ignore_index,
                               rr_dtype dtype, cudaStream_t stream);

/*
 * Self-test of the bounded device-side waits (a diagnostic of this library;
 * the pages have no counterpart).  Launches one block that arms an mbarrier
 * for 16 bytes of bulk-copy data that no copy ever delivers and waits on it
 * with the same bounded wait the kernels use, giving up after limit_ns
 * nanoseconds of device time (1 .. 10^9; otherwise RR_ERR_INVALID_ARG).  The
 * wait gives up, RR_ERR_DEVICE_TIMEOUT is recorded in the current device's
 * error word (see rr_read_device_error) and the block returns; no memory of
 * the caller is touched and the context stays usable.  Asynchronous on
 * `stream`.
 */
rr_status rr_selftest_bounded_wait(int64_t limit_ns, cudaStream_t stream);

/*
 * Reads (and if `reset` is non-zero clears) the error word of `device` that
 * the kernels set when a bounded wait gives up.  *value receives 0 or an
 * rr_status such as RR_ERR_DEVICE_TIMEOUT.  Synchronous: it waits for the
 * device's outstanding work.
 */
rr_status rr_read_device_error(int device, int *value, int reset);

#ifdef __cplusplus
}
#endif

#endif /* RR_H */
