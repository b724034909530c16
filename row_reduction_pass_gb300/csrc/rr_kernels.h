// rr_kernels.h -- host-side view of the compiled kernel variants.
#pragma once

#include <cstdint>
#include <cuda_runtime_api.h>

namespace rr {

constexpr int kNumDirectG = 11;  // row groups of 1, 2, 4, ..., 1024 threads

// The variants of one operation for one storage type.  Index [m] is the mode:
// 0 = 16-byte chunks, 1 = single elements.
struct KernelSet {
  const void* direct[2][kNumDirectG];
  const void* staged[2];
  int nq_direct[2];
  int nq_staged[2];
  int maxt_direct;
  int maxt_staged;
};

// Row-group LayerNorm kernels (rr_ln.cuh).  Index [m][i]: m = 0 chunk mode
// with every row start 16-byte aligned, 1 chunk mode with any element
// alignment, 2 element mode; G = 2^i threads per row group.
constexpr int kNumLnG = 11;
struct LnKernelSet {
  const void* k[3][kNumLnG];
  int nq[3];  // chunks (elements in element mode) per thread
  // One chunk per thread, G <= 32 (backward: fewer registers, so more warps
  // per SM for short rows); null where not built.
  const void* k1[3][kNumLnG];
  // Forward rows split over a thread-block cluster: one group of 256 / 512 /
  // 1024 threads per block with nq chunks per thread, and [3] a 256-thread
  // group with 2 * nq; null where not built.
  const void* kc[3][4];
  // Chunk modes, rows of many chunks: nqd (> nq) chunks per thread so a row
  // needs fewer threads and each pays the per-row reductions over more data;
  // G >= 64 only, null where not built.
  const void* kd[2][kNumLnG];
  int nqd;
};

// Phase-aligned LayerNorm / RMSNorm kernels for long rows (rr_lnx.cuh):
// [rms][cluster]; nq_* chunks per thread.  Each function fills its half.
struct LnxKernels {
  const void* fwd[2][2];
  const void* bwd[2][2];
  const void* bwd2[2];  // backward, one block, at most 320 threads, two blocks per SM
  int nq_fwd, nq_bwd;
};
LnxKernels lnx_fwd_kernels_f32();
LnxKernels lnx_fwd_kernels_bf16();
LnxKernels lnx_bwd_kernels_f32();
LnxKernels lnx_bwd_kernels_bf16();

// Phase-aligned softmax-family kernels for long rows (rr_smx.cuh): [mode]
// [cluster], mode 0 softmax, 1 log-softmax, 2 cross-entropy; nq chunks per
// thread.
struct SmxKernels {
  const void* k[3][2];
  int nq;  // target chunks per thread
};
constexpr int kSmxMaxT = 512;  // threads per block

// Softmax / log-softmax backward for long rows (rr_smb.cuh): [log][cluster].
struct SmbKernels {
  const void* k[2][2];
};
SmbKernels smb_kernels_f32();
SmbKernels smb_kernels_bf16();

// Pipelined LayerNorm / RMSNorm kernels for long rows (rr_lnp.cuh): [rms]
// [cluster]; nq_bwd chunks per thread at most in the backward.
struct LnpKernels {
  const void* fwd[2][2];
  const void* bwd[2][2];
  const void* bwd2[2];  // backward, one block, at most 320 threads, two blocks per SM
  int nq_bwd;
};
LnpKernels lnp_fwd_kernels_f32();
LnpKernels lnp_fwd_kernels_bf16();
LnpKernels lnp_bwd_kernels_f32();
LnpKernels lnp_bwd_kernels_bf16();
SmxKernels smx_kernels_f32();
SmxKernels smx_kernels_bf16();

// Column-block LayerNorm / RMSNorm kernels for very long rows (rr_lnc.cuh):
// [rms].  Forward: stats, merge, norm launches; backward: part, dx launches
// (then the column reduce).  A work item (one block) is (class, column block,
// row group): item = cls + P * (b + nb * grp).
struct LncGeo {
  int64_t rows;
  int64_t cols;
  int32_t P;        // phase classes
  int32_t nb;       // column blocks of kCB chunks
  int32_t ng;       // row groups per class
  int32_t rg;       // rows per group (of its class)
  int32_t cb;       // chunks per column block (<= 32 * kLncWarps * CPL)
  int64_t rec_off;  // backward: floats from the workspace to the (S1, S2) records
};
constexpr int kLncWarps = 4;    // warps per block (128 threads)
constexpr int kLncCplFwd = 4;  // chunks per lane of a row, forward
constexpr int kLncCplBwd = 2;  // chunks per lane of a row, backward
constexpr int kLncDepth = 4;   // row stages of a block's copy ring (a pair of rows ahead)
// dynamic shared memory of a column-block kernel: its ring of row stages and
// their mbarriers
constexpr int lnc_ring_bytes(bool bwd) {
  return kLncDepth * (bwd ? 2 * kLncCplBwd : kLncCplFwd) * 32 * kLncWarps * 16 + 8 * kLncDepth;
}
struct LncKernels {
  const void* stats[2];
  const void* merge[2];
  const void* norm[2];
  const void* part[2];
  const void* dx[2];
};
LncKernels lnc_kernels_f32();
LncKernels lnc_kernels_bf16();

// LayerNorm / RMSNorm backward of short misaligned rows by phase class
// (rr_lns.cuh): bwd[rms][v], v = (lanes a row, chunks a lane): 0 (8, 1),
// 1 (16, 1), 2 (32, 1), and fp32 only (null for bf16) 3 (32, 2); a row of up
// to lanes x chunks 16-byte chunks, 32 / lanes rows a warp.  Blocks of
// kLnsWarps warps, one column partial ([planes][cols] floats) per block.
constexpr int kLnsWarps = 8;
struct LnsGeo {
  int64_t rows;
  int32_t cols;
  int32_t P;    // phase classes (divides kLnsWarps)
  int32_t hb0;  // byte of row 0 within its 16-byte block (x, dy and dx alike)
  int32_t rb;   // bytes per row
};
struct LnsKernels {
  const void* bwd[2][4];
};
LnsKernels lns_kernels_f32();
LnsKernels lns_kernels_bf16();

// Rows of one column (rr_one.cuh), elementwise: fwd [mode] 0 softmax,
// 1 log-softmax, 2 cross-entropy; bwd [log]; norm_fwd / norm_bwd [rms].
// Blocks of kOneThreads threads; the norm backward writes one partial
// (planes floats) per block.
constexpr int kOneThreads = 256;
struct OneKernels {
  const void* fwd[3];
  const void* bwd[2];
  const void* norm_fwd[2];
  const void* norm_bwd[2];
};
OneKernels one_kernels_f32();
OneKernels one_kernels_bf16();

// Short-row span kernels (rr_span.cuh): [dtype][mode], mode 0 softmax,
// 1 log-softmax, 2 cross-entropy, 3 softmax backward, 4 log-softmax backward,
// 5 LayerNorm forward, 6 RMSNorm forward, 7 LayerNorm backward, 8 RMSNorm
// backward.
struct SpanKernelSet {
  const void* k[2][9];
};
SpanKernelSet span_kernels();

KernelSet softmax_kernels_f32();
KernelSet softmax_kernels_bf16();
KernelSet softmax_bwd_kernels_f32();
KernelSet softmax_bwd_kernels_bf16();
KernelSet lnfwd_kernels_f32();
KernelSet lnfwd_kernels_bf16();
KernelSet lnbwd_kernels_f32();
KernelSet lnbwd_kernels_bf16();
LnKernelSet ln_fwd_rowgroup_kernels_f32();
LnKernelSet ln_fwd_rowgroup_kernels_bf16();
LnKernelSet ln_bwd_rowgroup_kernels_f32();
LnKernelSet ln_bwd_rowgroup_kernels_bf16();
LnKernelSet rms_fwd_rowgroup_kernels_f32();
LnKernelSet rms_fwd_rowgroup_kernels_bf16();
LnKernelSet rms_bwd_rowgroup_kernels_f32();
LnKernelSet rms_bwd_rowgroup_kernels_bf16();
// Scaled dot-product attention forward (k_attn.cu): bf16 [bh][seq][d]
// tensors, scores scaled by scale_log2 = scale * log2 e.
struct AttnParams {
  const char* q;
  const char* k;
  const char* v;
  char* o;
  float* lse;  // [bh][seq] natural-log sum of exp of the scaled scores, or null
  int* err;    // device error word (a bounded wait that gave up)
  int64_t bh;  // heads (batch x heads)
  int64_t seq;
  float scale_log2;
  int32_t causal;
};
struct AttnKernel {
  const void* fn;  // null for an unsupported head dimension
  int smem;        // dynamic shared memory bytes
};
AttnKernel attn_fwd_kernel_for(int d);
// Encodes the TMA tensor maps of q, k, v and launches the kernel for head
// dimension d on stream (persistent: at most `sms` CTAs): null on success,
// else a short reason (nothing launched, or the launch failed).
const char* attn_fwd_launch(const AttnParams& p, int d, int sms, cudaStream_t stream);
// Distillation from a teacher's top entries (k_distill.cu).
struct DistillParams {
  const char* x;         // [rows][cols] student logits
  const int32_t* index;  // [rows][k] listed columns; negative: absent
  const float* value;    // [rows][k] teacher logits, or log-probabilities (tail)
  const float* grad;     // [rows] upstream gradient of the loss, or null (1)
  float* loss;           // [rows]
  char* y;               // [rows][cols] dlogits, or null (loss only)
  int32_t* bad;          // counter of listed columns >= cols, or null
  int* err;              // device error word (a bounded wait that gave up)
  int64_t rows;
  int64_t cols;
  int32_t k;
  int32_t tail;          // keep the mass outside the list as one bucket
  uint32_t filter_bits;  // power of two >= 32
  float temperature;
  float inv_t, inv_t_lo;  // 1 / temperature in two parts
  float c;               // log2 e / temperature
};
// Launch geometry of the streaming kernel: a block (one of K of a cluster)
// holds a slice of S 16-byte chunks of a row, at most kDistNQ a row thread;
// byte offsets into its shared memory.
constexpr int kDistNQ = 7;
struct DistillGeo {
  int32_t S;
  int32_t words;     // 32-bit words of a slice's column bits
  int32_t list_off;  // lists: [4][k] 16-byte entries
  int32_t bits_off;  // column bits: [2][words]
  int32_t buf_off;   // rows: [2][S] chunks
};
struct DistillKernels {
  const void* rows;       // a block per row, any alignment and length
  int rows_threads;
  const void* stream[2];  // [cluster]
  int slots_off;          // stream: byte offset of the [4][K * (row warps + 1)] slots
};
DistillKernels distill_kernels(int dtype, bool tail);

// Verification of drafted tokens (k_verify.cu).
struct VerifyParams {
  const char* target;        // [batch][nodes + 1][cols] logits
  const char* draft;         // [batch][nodes][cols] logits
  const int32_t* tokens;     // [batch][nodes]; outside [0, cols): absent
  const int32_t* parents;    // [batch][nodes], or null (a chain)
  const float* uniform;      // [batch][nodes]
  const float* race;         // [batch][cols] exponential noise
  const float* temperature;  // [batch], or null (1)
  int32_t* out_tokens;       // [batch][nodes + 1]
  int32_t* out_nodes;        // [batch][nodes + 1]
  int32_t* out_count;        // [batch]
  int* err;
  int64_t batch;
  int64_t cols;
  int32_t nodes;
};
// Launch geometry of the cluster kernel: columns of a block's slice, byte
// offsets into its shared memory.
struct VerifyGeo {
  int32_t C;
  int32_t row_bytes;  // of a slice, with room for its head
  int32_t buf_off;    // [buffers][target, draft][row_bytes]
  int32_t buffers;    // 2: the first child's rows are loaded ahead
  int32_t noise_off;  // the noise's slice, -1: read from global memory
  int32_t nodes_off;  // tokens, parents, uniform numbers: 12 bytes a node
};
struct VerifyKernels {
  const void* block;  // a block per sequence, rows of any length
  int block_threads;
  const void* cluster;
};
VerifyKernels verify_kernels(int dtype);

// Attention of a tree of new tokens over a paged cache (k_tree.cu): bf16.
struct TreeParams {
  const char* q;              // [batch][nodes][heads][d]
  const char* k;              // [pages][page][kv_heads][d]
  const char* v;
  const int32_t* table;       // [batch][width] page of each page_size positions
  const int32_t* length;      // [batch] keys before the tree
  const int32_t* parents;     // [batch][nodes], or null (a chain)
  char* o;                    // [batch][nodes][heads][d]
  float* lse;                 // [batch][nodes][heads], or null
  float* ws;                  // partial results of split sequences
  int* err;
  int64_t batch, pages, width;
  int32_t nodes, heads, kv_heads, page;
  float scale_log2;           // scale * log2 e
};
constexpr int kTreeMaxNodes = 256;  // with parents (one mask bit a node)
const void* tree_rows_kernel(int d);
struct TreeGeo {
  int32_t box;        // positions of one tensor-map box, a power of two
  int32_t box_shift, page_shift;  // their logarithms (page: -1 if no power of two)
  int32_t G;          // heads per key head
  int32_t MT;         // row tiles per key head
  int32_t HB, RB;     // key heads and row tiles side by side in a group of pipelines
  int32_t side;       // HB * RB
  int32_t KM;         // items of a sequence: kv_heads / HB * MT / RB
  int32_t groups;     // of `side` pipelines
  int32_t cap;        // positions of the page table
  int32_t min_tiles;  // fewest key tiles of a run
  int32_t max_slots;  // pipelines
};
// fewest key tiles a pipeline takes: a shorter run would cost more in its
// piece's trip through the workspace than it saves (one token over 4001 keys of 8 key
// heads: 4 tiles 14.4 us, 3 15.3, 2 15.1; 16 trees of 30 nodes the same within 1 %)
constexpr int kTreeMinTiles = 4;
struct TreeKernels {
  const void* main;
  const void* join;
  int threads;
  int smem;
  int bn;  // keys per tile
};
TreeKernels tree_kernels(int d);
// Encodes the tensor maps and launches the two kernels (`sms` blocks): null on
// success, else a short reason.
const char* tree_tc_launch(const TreeParams& p, int d, int sms, cudaStream_t stream);
size_t tree_ws_bytes(int64_t batch, int64_t nodes, int heads, int kv_heads, int d, int sms);

// Norms of queries and keys with the position rotation (k_rope.cu).  Strides are in
// elements, from a token to the next.
struct RopeParams {
  const char *q, *k;          // [tokens][heads | kv_heads][dim]
  const char *qw, *kw;        // [dim], or null (1)
  const char *dyq, *dyk;      // backward: gradients of the outputs
  char *qo, *ko;              // outputs; backward: dq, dk
  const float *cos, *sin;     // [positions_n][rot / 2]
  const int32_t* positions;   // [tokens], or null (the token's index)
  int32_t* bad;               // counter of positions beyond the table, or null
  float* ws;                  // backward: [blocks][2][dim] sums, or null (no weight gradients)
  int64_t tokens, q_stride, k_stride, qo_stride, ko_stride, dyq_stride, dyk_stride;
  int64_t positions_n;
  int32_t heads, kv_heads, dim, rot;
  int32_t group;              // lanes of a row, a power of two
  int32_t q_segs, q_rows;     // a token's queries are cut into q_segs units of q_rows heads
  int32_t k_segs, k_rows;     // and its keys (none: k_segs 0)
  int32_t interleaved;
  float eps, inv_dim;
};
struct RopeKernels {
  const void *fwd, *bwd, *join;  // join: (sums, their rows, dim, two outputs), 32 columns a block
  int threads;                   // of the first two
};
// vec: slots of two 16-byte chunks, a row on up to 32 lanes; else of two elements.
RopeKernels rope_kernels(int dtype, bool vec);

// Log probabilities of given tokens (k_logprob.cu).  Strides in elements.
constexpr int kLogprobMaxK = 128;
struct LogprobParams {
  const char* x;          // [rows][cols] logits
  const int32_t* tokens;  // [rows]
  float *logprob, *entropy, *row_max, *log_sum;  // [rows]; all but the first may be null
  int32_t* rank;          // [rows], or null
  int32_t* top_index;     // [rows][k]
  float* top_logprob;     // [rows][k]
  int32_t* bad;           // counter of tokens out of range, or null
  int64_t rows, cols, stride;
  int32_t k, ignore;
  float temperature, c;   // c = log2 e / temperature
};
struct LogprobBwdParams {
  const char* x;
  const int32_t* tokens;
  const float *row_max, *log_sum, *entropy;  // entropy: null without h
  const float *g, *h;     // [rows] gradients of logprob and entropy, or null (0)
  char* y;                // dlogits
  int64_t rows, cols, x_stride, y_stride;
  int32_t segs, ignore;   // blocks a row
  float temperature, c;
};
struct LogprobKernels {
  const void* rows[2];     // [rank wanted] a row a block at a time
  const void* cluster[2];  // [rank wanted] a row on a cluster of up to 8 blocks
  const void* bwd[2];      // [elements, 16-byte chunks]
  int threads;             // of the cluster and backward kernels
  int rows_threads, rows_smem;
  int bwd_bytes;          // of a row that a block of the backward takes
};
LogprobKernels logprob_kernels(int dtype);

// Causal attention over packed sequences (k_packed.cu, k_packed_tc.cu).  Strides in
// elements, from a token to the next; heads are dim apart.
struct PackedParams {
  const char *q, *k, *v;      // [tokens][heads | kv_heads][dim]
  const char* o;              // the forward's output, the backward's input
  float* lse;                 // [heads][tokens]
  const int32_t* cu;          // [batch + 1] bounds of the sequences
  const char* dout;           // backward: gradient of o
  const char *dq, *dk, *dv;   // backward: outputs
  float* delta;               // backward: [heads][tokens] sums of dout o
  int* err;
  int64_t tokens, batch;
  int64_t sq, sk, sv, so, sdo, sdq, sdk, sdv;
  int32_t heads, kv_heads, dim;
  float scale, scale_log2;    // scale_log2 = scale log2 e
};
struct PackedRowKernels {
  const void *fwd, *dq, *dkv;
  int warps;                  // rows a block
};
PackedRowKernels packed_row_kernels(int dtype);
struct PackedTcKernels {
  const void *fwd, *delta, *bwd;
  int fwd_smem, bwd_smem;
};
// Tensor-core kernels for bf16 of this head dimension; fwd null where there are none.
PackedTcKernels packed_tc_kernels(int d, int64_t batch);
// Encodes the tensor maps and launches: null on success, else a short reason.
const char* packed_tc_fwd_launch(const PackedParams& p, int sms, cudaStream_t stream);
const char* packed_tc_bwd_launch(const PackedParams& p, int sms, cudaStream_t stream);

// The column reduce's split of its 32 warps over the P partial rows: the
// smallest power of two >= P / 16, at most 32 (the rest of the warps take
// further columns), so each warp sums about 16 partials.  A block covers
// 32 * (32 / split) columns.
inline __host__ __device__ int col_reduce_split(int64_t P) {
  int s = 1;
  while (s < 32 && (int64_t)s * 16 < P) s <<= 1;
  return s;
}
const void* col_reduce_kernel_ptr_f32();
const void* col_reduce_kernel_ptr_bf16();

}  // namespace rr
