// k_distill.cu -- distillation from a teacher's top entries: per-row loss and
// dlogits in one call (the sparse soft-label counterpart of the fused softmax
// cross-entropy; the loss of Hinton, Vinyals & Dean 2015 with its T^2 factor).
//
// Per row, with s = softmax(x / T) over all columns and the teacher's list
// (i_k, t_k), k < K:
//   loss    = T^2 [ sum_k t_k (ln t_k - ln s_{i_k}) + tt (ln tt - ln (Zt / Z)) ]
//   dx_j    = g T [ M s_j - [j unlisted] tt e_j / Zt - sum_{k: i_k = j} t_k ]
// e_j = exp((x_j - max) / T), Z = sum e, Zt = its part over unlisted columns,
// tt = the teacher's mass outside the list (0 when the list is renormalised),
// M = sum t + tt.  The student's mass is summed in two parts, Zt over the unlisted
// and Zl over the listed columns, and Z = Zt + Zl, so that neither part is the
// difference of two sums: Z - Zl loses every digit of Zt where the list holds nearly
// all of the mass, and where it holds little (a list of 4 of 131072 columns at T = 4:
// 6e-4 of it) ln tt and ln(Zt / Z), both near 0, are the logarithms of numbers near 1
// whose rounding, 2^-24, is a thousandth of them, and they nearly cancel against the
// list's terms.  So
//   ln tt = log1p(-sum t),   ln(Zt / Z) = log1p(-Zl / Z) where Zl < Z / 2,
//   M s_j - tt e_j / Zt = (e_j / Z) (sum t - tt Zl / Zt)   at an unlisted column
// (M Zt - tt Z = sum t Zt - tt Zl).  By the first forms the loss was off by up to 1e-3
// there (2-norm over the rows), by these 7e-6.
//
// Two kernels: one of rows in registers (below), and for rows whose logits and
// gradients differ in alignment, or that a cluster cannot hold, one of single-element
// accesses.  There a bit filter of up to 2^16 bits in shared memory holds (column mod
// its size) of the listed columns; a column whose bit is clear is unlisted, one whose
// bit is set is looked up in the list (only rows longer than the filter ever find it is
// not there).  Listed columns are stored again after the row's sweep, by the one
// thread whose entry is the first with that column.
#include <cstdint>

#include "rr_device.cuh"
#include "rr_kernels.h"

namespace rr {
namespace {

constexpr int kDistT = 256;

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < (int)(blockDim.x >> 5); ++i) v = fmaxf(v, red[i]);
  return v;
}
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int i = 1; i < (int)(blockDim.x >> 5); ++i) v += red[i];
  return v;
}

// The tail's part of the loss, tt (ln tt - ln(Zt / Z)), with tt = 1 - st > 0.
__device__ __forceinline__ float tail_loss(float st, float tt, float Z, float Zt, float Zl) {
  const float lns = Zl < 0.5f * Z ? log1pf(-Zl / Z) : logf(Zt / Z);
  return tt * (log1pf(-st) - lns);
}

// One block per row, single-element accesses: any alignment, any length.
template <int DT>
__global__ void __launch_bounds__(kDistT) distill_rows_kernel(const DistillParams p) {
  constexpr int E = DType<DT>::E;
  extern __shared__ __align__(128) unsigned char smem[];
  float* red = reinterpret_cast<float*>(smem);
  float* tval = red + 32;                                  // teacher values, then t_k
  float* tx = tval + p.k;                                  // the student's logits there
  int* tidx = reinterpret_cast<int*>(tx + p.k);            // columns, -1 absent
  uint32_t* filter = reinterpret_cast<uint32_t*>(tidx + p.k);
  __shared__ int s_dup;
  const int tid = threadIdx.x;
  const uint32_t fmask = p.filter_bits - 1;
  for (uint32_t i = tid; i < p.filter_bits / 32; i += kDistT) filter[i] = 0;
  if (tid == 0) s_dup = 0;
  __syncthreads();
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const char* x = p.x + r * p.cols * E;
    char* y = p.y != nullptr ? p.y + r * p.cols * E : nullptr;
    // the teacher's list
    float vm = -INFINITY;
    int any = 0;
    for (int i = tid; i < p.k; i += kDistT) {
      int j = p.index[r * p.k + i];
      const float v = p.value[r * p.k + i];
      if (j >= p.cols) {
        if (p.bad != nullptr) atomicAdd(p.bad, 1);
        j = -1;
      }
      tidx[i] = j;
      tval[i] = v;
      if (j >= 0) {
        any |= v == v ? 1 : 3;  // (a NaN is not a list without weight)
        vm = fmaxf(vm, v);
        tx[i] = ld_elem<DT>(x + (int64_t)j * E);
        const uint32_t b = (uint32_t)j & fmask;
        if (atomicOr(&filter[b >> 5], 1u << (b & 31)) & (1u << (b & 31))) s_dup = 1;
      }
    }
    const bool undefined = __syncthreads_or(any & 2);
    any = __syncthreads_or(any);
    vm = block_max(vm, red);
    const bool live = any && (p.tail || vm != -INFINITY || undefined);
    // the row's maximum and sums (online, per thread, then merged)
    float m = -INFINITY, d = 0.f, dt = 0.f, dl = 0.f;  // d: no tail
    if (live) {
      for (int64_t j = tid; j < p.cols; j += kDistT) {
        const float v = ld_elem<DT>(x + j * E);
        if (v > m) {
          const float a = ex2((m - v) * p.c);
          d *= a;
          dt *= a;
          dl *= a;
          m = v;
        }
        const float e = v == -INFINITY ? 0.f : ex2((v - m) * p.c);
        if (!p.tail) {
          d += e;
        } else {
          const uint32_t b = (uint32_t)j & fmask;
          bool listed = (filter[b >> 5] >> (b & 31)) & 1;
          if (listed && p.filter_bits < p.cols) {
            listed = false;
            for (int i = 0; i < p.k; ++i) listed = listed || tidx[i] == (int)j;
          }
          if (listed) dl += e;
          else dt += e;
        }
      }
    }
    const float M = block_max(m, red);
    const float a = m == -INFINITY ? 0.f : ex2((m - M) * p.c);
    const float Zt = p.tail ? block_sum(dt * a, red) : 0.f;
    const float Zl = p.tail ? block_sum(dl * a, red) : 0.f;
    const float Z = p.tail ? Zt + Zl : block_sum(d * a, red);
    const float g = p.temperature * (p.grad != nullptr ? p.grad[r] : 1.f);
    // (a row of NaN and -inf has a maximum of -inf too, but not a sum of 0)
    if (!live || (M == -INFINITY && Z == 0.f)) {  // no teacher, or nothing to learn from: zeros
      if (tid == 0) p.loss[r] = 0.f;
      if (y != nullptr)
        for (int64_t j = tid; j < p.cols; j += kDistT) st_elem<DT>(y + j * E, 0.f);
    } else {
      // t_k and the loss / T, T ln t_k - T ln s in the logits' own units
      const float lnZ = logf(Z);
      float lnt = 0.f;  // ln of the list's normaliser
      if (!p.tail) {
        float zt = 0.f;
        for (int i = tid; i < p.k; i += kDistT)
          if (tidx[i] >= 0) zt += expf((tval[i] - vm) * p.inv_t);
        lnt = logf(block_sum(zt, red));
      }
      float l = 0.f, st = 0.f;
      for (int i = tid; i < p.k; i += kDistT) {
        if (tidx[i] < 0) continue;
        const float lt = p.tail ? tval[i] : (tval[i] - vm) * p.inv_t - lnt;
        const float t = expf(lt);
        const float ltT = p.tail ? p.temperature * lt : (tval[i] - vm) - p.temperature * lnt;
        if (t > 0.f) l += t * (ltT - ((tx[i] - M) - p.temperature * lnZ));
        else if (t != t) l = t;
        st += t;
        tval[i] = t;
      }
      l = block_sum(l, red);
      st = block_sum(st, red);
      float mass = st == st ? 1.f : st, tt = 0.f;
      if (p.tail) {
        tt = Zt > 0.f ? fmaxf(1.f - st, 0.f) : 0.f;
        mass = st + tt;
        if (tt > 0.f) l += p.temperature * tail_loss(st, tt, Z, Zt, Zl);
      }
      if (Z != Z) l = Z;
      if (tid == 0) p.loss[r] = p.temperature * l;
      if (y != nullptr) {
        const float A = g * (mass / Z);                                  // listed
        const float U = p.tail ? g * ((st - (tt > 0.f ? tt * (Zl / Zt) : 0.f)) / Z) : A;
        for (int64_t j = tid; j < p.cols; j += kDistT) {
          const float v = ld_elem<DT>(x + j * E);
          const float e = v == -INFINITY ? 0.f : ex2((v - M) * p.c);
          st_elem<DT>(y + j * E, e * U);
        }
        __syncthreads();
        for (int i = tid; i < p.k; i += kDistT) {
          const int j = tidx[i];
          if (j < 0) continue;
          float t = tval[i];
          bool first = true;
          if (s_dup) {
            for (int n = 0; n < i; ++n) first = first && tidx[n] != j;
            if (first)
              for (int n = i + 1; n < p.k; ++n) t += tidx[n] == j ? tval[n] : 0.f;
          }
          if (first) {
            const float e = tx[i] == -INFINITY ? 0.f : ex2((tx[i] - M) * p.c);
            st_elem<DT>(y + (int64_t)j * E, e * A - g * t);
          }
        }
      }
    }
    __syncthreads();
    for (int i = tid; i < p.k; i += kDistT)
      if (tidx[i] >= 0) filter[((uint32_t)tidx[i] & fmask) >> 5] = 0;
    if (tid == 0) s_dup = 0;
    __syncthreads();
  }
}


// ------------------------------------------------------- rows in registers ---
//
// One block (or a cluster of K blocks, each with a slice of S 16-byte chunks)
// per row at a time, grid-stride over the rows; x and y share their address
// modulo 16, so a chunk of one is a chunk of the other whatever the row's
// alignment.  The block's last three warps, a merge warp and two list warps, are
// set apart from the rest, the row warps:
//   row warp, per row j: waits for the row and its list, takes its chunks into
//     registers, publishes the warp's maximum and sum to every block of the
//     cluster, waits for the merged statistics, stores its chunks of dlogits.
//   merge warp, per row j: waits until every warp has published row j, refills the
//     row's buffer with row j + 2 (one bulk copy), merges the partials and hands
//     the row's statistics to the other warps (every warp merging for itself
//     took 1000 cycles of a row's 10300, 2200 in a cluster of three).
//   list warp, per row j (of its parity): waits for row j's statistics, prepares
//     row j + 2's list, writes row j's loss, and, once row j + 1 is published (every
//     chunk of row j then stored), takes the listed columns out of row j + 2 (with a
//     tail) and stores row j's listed columns.
// So a block meets once a row (an mbarrier of the published statistics), the
// two latencies of a list (its entries, then the student's logits there) are a
// row ahead of their use, and two rows are in flight while one is worked on.
// One list warp alone was the bottleneck: 8192 x 50304 bf16 took 265 us without
// entries, 357 us with 64 a row, 451 us with 128 (54 rows a block).
//
// Bound: HBM (a row in, a row out), where a block has rows enough: 8192 x 50304 bf16
// with 64 entries 251 us, 97 % of the copy bandwidth.  With a tail and 100 entries
// (2048 x 50304, 13-14 rows a block) 82 us, 74 %: a row's chain of maximum, sum,
// meeting and outputs, 5.8 us, is longer than its traffic, 4.4.  In clusters the
// meeting adds 1 us to that: 255 x 65537 fp32 29 us, 68 %.  (Replayed in a graph.)
//
// Bits of the listed columns of a slice, by place in the slice, tell the list warp
// whether a column came twice.  (They also told the row warps which lanes to leave out
// of Zt, a byte a chunk: 8192 x 50304 bf16 with a tail and 100
// entries 372 us, and 299 us since the list warp takes them out of the landed row.)
struct __align__(16) DistHead {
  float g;        // upstream gradient times T
  float tn;       // t_k = tn * (the entries' t)
  float st;       // sum of t_k (with no tail 1, or NaN)
  int live;       // some entry has weight
  int dup;        // a column of this slice may be listed twice
  float m, d;     // maximum of the slice's listed columns, sum of exp((x - m) / T)
  float ref;      // the logit that a0 is relative to
  double a0;      // sum t_k (T ln t_k - top - (x - ref))
  float top;      // T times the greatest ln t_k (0 with no tail)
};
struct __align__(16) DistEntry {
  float t, x;  // the teacher's weight (before tn; 0: absent), the student's logit
  int place;   // element place in this block's slice, -1 none; + kDistAgain if listed before
  int pad;
};
constexpr int kDistAgain = 1 << 30;
constexpr int kDistOffSlots = 416;  // shared memory: statistics' slots on

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// The lanes of a chunk outside bytes [lo, hi) become -inf.
template <int DT>
__device__ __forceinline__ void dist_mask(uint4& c, int lo, int hi) {
  constexpr int E = DType<DT>::E;
#pragma unroll
  for (int e = 0; e < DType<DT>::V; ++e)
    if (e * E < lo || e * E >= hi) chunk_set_bits<DT>(c, e, DT == kBF16 ? 0xff80u : 0xff800000u);
}

template <int DT, bool TAIL, bool CL>
__global__ void __launch_bounds__(1024, 1) distill_stream_kernel(const DistillParams p,
                                                                const DistillGeo g) {
  constexpr int E = DType<DT>::E, W = DType<DT>::V, NQ = kDistNQ;
  extern __shared__ __align__(128) unsigned char smem[];
  const int nw = (int)(blockDim.x >> 5) - 3;  // row warps
  const int G = nw * 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int K = 1, rank = 0;
  if constexpr (CL) {
    K = (int)cluster_nrank();
    rank = (int)cluster_rank();
  }
  const int64_t owner = blockIdx.x / K, owners = gridDim.x / K;
  const int k = p.k;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);  // [2] the row has landed
  uint64_t* mrg = full + 2;                            // [4] statistics published
  uint64_t* ready = full + 6;                          // [2] the list is prepared
  uint64_t* done = full + 8;                           // [4] statistics merged
  DistHead* heads = reinterpret_cast<DistHead*>(smem + 96);      // [4]
  uint4* edges = reinterpret_cast<uint4*>(smem + 288);           // [2][2] a row's ragged chunks
  float4* final_ = reinterpret_cast<float4*>(smem + 352);        // [4] (M, Z, Zt, Zl) of a row
  float4* slots = reinterpret_cast<float4*>(smem + kDistOffSlots);  // [4][nslot]
  DistEntry* lists = reinterpret_cast<DistEntry*>(smem + g.list_off);  // [4][k]
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem + g.bits_off);     // [2][words]
  // with a tail the list warps publish too (the listed columns' part of Z)
  const int nwp = nw + (TAIL ? 1 : 0), nslot = K * nwp;
  const int64_t rowb = p.cols * E;
  const int k0 = rank * g.S;
  auto row_addr = [&](int64_t r) { return reinterpret_cast<uintptr_t>(p.x) + r * rowb; };
  // chunks of this rank's slice of a row that starts h bytes into its first chunk
  auto chunks = [&](int h) {
    const int n = (int)((h + rowb + 15) >> 4) - k0;
    return n < g.S ? n : g.S;
  };
  auto row_of = [&](int64_t j) { return owner + j * owners; };

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&ready[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&mrg[i], CL ? 1 : nslot);  // (in a cluster: the bytes of the slots)
      mbar_init(&done[i], 1);
    }
    fence_mbar_init();
  }
  for (int i = tid; i < 2 * g.words; i += blockDim.x) bits[i] = 0;
  if constexpr (CL) cluster_sync();  // peers arrive on this block's barriers
  else __syncthreads();

  bool dead = false;  // a wait gave up: later waits are skipped (the kernel still ends)
  // Waits until row j's statistics are merged (every warp of the cluster has then
  // published it).  No warp runs so late that the barrier's next phase, row j + 4,
  // ends before it looks: that row waits for this block's row warps and lists.
  auto merged = [&](int64_t j) {
    if (!dead) dead = !mbar_wait_bounded(&done[j & 3], (uint32_t)((j >> 2) & 1), p.err);
    return final_[j & 3];
  };
  // warp w's partial of row j, to the slots of every rank
  auto publish = [&](int64_t j, int w, float m, float d) {
    const float M = warp_max(m);
    const float a = m == -INFINITY ? 0.f : ex2((m - M) * p.c);
    d = warp_sum(d * a);
    float4* sl = slots + (j & 3) * nslot + rank * nwp + w;
    // (maximum, sum; with a tail the sum of unlisted, of listed columns)
    const float4 v = make_float4(M, w < nw ? d : 0.f, w < nw ? 0.f : d, 0.f);
    // (this row's predecessor is stored before its listed columns are: finish)
    __threadfence_block();
    __syncwarp();
    if constexpr (CL) {
      // lane t writes to rank t (one lane after the other took 5500 cycles a row for
      // four ranks)
      if (lane < K)
        st_async_f32x4(map_to_rank(sl, lane), map_to_rank(&mrg[j & 3], lane), v.x, v.y, v.z, v.w);
      __syncwarp();
    } else if (lane == 0) {
      *sl = v;
      mbar_arrive(&mrg[j & 3]);
    }
  };
  // the teacher's mass outside the list, and the weight of the student's softmax
  auto masses = [&](const DistHead& hd, float dt, float& mass, float& tt) {
    tt = TAIL && dt > 0.f ? fmaxf(1.f - hd.st, 0.f) : 0.f;
    mass = hd.st + tt;
  };
  // a row with no teacher, or nothing to learn from (a row of NaN and -inf has a maximum
  // of -inf too, but not a sum of 0)
  auto empty = [&](const DistHead& hd, float M, float d) {
    return !hd.live || (M == -INFINITY && d == 0.f);
  };

  int64_t asked = -1;  // the last row asked for
  auto load_row = [&](int64_t j) {
    if (row_of(j) >= p.rows || dead) return;
    // (the row before in this buffer has landed, unless the warps that use it gave up)
    if (j >= 2 && !mbar_wait_bounded(&full[j & 1], (uint32_t)(((j >> 1) - 1) & 1), p.err)) {
      dead = true;
      return;
    }
    asked = j;
    const uintptr_t a = row_addr(row_of(j));
    const uint32_t bytes = (uint32_t)chunks((int)(a & 15)) * 16u;
    mbar_arrive_expect_tx(&full[j & 1], bytes);
    bulk_load(smem + g.buf_off + (j & 1) * g.S * 16,
              reinterpret_cast<const void*>((a & ~uintptr_t(15)) + (int64_t)k0 * 16), bytes,
              &full[j & 1], policy_evict_first());
  };

  if (warp == nw) {
    // ------------------------------------------------------ the merge warp
    // (A slot is written again four rows later by warps that wait for the rows
    // between, which wait for this block's row warps, which wait for this warp.)
    // (the second row is asked for when the first is there, or all blocks' first rows
    // would come at the pace of two: 128 x 131072 bf16 21.2 -> 20.3 us; short rows the
    // same either way)
    if (lane == 0) load_row(0);
    if (row_of(0) < p.rows) dead = !mbar_wait_bounded(&full[0], 0, p.err);
    if (lane == 0) load_row(1);
    for (int64_t j = 0; row_of(j) < p.rows; ++j) {
      const uint32_t ph = (uint32_t)((j >> 2) & 1);
      if (CL && lane == 0) mbar_arrive_expect_tx(&mrg[j & 3], (uint32_t)(nslot * 16));
      if (!dead) {
        if constexpr (CL) dead = !mbar_wait_bounded_cluster(&mrg[j & 3], ph, p.err);
        else dead = !mbar_wait_bounded(&mrg[j & 3], ph, p.err);
      }
      if (lane == 0) load_row(j + 2);  // every row warp has taken its chunks of row j
      const float4* sl = slots + (j & 3) * nslot;
      float M = -INFINITY, d = 0.f, dt = 0.f, dl = 0.f;
      for (int i = lane; i < nslot; i += 32) M = fmaxf(M, sl[i].x);
      M = warp_max(M);
      for (int i = lane; i < nslot; i += 32) {
        const float4 t = sl[i];
        const float a = t.x == -INFINITY ? 0.f : ex2((t.x - M) * p.c);
        if (!TAIL) {
          d += t.y * a;
        } else {
          dt += t.y * a;
          dl += t.z * a;
        }
      }
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) {
        if (!TAIL) {
          d += __shfl_xor_sync(0xffffffffu, d, off);
        } else {
          dt += __shfl_xor_sync(0xffffffffu, dt, off);
          dl += __shfl_xor_sync(0xffffffffu, dl, off);
        }
      }
      if (TAIL) d = dt + dl;
      if (lane == 0) {
        final_[j & 3] = make_float4(M, d, dt, dl);
        mbar_arrive(&done[j & 3]);
      }
      __syncwarp();
    }
    // Copies of this block end before it does (they have, but where a wait gave up).
    if (lane == 0)
      for (int64_t j = asked > 0 ? asked - 1 : 0; j <= asked; ++j)
        mbar_wait_bounded(&full[j & 1], (uint32_t)((j >> 1) & 1), p.err);
    __syncthreads();
  } else if (warp > nw) {
    // ------------------------------------------------------ the list warps
    // a / T, 1 / T in two parts
    auto over_t = [&](float a) {
      const float q = a * p.inv_t;
      return isfinite(q) ? fmaf(a, p.inv_t, a * p.inv_t_lo) : q;
    };
    // The list of a row passes through registers, 4 entries a lane (lists of up
    // to 128) at a time: its entries are loaded one row before the student's
    // logits there, and those one row's wait before they are used.
    int ci[4];
    float cv[4], cx[4];
    auto load_entries = [&](int64_t j, int base) {
      const int64_t at = row_of(j) * k + base + lane;
      const bool any = row_of(j) < p.rows;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        ci[q] = -1;
        if (any && base + lane + 32 * q < k) {
          ci[q] = __ldg(p.index + at + 32 * q);
          cv[q] = __ldg(p.value + at + 32 * q);
        }
      }
    };
    auto load_logits = [&](int64_t j) {
      const char* x = p.x + row_of(j) * rowb;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (ci[q] >= 0 && ci[q] < p.cols) cx[q] = ld_elem<DT>(x + (int64_t)ci[q] * E);
    };
    // What a list says before the row's statistics are known: the weights t (with
    // no tail relative to the greatest, tn brings them to sum 1), its part of the
    // loss relative to a logit of its own, the listed columns' part of Z.  Every
    // entry is touched once, in registers.  The loss is summed divided by T, in the
    // logits' units (T ln t_k is v itself without a tail): it neither overflows nor
    // underflows where T^2 or 1 / T would.
    auto prepare = [&](int64_t j) {
      const int64_t r = row_of(j);
      if (r >= p.rows) return;
      const int h = (int)(row_addr(r) & 15);
      const int first = h / E - k0 * W;  // place of column 0
      DistEntry* li = lists + (j & 3) * k;
      uint32_t* bm = bits + (j & 1) * g.words;
      float vm = -INFINITY, ref = -INFINITY;
      int any = 0;
      // maxima over the list (a list of more than 128: a pass of its own)
      for (int base = 0;;) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (base + 32 * q >= k) break;
          if (ci[q] < 0) continue;
          if (ci[q] >= p.cols) {
            if (rank == 0 && p.bad != nullptr) atomicAdd(p.bad, 1);
            ci[q] = -1;
            continue;
          }
          any |= cv[q] == cv[q] ? 1 : 3;  // (a NaN is not a list without weight)
          vm = fmaxf(vm, cv[q]);
          ref = fmaxf(ref, cx[q]);
        }
        base += 128;
        if (base >= k) break;
        load_entries(j, base);
        load_logits(j);
      }
      any = (int)__reduce_or_sync(0xffffffffu, (unsigned)any);
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) {
        vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, off));
        ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, off));
      }
      if (ref == -INFINITY) ref = 0.f;
      const bool live = any && (TAIL || vm != -INFINITY || any == 3);
      // With a tail T v and x - ref are both about T ln Z, some tens, and their difference
      // a few units or less: so the greatest T v is taken off first (one rounding of the
      // small difference), and put back in double, next to T ln Z.  (With the terms as
      // they are: drawn cases up to 8e-6 off in the loss, 2-norm over the rows.)
      const float v0 = TAIL ? 0.f : vm, top = TAIL && isfinite(vm) ? p.temperature * vm : 0.f;
      float st = 0.f, d = 0.f, a0 = 0.f;
      int dup = 0;
      for (int base = 0; base < k; base += 128) {
        if (k > 128) {
          load_entries(j, base);
          load_logits(j);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (base + 32 * q >= k) break;
          const int i = base + 32 * q + lane;
          if (i >= k) continue;
          DistEntry en{0.f, 0.f, -1, 0};
          if (ci[q] >= 0 && ci[q] < p.cols) {
            const float v = cv[q] - v0, lt = TAIL ? v : over_t(v);
            en.x = cx[q];
            if (live) {
              en.t = expf(lt);
              st += en.t;
              if (!(en.t <= 0.f))
                a0 += en.t * ((TAIL ? fmaf(p.temperature, v, -top) : v) - (en.x - ref));
            }
            const int e = ci[q] + first;
            if (e >= 0 && e < g.S * W) {
              en.place = e;
              if ((atomicOr(&bm[e >> 5], 1u << (e & 31)) >> (e & 31)) & 1) {
                dup = 1;
                en.place |= kDistAgain;
              } else if (TAIL) {
                d += ex2((en.x - ref) * p.c);
              }
            }
          }
          li[i] = en;
        }
      }
      dup = __any_sync(0xffffffffu, dup);
      double a = (double)a0;
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, off);
        st += __shfl_xor_sync(0xffffffffu, st, off);
        if (TAIL) d += __shfl_xor_sync(0xffffffffu, d, off);
      }
      if (lane == 0) {
        DistHead hd;
        hd.g = p.temperature * (p.grad != nullptr ? __ldg(p.grad + r) : 1.f);
        hd.tn = TAIL ? 1.f : 1.f / st;
        hd.st = TAIL || st != st ? st : 1.f;
        hd.live = live;
        hd.dup = dup;
        hd.m = d > 0.f ? ref : d == d ? -INFINITY : ref;
        hd.d = d;
        hd.ref = ref;
        hd.top = top;
        // sum t ln t has ln t_k = lt - ln(sum of t) where the list is normalised
        hd.a0 = TAIL ? a : a / (double)st - (double)p.temperature * (double)logf(st);
        heads[j & 3] = hd;
      }
      __syncwarp();
      if (!TAIL && lane == 0) mbar_arrive(&ready[j & 1]);
    };
    // With a tail: the listed columns of row j become -inf where it has landed, so that
    // the row warps' sum is that of the unlisted ones.
    auto take_out = [&](int64_t j) {
      if (!TAIL || row_of(j) >= p.rows) return;
      if (!dead) dead = !mbar_wait_bounded(&full[j & 1], (uint32_t)((j >> 1) & 1), p.err);
      const DistEntry* li = lists + (j & 3) * k;
      char* buf = reinterpret_cast<char*>(smem + g.buf_off + (j & 1) * g.S * 16);
      for (int i = lane; i < k; i += 32)
        if (li[i].place >= 0) {
          char* at = buf + (li[i].place & (kDistAgain - 1)) * E;
          if constexpr (DT == kBF16) *reinterpret_cast<unsigned short*>(at) = 0xff80u;
          else *reinterpret_cast<float*>(at) = -INFINITY;
        }
      fence_proxy_async_smem();  // (before the copy that refills the buffer)
      __syncwarp();
      if (lane == 0) mbar_arrive(&ready[j & 1]);
    };
    auto clear_bits = [&](int64_t j) {
      const DistEntry* li = lists + (j & 3) * k;
      uint32_t* bm = bits + (j & 1) * g.words;
      for (int i = lane; i < k; i += 32)
        if (li[i].place >= 0) bm[(li[i].place & (kDistAgain - 1)) >> 5] = 0;
      __syncwarp();
    };
    // dlogits at row j's listed columns of this slice
    auto finish = [&](int64_t j, float M, float d, float dt) {
      const int64_t r = row_of(j);
      const DistHead hd = heads[j & 3];
      if (p.y == nullptr || empty(hd, M, d)) return;
      const int h = (int)(row_addr(r) & 15);
      const DistEntry* li = lists + (j & 3) * k;
      float mass, tt;
      masses(hd, dt, mass, tt);
      const float A = hd.g * (mass / d), B = hd.g * hd.tn;
      char* y = p.y + r * rowb - h + (int64_t)k0 * 16;
      for (int i = lane; i < k; i += 32) {
        const DistEntry en = li[i];
        if (en.place < 0 || en.place >= kDistAgain) continue;
        float t = en.t;
        if (hd.dup)
          for (int n = 0; n < k; ++n) t += li[n].place == (en.place | kDistAgain) ? li[n].t : 0.f;
        st_elem<DT>(y + en.place * E, fmaf(ex2((en.x - M) * p.c), A, -B * t));
      }
    };
    // The loss: a0 plus st times the distance of ref from T times the row's logarithm
    // of Z, two numbers of some tens whose sum is small, hence in double (a few
    // operations a row).
    auto write_loss = [&](int64_t j, float M, float d, float dt, float dl) {
      const DistHead hd = heads[j & 3];
      float l = 0.f;
      if (!empty(hd, M, d)) {
        const int ez = (__float_as_int(d) >> 23) - 127;
        const double lnz = (double)ez * 0.69314718055994531 +
                           (double)logf(__int_as_float(__float_as_int(d) - (ez << 23)));
        const double T = (double)p.temperature;
        double s = hd.a0 + (double)hd.st * (((double)M - (double)hd.ref) + T * lnz + (double)hd.top);
        float mass, tt;
        masses(hd, dt, mass, tt);
        if (tt > 0.f) s += T * (double)tail_loss(hd.st, tt, d, dt, dl);
        l = (float)(s * T);
        if (d != d) l = d;
      }
      if (lane == 0) p.loss[row_of(j)] = l;
    };
    int64_t j = warp - nw - 1;
    load_entries(j, 0);
    load_logits(j);
    prepare(j);
    take_out(j);
    load_entries(j + 2, 0);
    float M = 0.f, d = 0.f, dt = 0.f, dl = 0.f;
    bool open = false;  // the block's last row: listed columns still to be stored
    for (; row_of(j) < p.rows; j += 2) {
      load_logits(j + 2);
      if (TAIL)
        publish(j, nw, lane == 0 ? heads[j & 3].m : -INFINITY, lane == 0 ? heads[j & 3].d : 0.f);
      const float4 f = merged(j);
      M = f.x;
      d = f.y;
      dt = f.z;
      dl = f.w;
      clear_bits(j);
      prepare(j + 2);
      load_entries(j + 4, 0);
      if (rank == 0) write_loss(j, M, d, dt, dl);
      open = row_of(j + 1) >= p.rows;
      if (!open) {
        merged(j + 1);
        take_out(j + 2);
        finish(j, M, d, dt);
      }
    }
    __syncthreads();
    if (open) finish(j - 2, M, d, dt);
  } else {
    // ------------------------------------------------------- the row warps
    for (int64_t j = 0; row_of(j) < p.rows; ++j) {
      const int64_t r = row_of(j);
      const uintptr_t a = row_addr(r);
      const int h = (int)(a & 15);
      const int n = chunks(h);
      const int64_t nch = (h + rowb + 15) >> 4;                // chunks of the row
      const int last = (int)(nch - 1 - k0);                    // place of its last chunk
      const int tail_bytes = (int)(h + rowb - 16 * (nch - 1));
      const uint32_t ph = (uint32_t)((j >> 1) & 1);
      uint4* buf = reinterpret_cast<uint4*>(smem + g.buf_off + (j & 1) * g.S * 16);
      if (!dead) dead = !mbar_wait_bounded(&full[j & 1], ph, p.err);
      if (!dead) dead = !mbar_wait_bounded(&ready[j & 1], ph, p.err);
      // the lanes of the row's first and last chunk that belong to its
      // neighbours become -inf in the buffer, by the chunk's only reader (the
      // proxy fence orders this before the copy that refills the buffer)
      const int nq = n > tid ? (n - tid + G - 1) / G : 0;
      // (two rows' copies: a row's last chunk may be another thread's than that of the
      // row before, which reads its copy when it stores its outputs; by row j + 2 every
      // warp has published row j + 1, and so stored row j)
      uint4* edge = edges + 2 * (j & 1);
      const bool head = tid == 0 && rank == 0 && h != 0;
      const bool end = tail_bytes != 16 && last < n && tid + (nq - 1) * G == last;
      if (head || end) {
        if (head) dist_mask<DT>(buf[0], h, 16);
        if (end) dist_mask<DT>(buf[last], 0, tail_bytes);
        if (head) edge[0] = buf[0];
        if (end) edge[1] = buf[last];
        fence_proxy_async_smem();
      }
      uint4 v[NQ];
      float m = -INFINITY;
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        if (q >= nq) break;
        v[q] = buf[tid + q * G];
        if constexpr (DT == kBF16) {
          const uint32_t w = bf16x2_max(bf16x2_max(v[q].x, v[q].y), bf16x2_max(v[q].z, v[q].w));
          m = fmaxf(m, fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)));
        } else {
          m = fmaxf(fmaxf(m, fmaxf(__uint_as_float(v[q].x), __uint_as_float(v[q].y))),
                    fmaxf(__uint_as_float(v[q].z), __uint_as_float(v[q].w)));
        }
      }
      // sum of 2^((x - m) c)  (a share of -inf sums to 0; about 0 a NaN still gives NaN)
      const float about = m == -INFINITY ? 0.f : m;
      float d = 0.f, d1 = 0.f;
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        if (q >= nq) break;
#pragma unroll
        for (int i = 0; i < W; i += 2) {
          float t0, t1;
          scaled2(t0, t1, chunk_get<DT>(v[q], i), chunk_get<DT>(v[q], i + 1), about, p.c);
          add2(d, d1, d, d1, ex2(t0), ex2(t1));
        }
      }
      d += d1;
      publish(j, warp, m, d);
      const float4 fin = merged(j);
      const float M = fin.x, dt = fin.z, dl = fin.w;
      d = fin.y;
      if (p.y == nullptr) continue;
      char* y = p.y + r * rowb - h + (int64_t)k0 * 16;
      const DistHead hd = heads[j & 3];
      float f = 0.f;
      const bool zero = empty(hd, M, d);
      if (!zero) {
        float mass, tt;
        masses(hd, dt, mass, tt);
        // (of an unlisted column: the listed ones are stored again)
        const float u = TAIL ? hd.st - (tt > 0.f ? tt * (dl / dt) : 0.f) : mass;
        f = hd.g * (u / d);
      }
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        if (q >= nq || zero) break;
        float e[W];
#pragma unroll
        for (int i = 0; i < W; i += 2) {
          float t0, t1;
          scaled2(t0, t1, chunk_get<DT>(v[q], i), chunk_get<DT>(v[q], i + 1), M, p.c);
          mul2(e[i], e[i + 1], ex2(t0), ex2(t1), f, f);
        }
        if (!(head && q == 0) && !(end && q == nq - 1))
          st_chunk_stream(y + (int64_t)(tid + q * G) * 16, chunk_pack<DT>(e));
      }
      if (zero)
        for (int q = head ? 1 : 0; q < nq - (end ? 1 : 0); ++q)
          st_chunk_stream(y + (int64_t)(tid + q * G) * 16, make_uint4(0u, 0u, 0u, 0u));
      // the first and last chunk of a row that starts or ends inside one: the
      // row's own lanes, from the copies kept
      for (int s = 0; s < 2; ++s) {
        if (!(s == 0 ? head : end)) continue;
        const int lo = s == 0 ? h : (nch == 1 ? h : 0), hi = s == 0 && nch > 1 ? 16 : tail_bytes;
        if (s == 1 && head && nch == 1) continue;  // one chunk in all: done
        for (int i = lo; i < hi; i += E) {
          const float x = ld_smem_elem<DT>(reinterpret_cast<const char*>(edge + s) + i);
          st_elem<DT>(y + (s == 0 ? 0 : (int64_t)last * 16) + i,
                      zero ? 0.f : ex2((x - M) * p.c) * f);
        }
      }
    }
    __syncthreads();  // every chunk stored: the last row's listed columns may be
  }
  if constexpr (CL) cluster_sync();  // no peer still writes this block's slots
}

}  // namespace

DistillKernels distill_kernels(int dtype, bool tail) {
  DistillKernels d{};
  if (dtype == kBF16) {
    d.rows = (const void*)distill_rows_kernel<kBF16>;
    d.stream[0] = tail ? (const void*)distill_stream_kernel<kBF16, true, false>
                       : (const void*)distill_stream_kernel<kBF16, false, false>;
    d.stream[1] = tail ? (const void*)distill_stream_kernel<kBF16, true, true>
                       : (const void*)distill_stream_kernel<kBF16, false, true>;
  } else {
    d.rows = (const void*)distill_rows_kernel<kF32>;
    d.stream[0] = tail ? (const void*)distill_stream_kernel<kF32, true, false>
                       : (const void*)distill_stream_kernel<kF32, false, false>;
    d.stream[1] = tail ? (const void*)distill_stream_kernel<kF32, true, true>
                       : (const void*)distill_stream_kernel<kF32, false, true>;
  }
  d.rows_threads = kDistT;
  d.slots_off = kDistOffSlots;
  return d;
}

}  // namespace rr
