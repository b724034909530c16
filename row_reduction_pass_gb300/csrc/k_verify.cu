// k_verify.cu -- verification of drafted tokens against the target's
// probabilities (speculative sampling of Leviathan, Kalman & Matias 2023 and
// Chen et al. 2023, over a tree: at a node the drafted children are tried one
// after the other, as in Miao et al. 2024).
//
// At the node reached so far, p = softmax(target / T) and q = softmax(draft /
// T), the distribution its children were drawn from.  A child with token x is
// accepted with probability min(1, r_x / q_x), r the current residual (p at
// first); a rejection replaces r by max(r - q, 0) / sum.  Written without the
// divisions: after t rejections r = max(p - c q, 0) / W, with c_0 = 0, W_0 =
// 1, c_{t+1} = c_t + W_t, W = sum_j max(p_j - c q_j, 0), because max(max(a, 0)
// - b, 0) = max(a - b, 0) for b >= 0.  So a node's state is two numbers, and a
// child is accepted iff u W q_x < p_x - c q_x.  When no child is accepted the
// token is drawn from the residual as argmax_j max(p_j - c q_j, 0) / e_j with
// given exponential noise e (of independent exponentials with rates w_j the
// smallest is j's with probability w_j / sum w), the lowest index at a tie.
//
// A sequence at temperature <= 0 has p and q all on their largest logits (the lowest
// index at a tie), and the same formulas: the first child tried is accepted iff it is
// p's token; a rejected one leaves max(p - c q, 0) = p, or nothing if q's token is
// p's.  So a later child is accepted iff it is p's token and q's is another, and q is
// looked at only for such a child.
//
// Only the rows of visited nodes are read: the walk depends on the tokens
// accepted so far.
//
// A cluster of K blocks walks a sequence, each with a slice of the columns: the
// slices of a node's two rows come to shared memory by bulk copies and stay there
// for every pass over them (maximum and sum, the residual's mass after each rejection,
// the final draw), so a row is read from memory once.  After each pass every warp
// puts its partial into a slot of every block of the cluster and arrives on its
// mbarrier; every warp then merges all slots in the same order, so all threads of
// the cluster hold the same numbers and take the same decisions.  With few
// sequences a walk is bound by latency (a row's 1.5-2 us, then about 0.6 us a
// meeting), so the first child's rows are loaded while its parent's are worked
// on; with many it is bound by memory, several clusters share an SM, and nothing
// is loaded that the walk does not reach.  Measured (in a graph): one chain of 5 over
// 50304 bf16 columns 19 us, 8 trees of 39 over 65537 fp32 columns 25.7 us, 256 chains
// of 8 over 50304 88 us (the cluster's meetings and exponentials; reading the rows
// visited takes 32).  Rows that a cluster cannot hold go to
// a kernel of one block per sequence that reads them again for every pass.
#include <cstdint>

#include "rr_device.cuh"
#include "rr_kernels.h"

namespace rr {
namespace {

constexpr int kVerT = 512;    // a block a sequence
constexpr int kVerClT = 256;  // a cluster a sequence, threads per block

struct BestTok {
  float s;
  int j;  // -1 none
  __device__ __forceinline__ void take(float s2, int j2) {
    if (j2 >= 0 && (j < 0 || s2 > s || (s2 == s && j2 < j))) {
      s = s2;
      j = j2;
    }
  }
};

struct VerRed {
  float f[32];
  int j[32];
};

__device__ __forceinline__ float ver_max(float v, VerRed& red) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red.f[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red.f[0];
  for (int i = 1; i < kVerT / 32; ++i) v = fmaxf(v, red.f[i]);
  return v;
}
__device__ __forceinline__ float ver_sum(float v, VerRed& red) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red.f[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red.f[0];
  for (int i = 1; i < kVerT / 32; ++i) v += red.f[i];
  return v;
}
__device__ __forceinline__ BestTok ver_best(BestTok b, VerRed& red) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    const float s = __shfl_xor_sync(0xffffffffu, b.s, off);
    const int j = __shfl_xor_sync(0xffffffffu, b.j, off);
    b.take(s, j);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    red.f[threadIdx.x >> 5] = b.s;
    red.j[threadIdx.x >> 5] = b.j;
  }
  __syncthreads();
  for (int i = 0; i < kVerT / 32; ++i) b.take(red.f[i], red.j[i]);
  return b;
}

// softmax(row / T) as (maximum, 1 / sum): prob(x) = 2^((x - m) c) * inv; a row
// without a finite logit has probability 0 everywhere
struct VerRow {
  const char* x;
  float m, inv;
  template <int DT>
  __device__ __forceinline__ float prob(int64_t j, float c) const {
    const float v = ld_elem<DT>(x + j * DType<DT>::E);
    return v == -INFINITY ? 0.f : ex2((v - m) * c) * inv;
  }
};
template <int DT>
__device__ __forceinline__ VerRow ver_row(const char* x, int64_t cols, float c, VerRed& red) {
  float m = -INFINITY, d = 0.f;
  for (int64_t j = threadIdx.x; j < cols; j += kVerT) {
    const float v = ld_elem<DT>(x + j * DType<DT>::E);
    if (v > m) {
      d *= ex2((m - v) * c);
      m = v;
    }
    d += v == -INFINITY ? 0.f : ex2((v - m) * c);
  }
  const float M = ver_max(m, red);
  const float Z = ver_sum(m == -INFINITY ? d : d * ex2((m - M) * c), red);
  return {x, M, Z == 0.f ? 0.f : 1.f / Z};
}

// One block per sequence.
template <int DT>
__global__ void __launch_bounds__(kVerT) verify_kernel_t(const VerifyParams p) {
  constexpr int E = DType<DT>::E;
  __shared__ VerRed red;
  const int64_t b = blockIdx.x, V = p.cols;
  const int n = p.nodes, tid = threadIdx.x;
  const int32_t* tok = p.tokens + b * n;
  const int32_t* par = p.parents != nullptr ? p.parents + b * n : nullptr;
  const float T = p.temperature != nullptr ? p.temperature[b] : 1.f;
  const bool greedy = T <= 0.f;
  const float c = kLog2e / T;
  int cur = -1, done = 0;
  int32_t token = -1;
  for (;;) {
    const char* tr = p.target + ((b * (n + 1) + cur + 1) * V) * E;
    const char* dr = p.draft + ((b * n + cur + 1) * V) * E;
    VerRow pr{}, qr{};
    auto row_top = [&](const char* x) {
      BestTok t{0.f, -1};
      for (int64_t j = tid; j < V; j += kVerT) {
        const float v = ld_elem<DT>(x + j * E);
        if (v > -INFINITY) t.take(v, (int)j);
      }
      return ver_best(t, red);
    };
    BestTok top{0.f, -1};
    if (greedy) {
      top = row_top(tr);
    } else {
      pr = ver_row<DT>(tr, V, c, red);
    }
    float ratio = 0.f, mass = 1.f;
    bool have_q = false, first = true;
    int next = -1;
    for (int i = cur + 1; i < n && next < 0; ++i) {
      const int32_t x = tok[i];
      if ((par != nullptr ? par[i] : i - 1) != cur || x < 0 || x >= V) continue;
      if (greedy) {
        if (x == top.j) {
          if (!first && row_top(dr).j == top.j) break;  // nothing of the target is left
          next = i;
        }
        first = false;
        continue;
      }
      if (!have_q) {
        qr = ver_row<DT>(dr, V, c, red);
        have_q = true;
      }
      const float px = pr.prob<DT>(x, c), qx = qr.prob<DT>(x, c);
      if (p.uniform[b * n + i] * mass * qx < px - ratio * qx) {
        next = i;
      } else {
        ratio += mass;
        float w = 0.f;
        for (int64_t j = tid; j < V; j += kVerT) {
          const float t = pr.prob<DT>(j, c) - ratio * qr.prob<DT>(j, c);
          w += t < 0.f ? 0.f : t;
        }
        mass = ver_sum(w, red);
        if (!(mass > 0.f)) break;  // nothing of the target is left
      }
    }
    if (next >= 0) {
      if (tid == 0) {
        p.out_tokens[b * (n + 1) + done] = tok[next];
        p.out_nodes[b * (n + 1) + done] = next;
      }
      ++done;
      cur = next;
      continue;
    }
    if (greedy) {
      token = top.j;
    } else {
      if (!(mass > 0.f)) ratio = 0.f;
      BestTok best{0.f, -1};
      for (int64_t j = tid; j < V; j += kVerT) {
        float w = pr.prob<DT>(j, c);
        if (ratio > 0.f) w -= ratio * qr.prob<DT>(j, c);
        if (w > 0.f) {
          const float s = w / p.race[b * V + j];
          if (s >= 0.f) best.take(s, (int)j);
        }
      }
      token = ver_best(best, red).j;
    }
    break;
  }
  for (int i = done + tid; i <= n; i += kVerT) {
    p.out_tokens[b * (n + 1) + i] = i == done ? token : -1;
    p.out_nodes[b * (n + 1) + i] = -1;
  }
  if (tid == 0) p.out_count[b] = done;
}

// ------------------------------------------------------ a cluster a sequence ---
//
// Per node: rows landed -> each thread's maximum and sum over its share of both
// slices -> block -> cluster (one meeting) -> the children's tests, a pass and a
// meeting for each rejection -> next node, or the draw (a pass and a meeting).
// Measured on one chain of 50304 bf16 columns (K = 8): first version, 256 threads
// and an IEEE division per column in the draw, 2800 cycles for the statistics and
// 10000 for the draw (29 us; now 19); hence the packed exponents, the chunk-wise maxima (a token
// is only looked for in a chunk that beats the best so far), and a warp of its own
// that issues the loads (the address arithmetic and the copies held its warp up for
// 1300 cycles a node).
//
// p = 2^((x - M) c) / Z, the maximum taken off before the scaling: in the form
// 2^(x c - fl(M c)), one packed operation less, the rounding residual of fl(M c) is
// greater than a float32 exponent for |M| c > 2^31, which masks of -1e10 or the
// type's lowest value reach (a thread whose columns are all masked has such a
// maximum), and so do ordinary logits at temperatures of 1e-9 and below.

// The greatest of a chunk's W scores, and the first place it stands at.
template <int W>
__device__ __forceinline__ void best_chunk(BestTok& best, const float (&s)[W], int j) {
  float m = s[0];
#pragma unroll
  for (int e = 1; e < W; ++e) m = fmaxf(m, s[e]);
  // (a thread's chunks come in ascending order: an equal score later loses)
  if (best.j < 0 ? m >= 0.f : m > best.s) {
    int at = 0;
#pragma unroll
    for (int e = W - 1; e >= 0; --e) at = s[e] == m ? e : at;
    best.s = m;
    best.j = j + at;
  }
}

template <int DT>
__global__ void __launch_bounds__(kVerClT, 4) verify_cluster_kernel(const VerifyParams p,
                                                                   const VerifyGeo g) {
  constexpr int E = DType<DT>::E, W = DType<DT>::V;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int NT = blockDim.x - 32, NW = NT >> 5;  // the working warps; then the loading one
  const bool works = warp < NW;
  const int K = (int)cluster_nrank(), rank = (int)cluster_rank();
  const int64_t b = blockIdx.x / K, V = p.cols;
  const int n = p.nodes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);       // [2] a node's rows have landed
  uint64_t* met = full + 2;                                 // [2] the blocks' partials published
  uint64_t* noise_bar = full + 4;
  float4* slots = reinterpret_cast<float4*>(smem + 64);     // [3][K * NW] partials
  const int nslot = K * NW;
  int32_t* tok = reinterpret_cast<int32_t*>(smem + g.nodes_off);  // [n] -1: absent
  int32_t* par = tok + n;
  float* uni = reinterpret_cast<float*>(par + n);
  const float T = p.temperature != nullptr ? __ldg(p.temperature + b) : 1.f;
  const bool greedy = T <= 0.f;
  const float c = kLog2e / T;
  const int64_t c0 = (int64_t)rank * g.C;                   // this block's columns
  const int nc = (int)max((int64_t)0, min((int64_t)g.C, V - c0));

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&met[i], 1);
    }
    mbar_init(noise_bar, 1);
    fence_mbar_init();
  }
  for (int i = tid; i < n; i += blockDim.x) {
    const int32_t x = __ldg(p.tokens + b * n + i);
    tok[i] = x >= 0 && x < V ? x : -1;
    par[i] = p.parents != nullptr ? __ldg(p.parents + b * n + i) : i - 1;
    uni[i] = __ldg(p.uniform + b * n + i);
  }
  cluster_sync();  // peers arrive on this block's barriers

  // A wait gave up, in any thread of the block (the threads agree on it after every
  // wait, since they meet at block barriers): the walk ends.
  bool dead = false;
  bool late = false;  // this thread gave up since they last agreed
  auto agree = [&](bool ok) { dead = __syncthreads_or(dead || late || !ok); };
  auto trow = [&](int node) { return p.target + ((b * (n + 1) + node + 1) * V) * E; };
  auto drow = [&](int node) { return p.draft + ((b * n + node + 1) * V) * E; };
  // A slice of a row in shared memory: its first element is h bytes into the buffer.
  auto head = [&](const char* row) {
    return (int)((reinterpret_cast<uintptr_t>(row) + (uint64_t)c0 * E) & 15);
  };
  auto pbuf = [&](int s) { return smem + g.buf_off + s * 2 * g.row_bytes; };
  // the next child of `cur` from node i on, -1 if none (every warp by itself)
  auto next_child = [&](int cur, int i) {
    for (int base = i & ~31; base < n; base += 32) {
      const int j = base + lane;
      const uint32_t m =
          __ballot_sync(0xffffffffu, j >= i && j < n && par[j] == cur && tok[j] >= 0);
      if (m != 0) return base + __ffs(m) - 1;
    }
    return -1;
  };
  int loads[2] = {0, 0};  // of each buffer (the same count in every thread)
  // brings a node's rows to buffer s (the draft's if a child is to be tried)
  auto load_rows = [&](int node, int child, int s) {
    ++loads[s];
    if (tid != NT || dead) return;
    const char* t = trow(node);
    const char* d = drow(node);
    const bool draft = child >= 0 && !greedy;
    const uint32_t tb = nc > 0 ? (uint32_t)((head(t) + nc * E + 15) & ~15) : 0;
    const uint32_t db = draft && nc > 0 ? (uint32_t)((head(d) + nc * E + 15) & ~15) : 0;
    mbar_arrive_expect_tx(&full[s], tb + db);
    if (tb > 0)
      bulk_load(pbuf(s), t + c0 * E - head(t), tb, &full[s], policy_evict_first());
    if (db > 0)
      bulk_load(pbuf(s) + g.row_bytes, d + c0 * E - head(d), db, &full[s], policy_evict_first());
  };
  // brings only the draft's row of a node to buffer s
  auto load_draft = [&](int node, int s) {
    ++loads[s];
    if (tid != NT || dead) return;
    const char* d = drow(node);
    const uint32_t db = nc > 0 ? (uint32_t)((head(d) + nc * E + 15) & ~15) : 0;
    mbar_arrive_expect_tx(&full[s], db);
    if (db > 0)
      bulk_load(pbuf(s) + g.row_bytes, d + c0 * E - head(d), db, &full[s], policy_evict_first());
  };
  // the logits of child i's token in the rows of `node`, as they are stored (a
  // conversion here would wait for them, 1000 cycles and more a node)
  auto logits_at = [&](int node, int i, uint32_t& t, uint32_t& d) {
    if (i < 0 || greedy) return;
    t = ld_elem_bits<DT>(trow(node) + (int64_t)tok[i] * E);
    d = ld_elem_bits<DT>(drow(node) + (int64_t)tok[i] * E);
  };
  auto wait_rows = [&](int s) {
    if (!dead && !late) late = !mbar_wait_bounded(&full[s], (uint32_t)((loads[s] - 1) & 1), p.err);
  };
  // Puts this warp's partial into every block's slots, and waits for all of them.
  // (Three sets of slots: a block that writes meeting m + 3's has met at m + 2, for
  // which this block's working warps published after all its warps, the loading one
  // too, had come to m + 1 and so read m's.  With two sets the loading warp, which
  // publishes nothing, might still be reading.)
  int meets = 0, set = 0;
  auto meet = [&](float4 v) -> const float4* {
    const int s = meets & 1;
    const uint32_t ph = (uint32_t)((meets >> 1) & 1);
    float4* to = slots + set * nslot;
    ++meets;
    set = set == 2 ? 0 : set + 1;
    if (works && lane < K)  // lane k writes to block k
      st_async_f32x4(map_to_rank(to + rank * NW + warp, lane), map_to_rank(&met[s], lane), v.x,
                     v.y, v.z, v.w);
    if (tid == NT) mbar_arrive_expect_tx(&met[s], (uint32_t)(nslot * 16));
    __syncwarp();
    agree(dead || mbar_wait_bounded_cluster(&met[s], ph, p.err));
    return to;
  };
  auto wsum = [&](float v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  };
  // two (m, z) pairs over the warp: z sums exp((x - m) / T)
  auto add_up2 = [&](float& m, float& z, float& m2, float& z2) {
    float M = m, M2 = m2;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
      M2 = fmaxf(M2, __shfl_xor_sync(0xffffffffu, M2, off));
    }
    if (m != -INFINITY) z *= ex2((m - M) * c);
    if (m2 != -INFINITY) z2 *= ex2((m2 - M2) * c);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      z += __shfl_xor_sync(0xffffffffu, z, off);
      z2 += __shfl_xor_sync(0xffffffffu, z2, off);
    }
    m = M;
    m2 = M2;
  };
  // The shares of a slice of nc elements whose first is h bytes into its buffer: a
  // lead of single elements up to a 16-byte boundary, whole chunks, a rest.
  struct Parts {
    int lead, chunks, rest;
  };
  auto parts = [&](int h) {
    Parts q;
    q.lead = h == 0 ? 0 : min((16 - h) / E, nc);
    q.chunks = (nc - q.lead) / W;
    q.rest = nc - q.lead - q.chunks * W;
    return q;
  };
  // this thread's single element of the lead or the rest, -1 if none
  auto single = [&](const Parts& q) {
    if (tid < q.lead) return tid;
    return tid >= 32 && tid - 32 < q.rest ? q.lead + q.chunks * W + tid - 32 : -1;
  };
  // maximum, and sum about it, of this thread's share of a row
  auto stats = [&](const unsigned char* buf, int h, float& m, float& z) {
    constexpr uint32_t ni = DT == kBF16 ? 0xff80ff80u : 0xff800000u;
    const Parts q = parts(h);
    const uint4* base = reinterpret_cast<const uint4*>(buf + h + q.lead * E);
    const int j = single(q);
    const float x = j >= 0 ? ld_smem_elem<DT>(reinterpret_cast<const char*>(buf) + h + j * E)
                           : -INFINITY;
    m = x;
    z = x == -INFINITY ? 0.f : x == x ? 1.f : x;
    // four chunks at a time: their maximum, the sum so far rescaled to it, then
    // their exponentials
    for (int k = tid; k < q.chunks; k += 4 * NT) {
      uint4 v[4];
      float cm = -INFINITY;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = k + i * NT < q.chunks ? base[k + i * NT] : make_uint4(ni, ni, ni, ni);
        if constexpr (DT == kBF16) {
          const uint32_t w = bf16x2_max(bf16x2_max(v[i].x, v[i].y), bf16x2_max(v[i].z, v[i].w));
          cm = fmaxf(cm, fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)));
        } else {
          cm = fmaxf(fmaxf(cm, fmaxf(__uint_as_float(v[i].x), __uint_as_float(v[i].y))),
                     fmaxf(__uint_as_float(v[i].z), __uint_as_float(v[i].w)));
        }
      }
      if (cm > m) {
        z = m == -INFINITY ? z : z * ex2((m - cm) * c);
        m = cm;
      }
      // (a share of -inf sums to 0; about 0 a NaN still gives NaN)
      const float r = m == -INFINITY ? 0.f : m;
      float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (k + i * NT >= q.chunks) break;
#pragma unroll
        for (int e = 0; e < W; e += 4) {
          float t0, t1, t2, t3;
          scaled2(t0, t1, chunk_get<DT>(v[i], e), chunk_get<DT>(v[i], e + 1), r, c);
          scaled2(t2, t3, chunk_get<DT>(v[i], e + 2), chunk_get<DT>(v[i], e + 3), r, c);
          add2(a0, a1, a0, a1, ex2(t0), ex2(t1));
          add2(a2, a3, a2, a3, ex2(t2), ex2(t3));
        }
      }
      z += (a0 + a1) + (a2 + a3);
    }
  };
  // softmax of a row: 2^((x - m) c) * inv
  struct Soft {
    float m, inv;
  };
  auto soft = [&](float M, float Z) {
    return Soft{M == -INFINITY ? 0.f : M, Z == 0.f ? 0.f : 1.f / Z};
  };
  auto merge = [&](BestTok t) {  // over the cluster
    auto lanes = [&](BestTok r) {
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) {
        const float s = __shfl_xor_sync(0xffffffffu, r.s, off);
        const int j = __shfl_xor_sync(0xffffffffu, r.j, off);
        r.take(s, j);
      }
      return r;
    };
    t = lanes(t);
    const float4* sl = meet(make_float4(t.s, __int_as_float(t.j), 0.f, 0.f));
    BestTok r{0.f, -1};
    for (int i = lane; i < nslot; i += 32) r.take(sl[i].x, __float_as_int(sl[i].y));
    return lanes(r);
  };

  const float* noise = p.race + b * V + c0;  // this block's part
  const int nh = (int)(reinterpret_cast<uintptr_t>(noise) & 15);
  int cur = -1, done = 0, s = 0;
  int child = next_child(-1, 0);
  load_rows(-1, child, 0);
  uint32_t tx = 0, dx = 0;  // the first child's logits
  logits_at(-1, child, tx, dx);
  if (g.noise_off >= 0 && !greedy && tid == NT) {
    const uint32_t nb = nc > 0 ? (uint32_t)((nh + nc * 4 + 15) & ~15) : 0;
    mbar_arrive_expect_tx(noise_bar, nb);
    if (nb > 0)
      bulk_load(smem + g.noise_off, reinterpret_cast<const char*>(noise) - nh, nb, noise_bar,
                policy_evict_first());
  }
  int32_t token = -1;
  for (;;) {
    const int hp = head(trow(cur)), hq = head(drow(cur));
    const unsigned char* pb = pbuf(s);
    const unsigned char* qb = pb + g.row_bytes;
    // with two buffers the first child's rows are loaded while this node is worked on
    int ahead = -1, ahead_child = -1;
    uint32_t atx = 0, adx = 0;
    if (g.buffers == 2 && child >= 0) {
      ahead = child;
      ahead_child = next_child(child, child + 1);
      load_rows(ahead, ahead_child, s ^ 1);
      logits_at(ahead, ahead_child, atx, adx);
    }
    wait_rows(s);
    Soft P{}, Q{};
    BestTok top{0.f, -1};
    // a row's largest logit, over the cluster
    auto row_top = [&](const unsigned char* buf, int h) {
      // a thread keeps its greatest chunk (the first of equal ones: its chunks come
      // in ascending order) and looks for the place in it at the end
      const Parts q = parts(h);
      const char* row = reinterpret_cast<const char*>(buf) + h;
      const uint4* base = reinterpret_cast<const uint4*>(row + q.lead * E);
      float m = -INFINITY;
      int at = -1, chunk = -1;
#pragma unroll 4
      for (int k = tid; works && k < q.chunks; k += NT) {
        const uint4 v = base[k];
        float cm;
        if constexpr (DT == kBF16) {
          const uint32_t w = bf16x2_max(bf16x2_max(v.x, v.y), bf16x2_max(v.z, v.w));
          cm = fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
        } else {
          cm = fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                     fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
        }
        if (cm > m) {
          m = cm;
          chunk = k;
        }
      }
      if (chunk >= 0) {
        const uint4 v = base[chunk];
#pragma unroll
        for (int e = W - 1; e >= 0; --e)
          if (chunk_get<DT>(v, e) == m) at = q.lead + chunk * W + e;
      }
      const int j1 = works ? single(q) : -1;
      if (j1 >= 0) {
        const float v = ld_smem_elem<DT>(row + j1 * E);
        if (v > m || (v == m && at >= 0 && j1 < at)) {
          m = v;
          at = j1;
        }
      }
      return merge(BestTok{m, m > -INFINITY ? (int)(c0 + at) : -1});
    };
    if (greedy) {
      top = row_top(pb, hp);
    } else {
      float mp = -INFINITY, zp = 0.f, mq = -INFINITY, zq = 0.f;
      if (works) {
        stats(pb, hp, mp, zp);
        if (child >= 0) stats(qb, hq, mq, zq);
        add_up2(mp, zp, mq, zq);
      }
      const float4* sl = meet(make_float4(mp, zp, mq, zq));
      // lane l takes slots l, l + 32, ...; every warp the same way
      float Mp = -INFINITY, Mq = -INFINITY, Zp = 0.f, Zq = 0.f;
      for (int i = lane; i < nslot; i += 32) {
        Mp = fmaxf(Mp, sl[i].x);
        Mq = fmaxf(Mq, sl[i].z);
      }
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) {
        Mp = fmaxf(Mp, __shfl_xor_sync(0xffffffffu, Mp, off));
        Mq = fmaxf(Mq, __shfl_xor_sync(0xffffffffu, Mq, off));
      }
      for (int i = lane; i < nslot; i += 32) {
        const float4 t = sl[i];
        Zp += t.x == -INFINITY ? t.y : t.y * ex2((t.x - Mp) * c);
        Zq += t.z == -INFINITY ? t.w : t.w * ex2((t.z - Mq) * c);
      }
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) {
        Zp += __shfl_xor_sync(0xffffffffu, Zp, off);
        Zq += __shfl_xor_sync(0xffffffffu, Zq, off);
      }
      P = soft(Mp, Zp);
      Q = soft(Mq, Zq);
    }
    auto prob = [&](const Soft& r, float v) { return ex2((v - r.m) * c) * r.inv; };
    float ratio = 0.f, mass = 1.f;
    // the factor of q's exponentials (0 with no ratio, also where q is not defined)
    auto weight_q = [&]() { return ratio > 0.f ? -ratio * Q.inv : 0.f; };
    // max(p - ratio q, 0) of W columns
    auto residual = [&](const uint4& x, const uint4& y, float (&w)[W]) {
      const float rq = weight_q();
#pragma unroll
      for (int e = 0; e < W; e += 2) {
        float t0, t1, u0, u1;
        scaled2(t0, t1, chunk_get<DT>(x, e), chunk_get<DT>(x, e + 1), P.m, c);
        scaled2(u0, u1, chunk_get<DT>(y, e), chunk_get<DT>(y, e + 1), Q.m, c);
        mul2(t0, t1, ex2(t0), ex2(t1), P.inv, P.inv);
        fma2(t0, t1, ex2(u0), ex2(u1), rq, rq, t0, t1);
        w[e] = fmaxf(t0, 0.f);
        w[e + 1] = fmaxf(t1, 0.f);
      }
    };
    auto residual1 = [&](int j) {
      const float v = ld_smem_elem<DT>(reinterpret_cast<const char*>(pb) + hp + j * E);
      const float u = ratio > 0.f ? ld_smem_elem<DT>(reinterpret_cast<const char*>(qb) + hq + j * E)
                                  : -INFINITY;
      return fmaxf(fmaf(ex2((u - Q.m) * c), weight_q(), prob(P, v)), 0.f);
    };
    int next = -1;
    for (int i = child; i >= 0 && !dead;) {
      if (greedy) {
        if (tok[i] == top.j) {
          if (i != child) {
            load_draft(cur, s);
            wait_rows(s);
            if (row_top(qb, hq).j == top.j) break;  // nothing of the target is left
          }
          next = i;
          break;
        }
      } else {
        if (i != child) logits_at(cur, i, tx, dx);
        const float px = prob(P, bits_to_f32<DT>(tx)), qx = prob(Q, bits_to_f32<DT>(dx));
        if (uni[i] * mass * qx < px - ratio * qx) {
          next = i;
          break;
        }
        ratio += mass;
        // (W is asked for only by another child; whether it is 0 the draw tells)
        if (next_child(cur, i + 1) < 0) break;
        float w = 0.f;
        if (!works) {
        } else if (hp == hq) {
          const Parts q = parts(hp);
          const uint4* pv = reinterpret_cast<const uint4*>(pb + hp + q.lead * E);
          const uint4* qv = reinterpret_cast<const uint4*>(qb + hp + q.lead * E);
          float w1 = 0.f;
#pragma unroll 2
          for (int k = tid; k < q.chunks; k += NT) {
            float r[W];
            residual(pv[k], qv[k], r);
#pragma unroll
            for (int e = 0; e < W; e += 2) add2(w, w1, w, w1, r[e], r[e + 1]);
          }
          w += w1;
          const int j = single(q);
          if (j >= 0) w += residual1(j);
        } else {
#pragma unroll 4
          for (int j = tid; j < nc; j += NT) w += residual1(j);
        }
        const float4* sl = meet(make_float4(wsum(w), 0.f, 0.f, 0.f));
        mass = 0.f;
        for (int k = lane; k < nslot; k += 32) mass += sl[k].x;
        mass = wsum(mass);
        if (!(mass > 0.f)) break;  // nothing of the target is left
      }
      i = next_child(cur, i + 1);
    }
    if (next >= 0 && !dead) {
      if (tid == 0 && rank == 0) {
        p.out_tokens[b * (n + 1) + done] = tok[next];
        p.out_nodes[b * (n + 1) + done] = next;
      }
      ++done;
      cur = next;
      // every warp of the cluster has done with this node's rows (the blocks have met
      // since it read them), so the buffers may be filled again
      if (next == ahead) {
        child = ahead_child;
        tx = atx;
        dx = adx;
        s ^= 1;
      } else {
        if (ahead >= 0) wait_rows(s ^ 1);  // the rows that were loaded in vain
        child = next_child(cur, cur + 1);
        load_rows(cur, child, s);
        logits_at(cur, child, tx, dx);
      }
      continue;
    }
    if (greedy) {
      token = top.j;
    } else if (!dead) {
      if (!(mass > 0.f)) ratio = 0.f;
      const float* ns = noise;
      if (g.noise_off >= 0) {
        agree(mbar_wait_bounded(noise_bar, 0, p.err));
        ns = reinterpret_cast<const float*>(smem + g.noise_off + nh);
      }
      // (a quotient within 2 steps: the weights themselves are some steps off)
      auto score = [&](float w, float e) { return w > 0.f ? __fdividef(w, e) : -1.f; };
#pragma unroll 1
      for (;; ratio = 0.f) {  // from the residual; from p where it holds nothing
        BestTok best{0.f, -1};
        if (!works) {
        } else if (ratio == 0.f || hp == hq) {
          const Parts q = parts(hp);
          const uint4* pv = reinterpret_cast<const uint4*>(pb + hp + q.lead * E);
          const uint4* qv = reinterpret_cast<const uint4*>(qb + hq + q.lead * E);
          const bool whole = ((nh + q.lead * 4) & 15) == 0;
          const uint32_t ni = DT == kBF16 ? 0xff80ff80u : 0xff800000u;
#pragma unroll 1
          for (int k = tid; k < q.chunks; k += NT) {
            const int j = q.lead + k * W;
            float e8[W];
            if (whole) {
#pragma unroll
              for (int e = 0; e < W; e += 4) {
                const float4 t = *reinterpret_cast<const float4*>(ns + j + e);
                e8[e] = t.x, e8[e + 1] = t.y, e8[e + 2] = t.z, e8[e + 3] = t.w;
              }
            } else {
#pragma unroll
              for (int e = 0; e < W; ++e) e8[e] = ns[j + e];
            }
            float r[W];
            residual(pv[k], ratio > 0.f ? qv[k] : make_uint4(ni, ni, ni, ni), r);
#pragma unroll
            for (int e = 0; e < W; ++e) r[e] = score(r[e], e8[e]);
            best_chunk<W>(best, r, (int)c0 + j);
          }
          const int j = single(q);
          if (j >= 0) {
            const float sc = score(residual1(j), ns[j]);
            if (sc >= 0.f) best.take(sc, (int)c0 + j);
          }
        } else {
#pragma unroll 4
          for (int j = tid; j < nc; j += NT) {
            const float sc = score(residual1(j), ns[j]);
            if (best.j < 0 ? sc >= 0.f : sc > best.s) {
              best.s = sc;
              best.j = (int)c0 + j;
            }
          }
        }
        token = merge(best).j;
        if (token >= 0 || ratio == 0.f) break;
      }
    }
    if (ahead >= 0) wait_rows(s ^ 1);  // no copy outlives the block
    break;
  }
  if (dead && tid == NT) {  // nor after a wait gave up
    for (int i = 0; i < 2; ++i)
      if (loads[i] > 0) mbar_wait_bounded(&full[i], (uint32_t)((loads[i] - 1) & 1), p.err);
    if (g.noise_off >= 0 && !greedy) mbar_wait_bounded(noise_bar, 0, p.err);
  }
  if (rank == 0) {
    for (int i = done + tid; i <= n; i += blockDim.x) {
      p.out_tokens[b * (n + 1) + i] = i == done ? token : -1;
      p.out_nodes[b * (n + 1) + i] = -1;
    }
    if (tid == 0) p.out_count[b] = done;
  }
  cluster_sync();  // no peer still writes this block's slots
}

}  // namespace

VerifyKernels verify_kernels(int dtype) {
  if (dtype == kBF16)
    return {(const void*)verify_kernel_t<kBF16>, kVerT, (const void*)verify_cluster_kernel<kBF16>};
  return {(const void*)verify_kernel_t<kF32>, kVerT, (const void*)verify_cluster_kernel<kF32>};
}

}  // namespace rr
