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
// Only the rows of visited nodes are read: the walk depends on the tokens
// accepted so far.
//
// A cluster of K blocks walks a sequence, each with a slice of the columns: the
// slices of a node's two rows come to shared memory by bulk copies and stay there
// for every pass over them (maximum, sum, the residual's mass after each rejection,
// the final draw), so a row is read from memory once.  After each pass every warp
// puts its partial into a slot of every block of the cluster and arrives on its
// mbarrier; every warp then merges all slots in the same order, so all threads of
// the cluster hold the same numbers and take the same decisions.  With few
// sequences a walk is bound by latency (a row's 1.5-2 us, then about 0.6 us a
// meeting), so the first child's rows are loaded while its parent's are worked
// on; with many it is bound by memory, several clusters share an SM, and nothing
// is loaded that the walk does not reach.  Rows that a cluster cannot hold go to
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
    BestTok top{0.f, -1};
    if (greedy) {
      for (int64_t j = tid; j < V; j += kVerT) {
        const float v = ld_elem<DT>(tr + j * E);
        if (v > -INFINITY) top.take(v, (int)j);
      }
      top = ver_best(top, red);
    } else {
      pr = ver_row<DT>(tr, V, c, red);
    }
    float ratio = 0.f, mass = 1.f;
    bool have_q = false;
    int next = -1;
    for (int i = cur + 1; i < n && next < 0; ++i) {
      const int32_t x = tok[i];
      if ((par != nullptr ? par[i] : i - 1) != cur || x < 0 || x >= V) continue;
      if (greedy) {
        if (x == top.j) next = i;
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

template <int DT>
__global__ void __launch_bounds__(kVerClT, 3) verify_cluster_kernel(const VerifyParams p,
                                                                const VerifyGeo g) {
  constexpr int E = DType<DT>::E, W = DType<DT>::V, NW = kVerClT / 32;
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = (int)cluster_nrank(), rank = (int)cluster_rank();
  const int64_t b = blockIdx.x / K, V = p.cols;
  const int n = p.nodes;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);       // [2] a node's rows have landed
  uint64_t* met = full + 2;                                 // [2] partials published
  uint64_t* noise_bar = full + 4;
  float4* slots = reinterpret_cast<float4*>(smem + 64);     // [2][K * NW]
  const int nslot = K * NW;
  const int32_t* tok = p.tokens + b * n;
  const int32_t* par = p.parents != nullptr ? p.parents + b * n : nullptr;
  const float T = p.temperature != nullptr ? __ldg(p.temperature + b) : 1.f;
  const bool greedy = T <= 0.f;
  const float c = kLog2e / T;
  const int64_t c0 = (int64_t)rank * g.C;                   // this block's columns
  const int nc = (int)max((int64_t)0, min((int64_t)g.C, V - c0));

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&met[i], nslot);
    }
    mbar_init(noise_bar, 1);
    fence_mbar_init();
  }
  cluster_sync();  // peers arrive on this block's barriers

  bool dead = false;  // a wait gave up: later waits are skipped (the kernel still ends)
  auto trow = [&](int node) { return p.target + ((b * (n + 1) + node + 1) * V) * E; };
  auto drow = [&](int node) { return p.draft + ((b * n + node + 1) * V) * E; };
  // A slice of a row in shared memory: its first element is h bytes into the buffer.
  auto head = [&](const char* row) {
    return (int)((reinterpret_cast<uintptr_t>(row) + (uint64_t)c0 * E) & 15);
  };
  auto pbuf = [&](int s) { return smem + g.buf_off + s * 2 * g.row_bytes; };
  // the next child of `cur` from node i on, -1 if none (every warp by itself)
  auto next_child = [&](int cur, int i) {
    if (par == nullptr) {
      if (i > cur + 1 || cur + 1 >= n) return -1;
      const int32_t x = __ldg(tok + cur + 1);
      return x >= 0 && x < V ? cur + 1 : -1;
    }
    for (int base = i & ~31; base < n; base += 32) {
      const int j = base + lane;
      bool hit = false;
      if (j >= i && j < n && __ldg(par + j) == cur) {
        const int32_t x = __ldg(tok + j);
        hit = x >= 0 && x < V;
      }
      const uint32_t m = __ballot_sync(0xffffffffu, hit);
      if (m != 0) return base + __ffs(m) - 1;
    }
    return -1;
  };
  int loads[2] = {0, 0};  // of each buffer (the same count in every thread)
  auto load_rows = [&](int node, bool with_draft, int s) {
    ++loads[s];
    if (tid != 0 || dead) return;
    const char* t = trow(node);
    const char* d = drow(node);
    const uint32_t tb = nc > 0 ? (uint32_t)((head(t) + nc * E + 15) & ~15) : 0;
    const uint32_t db = with_draft && nc > 0 ? (uint32_t)((head(d) + nc * E + 15) & ~15) : 0;
    mbar_arrive_expect_tx(&full[s], tb + db);
    if (tb > 0)
      bulk_load(pbuf(s), t + c0 * E - head(t), tb, &full[s], policy_evict_first());
    if (db > 0)
      bulk_load(pbuf(s) + g.row_bytes, d + c0 * E - head(d), db, &full[s], policy_evict_first());
  };
  auto wait_rows = [&](int s) {
    if (!dead) dead = !mbar_wait_bounded(&full[s], (uint32_t)((loads[s] - 1) & 1), p.err);
  };
  // Puts this warp's partial into every block's slots, and waits for all of them.
  int meets = 0;
  auto meet = [&](float4 v) -> const float4* {
    const int s = meets & 1;
    const uint32_t ph = (uint32_t)((meets >> 1) & 1);
    ++meets;
    float4* sl = slots + s * nslot + rank * NW + warp;
    if (lane < K) {  // lane k writes to block k
      st_cluster_f32x4(map_to_rank(sl, lane), v.x, v.y, v.z, v.w);
      mbar_arrive_cluster(map_to_rank(&met[s], lane));
    }
    __syncwarp();
    if (!dead) dead = !mbar_wait_bounded_cluster(&met[s], ph, p.err);
    return slots + s * nslot;
  };
  auto wmax = [&](float v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
  };
  auto wsum = [&](float v) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
  };
  // f(j, x) for this thread's share of a slice's elements, whole 16-byte chunks
  // where it can
  auto each = [&](const unsigned char* buf, int h, auto&& f) {
    const int lead = h == 0 ? 0 : min((16 - h) / E, nc);
    const int chunks = (nc - lead) / W, rest = nc - lead - chunks * W;
    const unsigned char* base = buf + h;
    if (tid < lead) f(tid, ld_smem_elem<DT>(reinterpret_cast<const char*>(base) + tid * E));
    for (int q = tid; q < chunks; q += kVerClT) {
      const uint4 x = *reinterpret_cast<const uint4*>(base + (lead + q * W) * E);
#pragma unroll
      for (int e = 0; e < W; ++e) f(lead + q * W + e, chunk_get<DT>(x, e));
    }
    if (tid < rest) {
      const int j = lead + chunks * W + tid;
      f(j, ld_smem_elem<DT>(reinterpret_cast<const char*>(base) + j * E));
    }
  };
  // f(j, x, y) over two slices
  auto each2 = [&](const unsigned char* pb, int hp, const unsigned char* qb, int hq, auto&& f) {
    if (hp == hq) {
      const int lead = hp == 0 ? 0 : min((16 - hp) / E, nc);
      const int chunks = (nc - lead) / W, rest = nc - lead - chunks * W;
      if (tid < lead || (tid >= 32 && tid - 32 < rest)) {
        const int j = tid < lead ? tid : lead + chunks * W + tid - 32;
        f(j, ld_smem_elem<DT>(reinterpret_cast<const char*>(pb) + hp + j * E),
          ld_smem_elem<DT>(reinterpret_cast<const char*>(qb) + hq + j * E));
      }
      for (int q = tid; q < chunks; q += kVerClT) {
        const int j = lead + q * W;
        const uint4 x = *reinterpret_cast<const uint4*>(pb + hp + j * E);
        const uint4 y = *reinterpret_cast<const uint4*>(qb + hq + j * E);
#pragma unroll
        for (int e = 0; e < W; ++e) f(j + e, chunk_get<DT>(x, e), chunk_get<DT>(y, e));
      }
    } else {
      for (int j = tid; j < nc; j += kVerClT)
        f(j, ld_smem_elem<DT>(reinterpret_cast<const char*>(pb) + hp + j * E),
          ld_smem_elem<DT>(reinterpret_cast<const char*>(qb) + hq + j * E));
    }
  };
  auto best_of = [&](BestTok t) {  // over the cluster
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      const float s = __shfl_xor_sync(0xffffffffu, t.s, off);
      const int j = __shfl_xor_sync(0xffffffffu, t.j, off);
      t.take(s, j);
    }
    const float4* sl = meet(make_float4(t.s, __int_as_float(t.j), 0.f, 0.f));
    BestTok r{0.f, -1};
    for (int i = lane; i < nslot; i += 32) r.take(sl[i].x, __float_as_int(sl[i].y));
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) {
      const float s = __shfl_xor_sync(0xffffffffu, r.s, off);
      const int j = __shfl_xor_sync(0xffffffffu, r.j, off);
      r.take(s, j);
    }
    return r;
  };

  const float* noise = p.race + b * V + c0;  // this block's part
  const int nh = (int)(reinterpret_cast<uintptr_t>(noise) & 15);
  int cur = -1, done = 0, s = 0;
  int child = next_child(-1, 0);
  load_rows(-1, child >= 0 && !greedy, 0);
  if (g.noise_off >= 0 && !greedy && tid == 0) {
    const uint32_t nb = nc > 0 ? (uint32_t)((nh + nc * 4 + 15) & ~15) : 0;
    mbar_arrive_expect_tx(noise_bar, nb);
    if (nb > 0)
      bulk_load(smem + g.noise_off, reinterpret_cast<const char*>(noise) - nh, nb, noise_bar,
                policy_evict_first());
  }
  int32_t token = -1;
  for (;;) {
    const char* tr = trow(cur);
    const char* dr = drow(cur);
    const int hp = head(tr), hq = head(dr);
    const unsigned char* pb = pbuf(s);
    const unsigned char* qb = pb + g.row_bytes;
    // the first child's logits here, and (with two buffers) its rows
    float tx = 0.f, dx = 0.f;
    int ahead = -1, ahead_child = -1;
    if (child >= 0 && !greedy) {
      const int32_t x = __ldg(tok + child);
      tx = ld_elem<DT>(tr + (int64_t)x * E);
      dx = ld_elem<DT>(dr + (int64_t)x * E);
    }
    if (g.buffers == 2 && child >= 0) {
      ahead = child;
      ahead_child = next_child(child, child + 1);
      load_rows(ahead, ahead_child >= 0 && !greedy, s ^ 1);
    }
    wait_rows(s);
    VerRow pr{}, qr{};
    BestTok top{0.f, -1};
    if (greedy) {
      each(pb, hp, [&](int j, float v) {
        if (v > -INFINITY) top.take(v, (int)(c0 + j));
      });
      top = best_of(top);
    } else {
      // maxima, then sums about the thread's maximum; merged with the cluster's
      float mp = -INFINITY, mq = -INFINITY, zp = 0.f, zq = 0.f;
      each(pb, hp, [&](int, float v) { mp = fmaxf(mp, v); });
      if (child >= 0) each(qb, hq, [&](int, float v) { mq = fmaxf(mq, v); });
      mp = wmax(mp);
      mq = wmax(mq);
      // (a row of -inf here gives 0; about 0 a NaN still gives NaN)
      const float rp = mp == -INFINITY ? 0.f : mp, rq = mq == -INFINITY ? 0.f : mq;
      each(pb, hp, [&](int, float v) { zp += ex2((v - rp) * c); });
      if (child >= 0) each(qb, hq, [&](int, float v) { zq += ex2((v - rq) * c); });
      const float4* sl = meet(make_float4(mp, wsum(zp), mq, wsum(zq)));
      float Mp = -INFINITY, Mq = -INFINITY;
      for (int i = lane; i < nslot; i += 32) {
        Mp = fmaxf(Mp, sl[i].x);
        Mq = fmaxf(Mq, sl[i].z);
      }
      Mp = wmax(Mp);
      Mq = wmax(Mq);
      float Zp = 0.f, Zq = 0.f;
      for (int i = lane; i < nslot; i += 32) {
        const float4 t = sl[i];
        Zp += t.x == -INFINITY ? t.y : t.y * ex2((t.x - Mp) * c);
        Zq += t.z == -INFINITY ? t.w : t.w * ex2((t.z - Mq) * c);
      }
      Zp = wsum(Zp);
      Zq = wsum(Zq);
      pr = {nullptr, Mp, Zp == 0.f ? 0.f : 1.f / Zp};
      qr = {nullptr, Mq, Zq == 0.f ? 0.f : 1.f / Zq};
    }
    auto prob = [&](const VerRow& r, float v) {
      return v == -INFINITY ? 0.f : ex2((v - r.m) * c) * r.inv;
    };
    float ratio = 0.f, mass = 1.f;
    int next = -1;
    for (int i = child; i >= 0 && !dead;) {
      const int32_t x = __ldg(tok + i);
      if (greedy) {
        if (x == top.j) {
          next = i;
          break;
        }
      } else {
        if (i != child) {
          tx = ld_elem<DT>(tr + (int64_t)x * E);
          dx = ld_elem<DT>(dr + (int64_t)x * E);
        }
        const float px = prob(pr, tx), qx = prob(qr, dx);
        if (__ldg(p.uniform + b * n + i) * mass * qx < px - ratio * qx) {
          next = i;
          break;
        }
        ratio += mass;
        float w = 0.f;
        each2(pb, hp, qb, hq, [&](int, float v, float u) {
          const float t = prob(pr, v) - ratio * prob(qr, u);
          w += t < 0.f ? 0.f : t;
        });
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
        p.out_tokens[b * (n + 1) + done] = __ldg(tok + next);
        p.out_nodes[b * (n + 1) + done] = next;
      }
      ++done;
      cur = next;
      // every warp of the cluster has done with this node's rows (it has met the
      // others since it read them), so the buffers may be filled again
      if (next == ahead) {
        child = ahead_child;
        s ^= 1;
      } else {
        if (ahead >= 0) wait_rows(s ^ 1);  // the rows that were loaded in vain
        child = next_child(cur, cur + 1);
        load_rows(cur, child >= 0 && !greedy, s);
      }
      continue;
    }
    if (greedy) {
      token = top.j;
    } else if (!dead) {
      if (!(mass > 0.f)) ratio = 0.f;
      const float* ns = noise;
      if (g.noise_off >= 0) {
        dead = !mbar_wait_bounded(noise_bar, 0, p.err);
        ns = reinterpret_cast<const float*>(smem + g.noise_off + nh);
      }
      BestTok best{0.f, -1};
      auto bid = [&](int j, float w) {
        if (w > 0.f) {
          const float sc = w / ns[j];
          if (sc >= 0.f) best.take(sc, (int)(c0 + j));
        }
      };
      if (ratio > 0.f)
        each2(pb, hp, qb, hq,
              [&](int j, float v, float u) { bid(j, prob(pr, v) - ratio * prob(qr, u)); });
      else
        each(pb, hp, [&](int j, float v) { bid(j, prob(pr, v)); });
      token = best_of(best).j;
    }
    if (ahead >= 0) wait_rows(s ^ 1);  // no copy outlives the block
    break;
  }
  if (rank == 0) {
    for (int i = done + tid; i <= n; i += kVerClT) {
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
    return {(const void*)verify_kernel_t<kBF16>, kVerT, (const void*)verify_cluster_kernel<kBF16>,
            kVerClT};
  return {(const void*)verify_kernel_t<kF32>, kVerT, (const void*)verify_cluster_kernel<kF32>,
          kVerClT};
}

}  // namespace rr
