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
#include <cstdint>

#include "rr_device.cuh"
#include "rr_kernels.h"

namespace rr {
namespace {

constexpr int kVerT = 512;

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

}  // namespace

VerifyKernel verify_kernel(int dtype) {
  return {dtype == kBF16 ? (const void*)verify_kernel_t<kBF16> : (const void*)verify_kernel_t<kF32>,
          kVerT};
}

}  // namespace rr
