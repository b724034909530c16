// k_logprob.cu -- log probabilities of given tokens, with the row's entropy, the token's
// rank and the row's largest alternatives, and their gradient.
//
// With z = x / T, m = max_j x_j, d = sum_j e^{z_j - m / T} and n = sum_j e^{z_j - m / T}
// (z_j - m / T), all from one pass over the row (the online normaliser, with n carried
// along: when m grows by delta, n becomes (n + delta d) e^delta):
//   log_sum = ln d,  logprob_t = (x_t - m) / T - log_sum,  entropy = log_sum - n / d.
// Every term of n is <= 0 and log_sum >= 0, so the entropy loses no digits.  m and log_sum
// are kept apart (not their sum) for the gradient: x - m is exact near the maximum, however
// large the logits are.
//   dlogits_j = [g (1_{j=t} - p_j) - h p_j (ln p_j + entropy)] / T
//             = p_j (A + B log2 p_j) + 1_{j=t} g / T  with two numbers A, B a row.
// Both are bound by memory: the forward reads the row once, the backward reads and writes it.
//
// The alternatives cost no second pass over the row: each thread's own maximum is known from
// the pass, the k-th largest of these is a lower bound of the k-th largest logit, and only
// the (about k) threads whose maximum reaches it can hold one; their elements, a 1 / 256 of
// the row each, are read again.
#include <cstdint>

#include "rr_device.cuh"
#include "rr_kernels.h"

namespace rr {
namespace {

constexpr int kT = 256;         // threads a row
constexpr int kU = 4;           // chunks a thread has in flight
constexpr int kCand = 1024;     // candidates kept for the list; more: the slow way
constexpr float kLow = -1.0e4f; // an exponent whose power of two is 0

// max(a, b), NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Maximum, sum of 2^((x - m) c), and of that times (x - m) c.
struct Stat {
  float m, d, n;
};
__device__ __forceinline__ Stat merge(const Stat& a, const Stat& b, float c) {
  const float m = fmaxf(a.m, b.m);
  const float ref = m == -INFINITY ? 0.f : m;
  const float da = fmaxf((a.m - ref) * c, kLow), db = fmaxf((b.m - ref) * c, kLow);
  const float fa = ex2(da), fb = ex2(db);
  return Stat{m, a.d * fa + b.d * fb, fa * (a.n + da * a.d) + fb * (b.n + db * b.d)};
}
__device__ __forceinline__ Stat shfl_xor(const Stat& s, int off) {
  return Stat{__shfl_xor_sync(0xffffffffu, s.m, off), __shfl_xor_sync(0xffffffffu, s.d, off),
              __shfl_xor_sync(0xffffffffu, s.n, off)};
}

__device__ __forceinline__ int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }
__device__ __forceinline__ void st_cluster_u64(uint32_t cl_addr, unsigned long long v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(cl_addr), "l"(v) : "memory");
}

// Order of the floats as an order of unsigned integers (both zeros alike).
__device__ __forceinline__ uint32_t order(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unorder(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
// The next float above a finite x or -infinity (for x >= y as x > below).
__device__ __forceinline__ float next_up(float x) { return unorder(order(x) + 1u); }

// A row's elements as memory-aligned chunks: `head` elements before the first, `tail` after
// the last of `chunks`.
template <int DT>
struct Cut {
  static constexpr int E = DType<DT>::E, W = 16 / E;
  const char* row;
  int64_t cols;
  int head, tail;
  int64_t chunks;
  __device__ __forceinline__ Cut(const char* r, int64_t n) : row(r), cols(n) {
    const int64_t h = ((16 - (int)(reinterpret_cast<uintptr_t>(r) & 15)) & 15) / E;
    head = (int)(h < n ? h : n);
    chunks = (n - head) / W;
    tail = (int)(n - head - chunks * W);
  }
  __device__ __forceinline__ const char* chunk(int64_t i) const {
    return row + (int64_t)head * E + i * 16;
  }
};

// f(x, column) for the ragged elements of thread `who`.
template <int DT, class F>
__device__ __forceinline__ void each_ragged(const Cut<DT>& cut, int who, F f) {
  constexpr int E = DType<DT>::E;
  if (who < cut.head) f(ld_elem<DT>(cut.row + who * E), (int64_t)who);
  if (who < cut.tail) {
    const int64_t j = cut.cols - cut.tail + who;
    f(ld_elem<DT>(cut.row + j * E), j);
  }
}

// One pass over chunks [0, n) from `base` (this block's slice of the row; the first element is
// column j0), thread tid taking tid, tid + kT, ...
template <int DT, bool kRank>
struct Pass {
  static constexpr int W = 16 / DType<DT>::E;
  float c, xt, above;
  int t;
  Stat st;
  int rank;
  // N chunks whose first columns are j, j + kT W, ...
  template <int N>
  __device__ __forceinline__ void take(const uint4 (&v)[N], int j) {
    float m = st.m;
    if constexpr (DT == kBF16) {
      uint32_t w = v[0].x;
#pragma unroll
      for (int u = 0; u < N; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) w = bf16x2_max(w, word_of(v[u], k));
      m = fmaxf(m, fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)));
    } else {
#pragma unroll
      for (int u = 0; u < N; ++u)
#pragma unroll
        for (int e = 0; e < W; ++e) m = fmaxf(m, chunk_get<DT>(v[u], e));
    }
    rescale(m);
    const float ref = m == -INFINITY ? 0.f : m;
    float d0 = 0.f, d1 = 0.f, n0 = 0.f, n1 = 0.f;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int j0 = j + u * kT * W;
      const float least = j0 < t ? xt : above;
#pragma unroll
      for (int e = 0; e < W; e += 2) {
        const float x0 = chunk_get<DT>(v[u], e), x1 = chunk_get<DT>(v[u], e + 1);
        float a0, a1;
        scaled2(a0, a1, x0, x1, ref, c);
        a0 = max_nan(a0, kLow);
        a1 = max_nan(a1, kLow);
        const float e0 = ex2(a0), e1 = ex2(a1);
        add2(d0, d1, d0, d1, e0, e1);
        fma2(n0, n1, a0, a1, e0, e1, n0, n1);
        if (kRank) rank += (x0 >= least) + (x1 >= least);
      }
      if (kRank && j0 < t && j0 + W > t)  // the token's own chunk: columns from t on
#pragma unroll
        for (int e = 1; e < W; ++e)
          if (j0 + e >= t) {
            const float x = chunk_get<DT>(v[u], e);
            rank += (x >= above) - (x >= xt);
          }
    }
    st.d += d0 + d1;
    st.n += n0 + n1;
  }
  __device__ __forceinline__ void take1(float x, int j) {
    const float m = fmaxf(st.m, x);
    rescale(m);
    const float a = max_nan((x - (m == -INFINITY ? 0.f : m)) * c, kLow), e = ex2(a);
    st.d += e;
    st.n += a * e;
    if (kRank) rank += x >= (j < t ? xt : above);
  }
  __device__ __forceinline__ void rescale(float m) {
    const float dm = fmaxf((st.m - (m == -INFINITY ? 0.f : m)) * c, kLow), f = ex2(dm);
    st.n = f * (st.n + dm * st.d);
    st.d *= f;
    st.m = m;
  }
};

// A row a block, or (kCl) a row a cluster whose blocks take a slice each and hand their
// statistics and their k largest to the first.
template <int DT, bool kRank, bool kCl>
__global__ void __launch_bounds__(kT, 4) logprob_fwd_kernel(const LogprobParams p) {
  constexpr int E = DType<DT>::E, W = 16 / E, NW = kT / 32;
  constexpr int kMost = 8;  // blocks of a cluster
  __shared__ Stat s_stat[NW];
  __shared__ int s_rank[NW], s_count, s_owners;
  __shared__ uint32_t s_key[kT], s_thr;
  __shared__ unsigned short s_owner[kT];
  __shared__ unsigned long long s_cand[kCand];
  __shared__ float s_part[kCl ? kMost : 1][4];
  __shared__ unsigned long long s_list[kCl ? kMost * kLogprobMaxK : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = kCl ? (int)cluster_nrank() : 1, me = kCl ? (int)cluster_rank() : 0;
  const float nan = __int_as_float(0x7fc00000);
  // (the first block's shared memory is written once all have started)
  if (kCl) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  bool waited = !kCl;
  for (int64_t r = blockIdx.x / K; r < p.rows; r += gridDim.x / K) {
    const int t = __ldg(p.tokens + r);
    if (t == p.ignore) {
      if (me == 0) {
        if (tid == 0) {
          p.logprob[r] = 0.f;
          if (p.entropy) p.entropy[r] = 0.f;
          if (p.row_max) p.row_max[r] = 0.f;
          if (p.log_sum) p.log_sum[r] = 0.f;
          if (p.rank) p.rank[r] = -1;
        }
        for (int i = tid; i < p.k; i += kT) {
          p.top_index[r * p.k + i] = -1;
          p.top_logprob[r * p.k + i] = 0.f;
        }
      }
      continue;
    }
    const Cut<DT> cut(p.x + r * p.stride * E, p.cols);
    const bool good = t >= 0 && t < p.cols;
    const float xt = good ? ld_elem_cached<DT>(cut.row + (int64_t)t * E) : 0.f;
    // this block's chunks [c0, c0 + n); the ragged elements go to the first and the last
    const int64_t per = cdiv64(cut.chunks, K), c0 = min(me * per, cut.chunks);
    const int n = (int)(min((me + 1) * per, cut.chunks) - c0);
    const char* base = cut.chunk(c0);
    const int j0 = (int)(cut.head + c0 * W);
    const int head = me == 0 ? cut.head : 0, tail = me == K - 1 ? cut.tail : 0;
    const char* tail_at = cut.row + (cut.cols - cut.tail) * E;
    // columns before t count from x_t on, those after it from the next float
    Pass<DT, kRank> pass{p.c, xt, next_up(xt), t, Stat{-INFINITY, 0.f, 0.f}, 0};
    int i = tid;
    for (; i + (kU - 1) * kT < n; i += kU * kT) {
      uint4 v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) v[u] = ld_chunk_cached(base + (int64_t)(i + u * kT) * 16);
      pass.template take<kU>(v, j0 + i * W);
    }
    for (; i < n; i += kT) {
      const uint4 v[1] = {ld_chunk_cached(base + (int64_t)i * 16)};
      pass.template take<1>(v, j0 + i * W);
    }
    if (tid < head) pass.take1(ld_elem_cached<DT>(cut.row + tid * E), tid);
    if (tid < tail) pass.take1(ld_elem_cached<DT>(tail_at + tid * E), (int)cut.cols - cut.tail + tid);
    const float c = p.c;
    Stat st = pass.st;
    const uint32_t key = order(st.m);
    s_key[tid] = key;
    if (tid == 0) s_count = s_owners = 0;
    for (int off = 16; off >= 1; off >>= 1) {
      const Stat o = shfl_xor(st, off);
      st = (lane & off) ? merge(o, st, c) : merge(st, o, c);
    }
    const int rank = kRank ? __reduce_add_sync(0xffffffffu, pass.rank) : 0;
    if (lane == 0) {
      s_stat[warp] = st;
      s_rank[warp] = rank;
    }
    __syncthreads();
    st = s_stat[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) st = merge(st, s_stat[w], c);
    int ranks = 0;
    if (kRank)
#pragma unroll
      for (int w = 0; w < NW; ++w) ranks += s_rank[w];
    // the slice's k largest: candidates in s_cand, or (long ties) one after the other
    int found = 0;
    const bool listed = p.k > 0 && st.m > -INFINITY;
    if (listed) {
      // a lower bound of the k-th largest: at least k, and not many more, of the threads'
      // maxima reach it (bisection of the bits; all of them when fewer are live)
      if (warp == 0) {
        uint32_t mine[NW];
#pragma unroll
        for (int w = 0; w < NW; ++w) mine[w] = s_key[w * 32 + lane];
        uint32_t lo = order(-INFINITY) + 1u, hi = order(st.m) + 1u;
        while (hi - lo > 1) {
          const uint32_t mid = lo + (hi - lo) / 2;
          int cnt = 0;
#pragma unroll
          for (int w = 0; w < NW; ++w) cnt += mine[w] >= mid;
          cnt = __reduce_add_sync(0xffffffffu, cnt);
          if (cnt < p.k) {
            hi = mid;
          } else {
            lo = mid;
            if (cnt <= p.k + p.k / 2) break;
          }
        }
        if (lane == 0) s_thr = lo;
      }
      __syncthreads();
      const uint32_t thr = s_thr;
      if (key >= thr) s_owner[atomicAdd(&s_owners, 1)] = (unsigned short)tid;
      auto put = [&](float x, int j) {
        const uint32_t k = order(x);
        if (k < thr) return;
        const int at = atomicAdd(&s_count, 1);
        if (at < kCand) s_cand[at] = ((unsigned long long)k << 32) | (uint32_t)~(uint32_t)j;
      };
      __syncthreads();
      // the elements of those threads again, a warp for each, four loads at a time
      const int owners = s_owners;
      for (int o = warp; o < owners; o += 4 * NW)
        for (int q = lane; q * kT < n; q += 32) {
          uint4 v[4];
          int at[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            at[u] = o + u * NW < owners ? (int)s_owner[o + u * NW] + q * kT : n;
            if (at[u] < n) v[u] = ld_chunk_cached(base + (int64_t)at[u] * 16);
          }
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (at[u] < n)
#pragma unroll
              for (int e = 0; e < W; ++e)
                put(chunk_get<DT>(v[u], e), j0 + at[u] * W + e);
        }
      if (tid < head && key >= thr) put(ld_elem_cached<DT>(cut.row + tid * E), tid);
      if (tid < tail && key >= thr)
        put(ld_elem_cached<DT>(tail_at + tid * E), (int)cut.cols - cut.tail + tid);
      __syncthreads();
      found = s_count;
      if (found > kCand) {
        // too many columns reach the bound: the largest below the last, k times
        unsigned long long last = ~0ull;
        for (int at = 0; at < p.k; ++at) {
          unsigned long long best = 0;
          auto look = [&](float x, int j) {
            const unsigned long long v =
                ((unsigned long long)order(x) << 32) | (uint32_t)~(uint32_t)j;
            if (v < last && v > best) best = v;
          };
          for (int q = tid; q < n; q += kT) {
            const uint4 v = ld_chunk_cached(base + (int64_t)q * 16);
#pragma unroll
            for (int e = 0; e < W; ++e) look(chunk_get<DT>(v, e), j0 + q * W + e);
          }
          if (tid < head) look(ld_elem_cached<DT>(cut.row + tid * E), tid);
          if (tid < tail) look(ld_elem_cached<DT>(tail_at + tid * E), (int)cut.cols - cut.tail + tid);
          for (int off = 16; off >= 1; off >>= 1)
            best = max(best, __shfl_xor_sync(0xffffffffu, best, off));
          if (lane == 0) s_cand[kLogprobMaxK + warp] = best;
          __syncthreads();
          for (int w = 0; w < NW; ++w) best = max(best, s_cand[kLogprobMaxK + w]);
          last = best;
          __syncthreads();
          if (tid == 0) s_cand[at] = best;
        }
        __syncthreads();
        found = p.k;
      }
    }
    if (kCl) {
      // to the first block: statistics, and the k largest in order (0: no column)
      if (!waited) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      waited = true;
      if (tid == 0) {
        st_cluster_f32x4(map_to_rank(s_part[me], 0), st.m, st.d, st.n, __int_as_float(ranks));
      }
      const uint32_t list = map_to_rank(s_list, 0) + me * p.k * 8;
      for (int q = found + tid; q < p.k; q += kT) st_cluster_u64(list + q * 8, 0ull);
      for (int q = tid; q < found; q += kT) {
        const unsigned long long v = s_cand[q];
        int at = 0;
        for (int w = 0; w < found; ++w) at += s_cand[w] > v;
        if (at < p.k) st_cluster_u64(list + at * 8, v);
      }
      cluster_sync();
      if (me != 0) continue;  // (a cluster takes one row)
      st = Stat{s_part[0][0], s_part[0][1], s_part[0][2]};
      ranks = __float_as_int(s_part[0][3]);
      for (int w = 1; w < K; ++w) {
        st = merge(st, Stat{s_part[w][0], s_part[w][1], s_part[w][2]}, c);
        ranks += __float_as_int(s_part[w][3]);
      }
      found = K * p.k;
    }
    const bool bad = !(st.d >= 0.f && st.m < INFINITY);  // a NaN or an infinity
    const bool none = st.m == -INFINITY && !bad;         // nothing but -infinity
    const float log_sum = bad ? nan : none ? 0.f : logf(st.d);
    if (tid == 0) {
      if (!good && p.bad) atomicAdd(p.bad, 1);
      p.logprob[r] = bad || !good ? nan : none ? 0.f : (xt - st.m) / p.temperature - log_sum;
      if (p.entropy) p.entropy[r] = bad ? nan : none ? 0.f : log_sum - st.n / st.d * kLn2;
      if (p.row_max) p.row_max[r] = bad ? nan : st.m;
      if (p.log_sum) p.log_sum[r] = log_sum;
      if (kRank) p.rank[r] = bad || !good ? -1 : ranks;
    }
    if (p.k > 0) {
      if (bad || none) {
        for (int q = tid; q < p.k; q += kT) {
          p.top_index[r * p.k + q] = -1;
          p.top_logprob[r * p.k + q] = bad ? nan : -INFINITY;
        }
      } else {
        // each candidate's place is the number of greater ones
        const unsigned long long* cand = kCl ? s_list : s_cand;
        int live = found;
        if (kCl) {
          live = 0;
          for (int q = 0; q < found; ++q) live += cand[q] != 0;
        }
        for (int q = tid; q < found; q += kT) {
          const unsigned long long v = cand[q];
          if (kCl && v == 0) continue;
          int at = 0;
          for (int w = 0; w < found; ++w) at += cand[w] > v;
          if (at < p.k) {
            p.top_index[r * p.k + at] = (int32_t)~(uint32_t)v;
            p.top_logprob[r * p.k + at] =
                (unorder((uint32_t)(v >> 32)) - st.m) / p.temperature - log_sum;
          }
        }
        for (int q = live + tid; q < p.k; q += kT) {
          p.top_index[r * p.k + q] = -1;
          p.top_logprob[r * p.k + q] = -INFINITY;
        }
      }
    }
    __syncthreads();
  }
  if (!waited) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A block takes kT * kU chunks of a row (kV: chunks of both tensors are aligned alike) or as
// many elements.
template <int DT, bool kV>
__global__ void __launch_bounds__(kT) logprob_bwd_kernel(const LogprobBwdParams p) {
  constexpr int E = DType<DT>::E, W = 16 / E;
  const int64_t r = blockIdx.x / p.segs;
  const int seg = (int)(blockIdx.x - r * p.segs);
  const int tid = threadIdx.x;
  const int t = __ldg(p.tokens + r);
  const Cut<DT> cut(p.x + r * p.x_stride * E, p.cols);
  char* out = p.y + r * p.y_stride * E;
  const float m = __ldg(p.row_max + r);
  const bool zero = t == p.ignore || m == -INFINITY;
  const float g = p.g ? __ldg(p.g + r) : 0.f, h = p.h ? __ldg(p.h + r) : 0.f;
  const float ent = p.h ? __ldg(p.entropy + r) : 0.f;
  const float inv = 1.f / p.temperature, c = p.c;
  const float A = -(g + h * ent) * inv, B = -h * kLn2 * inv, G = g * inv;
  const float ls = __ldg(p.log_sum + r) * kLog2e;
  auto grad = [&](float x, int64_t j) {
    if (zero) return 0.f;
    const float a = max_nan((x - m) * c - ls, kLow);
    const float v = ex2(a) * (A + B * a);
    return j == t ? v + G : v;
  };
  if constexpr (kV) {
    for (int u = 0; u < kU; ++u) {
      const int64_t i = ((int64_t)seg * kU + u) * kT + tid;
      if (i >= cut.chunks) break;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (!zero) v = ld_chunk_stream(cut.chunk(i));
      float f[W];
#pragma unroll
      for (int e = 0; e < W; ++e) f[e] = grad(chunk_get<DT>(v, e), cut.head + i * W + e);
      st_chunk_stream(out + (int64_t)cut.head * E + i * 16, chunk_pack<DT>(f));
    }
    if (seg == 0)
      each_ragged<DT>(cut, tid, [&](float x, int64_t j) { st_elem<DT>(out + j * E, grad(x, j)); });
  } else {
    for (int u = 0; u < kU * W; ++u) {
      const int64_t j = ((int64_t)seg * kU * W + u) * kT + tid;
      if (j >= p.cols) break;
      st_elem<DT>(out + j * E, grad(zero ? 0.f : ld_elem<DT>(cut.row + j * E), j));
    }
  }
}

}  // namespace

template <int DT>
static LogprobKernels kernels_of() {
  return LogprobKernels{
      {{(const void*)logprob_fwd_kernel<DT, false, false>, (const void*)logprob_fwd_kernel<DT, false, true>},
       {(const void*)logprob_fwd_kernel<DT, true, false>, (const void*)logprob_fwd_kernel<DT, true, true>}},
      {(const void*)logprob_bwd_kernel<DT, false>, (const void*)logprob_bwd_kernel<DT, true>},
      kT,
      kT * kU * 16};
}
LogprobKernels logprob_kernels(int dtype) {
  return dtype == kF32 ? kernels_of<kF32>() : kernels_of<kBF16>();
}

}  // namespace rr
