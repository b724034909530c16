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

// f(x, column) for each element that thread `who` of kT owns: whole chunks who, who + kT,
// ..., and one of the ragged ones.
template <int DT, class F>
__device__ __forceinline__ void each_ragged(const Cut<DT>& cut, int who, F f) {
  constexpr int E = DType<DT>::E;
  if (who < cut.head) f(ld_elem<DT>(cut.row + who * E), (int64_t)who);
  if (who < cut.tail) {
    const int64_t j = cut.cols - cut.tail + who;
    f(ld_elem<DT>(cut.row + j * E), j);
  }
}

template <int DT>
__global__ void __launch_bounds__(kT) logprob_fwd_kernel(const LogprobParams p) {
  constexpr int E = DType<DT>::E, W = 16 / E, NW = kT / 32;
  __shared__ Stat s_stat[NW];
  __shared__ int s_rank[NW], s_count;
  __shared__ uint32_t s_key[kT], s_thr;
  __shared__ unsigned long long s_cand[kCand];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const int t = __ldg(p.tokens + r);
    if (t == p.ignore) {
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
      continue;
    }
    const Cut<DT> cut(p.x + r * p.stride * E, p.cols);
    const bool good = t >= 0 && t < p.cols;
    const float xt = good ? ld_elem<DT>(cut.row + (int64_t)t * E) : 0.f;
    // columns before t count from x_t on, those after it from the next float
    const float above = next_up(xt);
    Stat st{-INFINITY, 0.f, 0.f};
    int rank = 0;
    const float c = p.c;
    auto take = [&](const float* x, int n, int64_t j) {
      float m = st.m;
      for (int i = 0; i < n; ++i) m = fmaxf(m, x[i]);
      const float ref = m == -INFINITY ? 0.f : m;
      const float dm = fmaxf((st.m - ref) * c, kLow), f = ex2(dm);
      st.n = f * (st.n + dm * st.d);
      st.d *= f;
      st.m = m;
      for (int i = 0; i < n; ++i) {
        const float a = max_nan((x[i] - ref) * c, kLow), e = ex2(a);
        st.d += e;
        st.n += a * e;
        rank += x[i] >= (j + i < t ? xt : above);
      }
    };
    for (int64_t i = tid; i < cut.chunks; i += kT) {
      const uint4 v = ld_chunk_stream(cut.chunk(i));
      float x[W];
#pragma unroll
      for (int e = 0; e < W; ++e) x[e] = chunk_get<DT>(v, e);
      take(x, W, cut.head + i * W);
    }
    each_ragged<DT>(cut, tid, [&](float x, int64_t j) { take(&x, 1, j); });
    const uint32_t key = order(st.m);
    s_key[tid] = key;
    if (tid == 0) s_count = 0;
    for (int off = 16; off >= 1; off >>= 1) {
      const Stat o = shfl_xor(st, off);
      st = (lane & off) ? merge(o, st, c) : merge(st, o, c);
    }
    rank = __reduce_add_sync(0xffffffffu, rank);
    if (lane == 0) {
      s_stat[warp] = st;
      s_rank[warp] = rank;
    }
    __syncthreads();
    st = s_stat[0];
    for (int i = 1; i < NW; ++i) st = merge(st, s_stat[i], c);
    const bool bad = !(st.d >= 0.f && st.m < INFINITY);  // a NaN or an infinity
    const bool none = st.m == -INFINITY && !bad;         // nothing but -infinity
    const float log_sum = bad ? __int_as_float(0x7fc00000) : none ? 0.f : logf(st.d);
    if (tid == 0) {
      if (!good && p.bad) atomicAdd(p.bad, 1);
      const float nan = __int_as_float(0x7fc00000);
      p.logprob[r] = bad || !good ? nan : none ? 0.f : (xt - st.m) / p.temperature - log_sum;
      if (p.entropy) p.entropy[r] = bad ? nan : none ? 0.f : log_sum - st.n / st.d * kLn2;
      if (p.row_max) p.row_max[r] = bad ? nan : st.m;
      if (p.log_sum) p.log_sum[r] = log_sum;
      if (p.rank) {
        int k = 0;
        for (int i = 0; i < NW; ++i) k += s_rank[i];
        p.rank[r] = bad || !good ? -1 : k;
      }
    }
    if (p.k > 0) {
      if (bad || none) {
        for (int i = tid; i < p.k; i += kT) {
          p.top_index[r * p.k + i] = -1;
          p.top_logprob[r * p.k + i] = bad ? __int_as_float(0x7fc00000) : -INFINITY;
        }
      } else {
        // the k-th largest of the threads' maxima, by bisection of its bits
        if (warp == 0) {
          uint32_t mine[NW], lo = 0;
          for (int i = 0; i < NW; ++i) mine[i] = s_key[i * 32 + lane];
          for (int b = 31; b >= 0; --b) {
            const uint32_t at = lo | (1u << b);
            int n = 0;
            for (int i = 0; i < NW; ++i) n += mine[i] >= at;
            if ((int)__reduce_add_sync(0xffffffffu, n) >= p.k) lo = at;
          }
          if (lane == 0) s_thr = max(lo, order(-INFINITY) + 1u);
        }
        __syncthreads();
        const uint32_t thr = s_thr;
        auto put = [&](float x, int64_t j) {
          const uint32_t k = order(x);
          if (k < thr) return;
          const int at = atomicAdd(&s_count, 1);
          if (at < kCand) s_cand[at] = ((unsigned long long)k << 32) | (uint32_t)~(uint32_t)j;
        };
        // a warp reads the elements of one of its threads at a time
        for (int w = 0; w < 32; ++w) {
          if (__shfl_sync(0xffffffffu, key, w) < thr) continue;
          const int who = warp * 32 + w;
          for (int64_t i = who + (int64_t)lane * kT; i < cut.chunks; i += 32 * kT) {
            const uint4 v = ld_chunk_stream(cut.chunk(i));
#pragma unroll
            for (int e = 0; e < W; ++e) put(chunk_get<DT>(v, e), cut.head + i * W + e);
          }
          if (lane == 0) each_ragged<DT>(cut, who, put);
        }
        __syncthreads();
        const int n = s_count;
        auto write = [&](int at, unsigned long long v) {
          p.top_index[r * p.k + at] = (int32_t)~(uint32_t)v;
          p.top_logprob[r * p.k + at] =
              (unorder((uint32_t)(v >> 32)) - st.m) / p.temperature - log_sum;
        };
        if (n <= kCand) {
          for (int i = tid; i < n; i += kT) {
            const unsigned long long v = s_cand[i];
            int at = 0;
            for (int j = 0; j < n; ++j) at += s_cand[j] > v;
            if (at < p.k) write(at, v);
          }
          for (int i = n + tid; i < p.k; i += kT) {
            p.top_index[r * p.k + i] = -1;
            p.top_logprob[r * p.k + i] = -INFINITY;
          }
        } else {
          // too many columns reach the bound (long ties): the largest below the last, k times
          unsigned long long last = ~0ull;
          for (int at = 0; at < p.k; ++at) {
            unsigned long long best = 0;
            auto look = [&](float x, int64_t j) {
              const unsigned long long v =
                  ((unsigned long long)order(x) << 32) | (uint32_t)~(uint32_t)j;
              if (v < last && v > best) best = v;
            };
            for (int64_t i = tid; i < cut.chunks; i += kT) {
              const uint4 v = ld_chunk_stream(cut.chunk(i));
#pragma unroll
              for (int e = 0; e < W; ++e) look(chunk_get<DT>(v, e), cut.head + i * W + e);
            }
            each_ragged<DT>(cut, tid, look);
            for (int off = 16; off >= 1; off >>= 1)
              best = max(best, __shfl_xor_sync(0xffffffffu, best, off));
            __syncthreads();
            if (lane == 0) s_cand[warp] = best;
            __syncthreads();
            for (int i = 0; i < NW; ++i) best = max(best, s_cand[i]);
            last = best;
            if (tid == 0) write(at, best);  // (more than kCand live columns: never short)
          }
        }
      }
    }
    __syncthreads();
  }
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

LogprobKernels logprob_kernels(int dtype) {
  LogprobKernels k{};
  k.threads = kT;
  k.bwd_bytes = kT * kU * 16;
  if (dtype == kF32) {
    k.fwd = (const void*)logprob_fwd_kernel<kF32>;
    k.bwd[0] = (const void*)logprob_bwd_kernel<kF32, false>;
    k.bwd[1] = (const void*)logprob_bwd_kernel<kF32, true>;
  } else {
    k.fwd = (const void*)logprob_fwd_kernel<kBF16>;
    k.bwd[0] = (const void*)logprob_bwd_kernel<kBF16, false>;
    k.bwd[1] = (const void*)logprob_bwd_kernel<kBF16, true>;
  }
  return k;
}

}  // namespace rr
