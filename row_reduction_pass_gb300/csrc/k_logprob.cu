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
//             = [p_j (A + B log2 p_j) + 1_{j=t} g] / T  with two numbers A, B a row.
// Both are bound by memory: the forward reads the row once, the backward reads and writes it.
//
// The alternatives cost no second pass over the row: each thread's own maximum is known from
// the pass, a value that at least k of these reach is a lower bound of the k-th largest logit, and
// only the (about k) threads whose maximum reaches it can hold one.  What they may hold is read
// again: with few rows (a cluster a row) all of a thread's part, a 1 / 256 of its block's slice;
// with many (128 streaming threads a row) those of the up to 16 pieces of its part whose maximum
// reaches the bound.  Where long ties leave too many candidates, the row is read k times.
#include <cstdint>

#include <cuda_bf16.h>

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

// Maximum, sum of 2^((x - m) c), and of that times (x - m) c.  Before any live column (d 0)
// the maximum is the least finite number, so that no difference of two is a NaN.
constexpr float kNone = -3.402823466e38f;
struct Stat {
  float m, d, n;
};
__device__ __forceinline__ Stat merge(const Stat& a, const Stat& b, float c) {
  const float m = fmaxf(a.m, b.m);
  const float da = fmaxf((a.m - m) * c, kLow), db = fmaxf((b.m - m) * c, kLow);
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

__device__ __forceinline__ uint32_t bf16x2_max_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t word_at(const uint4& c, int k) {  // (k not a constant)
  const uint32_t lo = (k & 1) ? c.y : c.x, hi = (k & 1) ? c.w : c.z;
  return (k & 2) ? hi : lo;
}
__device__ __forceinline__ __nv_bfloat162 bf162_of(uint32_t w) {
  return *reinterpret_cast<const __nv_bfloat162*>(&w);
}

// Order of the floats as an order of unsigned integers (both zeros alike).
__device__ __forceinline__ uint32_t order(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unorder(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
// The next value of the type above a finite x or -infinity (y >= it is y > x).
template <int DT>
__device__ __forceinline__ float next_up(float x) {
  return unorder(order(x) + (DT == kBF16 ? 0x10000u : 1u));
}

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


// A thread's statistics of its part of a row, chunks kS apart.  The reference of its sums is
// its maximum so far, so the greatest term is exactly 1 and a row of one likely column keeps
// the digits of its small log_sum.
template <int DT, bool kRank, int kS>
struct Pass {
  static constexpr int W = 16 / DType<DT>::E;
  float c, xt, above;
  int t;
  Stat st;
  int rank;
  bool common;  // c is not extreme
  __device__ __forceinline__ Pass(float c_, float xt_, int t_)
      : c(c_), xt(xt_), above(next_up<DT>(xt_)), t(t_), st{kNone, 0.f, 0.f}, rank(0),
        common(c_ > 0x1p-50f && c_ < 0x1p60f) {}
  // N chunks whose first columns are j, j + kS W, ...; returns their maximum.
  template <int N>
  __device__ __forceinline__ float take(const uint4 (&v)[N], int j) {
    float m;
    if constexpr (DT == kBF16) {
      uint32_t w = v[0].x;
#pragma unroll
      for (int u = 0; u < N; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) w = bf16x2_max(w, word_of(v[u], k));
      m = fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
      m = chunk_get<DT>(v[0], 0);
#pragma unroll
      for (int u = 0; u < N; ++u)
#pragma unroll
        for (int e = 0; e < W; ++e) m = fmaxf(m, chunk_get<DT>(v[u], e));
    }
    if (kRank) {
      // chunks before the token's count from x_t on, from its own on from the next value
      // (ties_before adds those in its own)
      if constexpr (DT == kBF16) {
        // A word's comparisons as two masks of 16 bits, summed as 32-bit numbers: a hits in the
        // low halves and b in the high ones give 2^16 (a - b) - a (mod 2^32).
        const uint32_t b0 = __float_as_uint(xt) >> 16, b1 = __float_as_uint(above) >> 16;
        uint32_t s0 = 0, s1 = 0;
        // one bound where all lanes' chunks are on one side of the token's (nearly always)
        const int first = kS == 32 ? j - (int)(threadIdx.x & 31) * W : j;
        const int last = kS == 32 ? first + 32 * N * W : j + (N - 1) * kS * W + W;
        if (last <= t || first + W > t) {
          const __nv_bfloat162 x2 = bf162_of((last <= t ? b0 : b1) * 0x10001u);
#pragma unroll
          for (int u = 0; u < N; ++u) {
            s0 += __hge2_mask(bf162_of(v[u].x), x2) + __hge2_mask(bf162_of(v[u].y), x2);
            s1 += __hge2_mask(bf162_of(v[u].z), x2) + __hge2_mask(bf162_of(v[u].w), x2);
          }
        } else {
#pragma unroll
          for (int u = 0; u < N; ++u) {
            const __nv_bfloat162 x2 = bf162_of((j + u * kS * W + W <= t ? b0 : b1) * 0x10001u);
            s0 += __hge2_mask(bf162_of(v[u].x), x2) + __hge2_mask(bf162_of(v[u].y), x2);
            s1 += __hge2_mask(bf162_of(v[u].z), x2) + __hge2_mask(bf162_of(v[u].w), x2);
          }
        }
        const uint32_t sum = s0 + s1, a = (0u - sum) & 0xffffu;
        rank += (int)(2 * a) - ((int)(sum + a) >> 16);
      } else {
#pragma unroll
        for (int u = 0; u < N; ++u) {
          const float x = j + u * kS * W + W <= t ? xt : above;
#pragma unroll
          for (int e = 0; e < W; ++e) rank += chunk_get<DT>(v[u], e) >= x;
        }
      }
    }
    const float ref = fmaxf(st.m, m);
    float d0 = 0.f, d1 = 0.f, n0 = 0.f, n1 = 0.f;
    if (common && fabsf(ref) < 0x1p50f) {
      // -infinity (and what is below -2^60) counts as -2^60: its power is 0, its exponent
      // finite, and the two of a pair take one instruction where a clamp of the exponents
      // takes two
#pragma unroll
      for (int u = 0; u < N; ++u)
#pragma unroll
        for (int e = 0; e < W; e += 2) {
          float x0, x1, a0, a1;
          if constexpr (DT == kBF16) {
            const uint32_t w = bf16x2_max_nan(word_of(v[u], e / 2), 0xdd80dd80u);
            x0 = __uint_as_float(w << 16);
            x1 = __uint_as_float(w & 0xffff0000u);
          } else {
            x0 = max_nan(chunk_get<DT>(v[u], e), -0x1p60f);
            x1 = max_nan(chunk_get<DT>(v[u], e + 1), -0x1p60f);
          }
          scaled2(a0, a1, x0, x1, ref, c);
          const float e0 = ex2(a0), e1 = ex2(a1);
          add2(d0, d1, d0, d1, e0, e1);
          fma2(n0, n1, a0, a1, e0, e1, n0, n1);
        }
    } else {
#pragma unroll
      for (int u = 0; u < N; ++u)
#pragma unroll 1
        for (int e = 0; e < W; ++e) {
          const uint32_t w = DT == kBF16 ? word_at(v[u], e >> 1) : word_at(v[u], e);
          const float x = DT == kF32 ? __uint_as_float(w)
                                     : __uint_as_float((e & 1) ? w & 0xffff0000u : w << 16);
          const float a = max_nan((x - ref) * c, kLow), p = ex2(a);
          d0 += p;
          n0 += a * p;
        }
    }
    add(ref, d0 + d1, n0 + n1);
    return m;
  }
  __device__ __forceinline__ void take1(float x, int j) {
    const float ref = fmaxf(st.m, x), a = max_nan((x - ref) * c, kLow), e = ex2(a);
    add(ref, e, a * e);
    if (kRank) rank += x >= (j < t ? xt : above);
  }
  // sums relative to a new maximum
  __device__ __forceinline__ void add(float ref, float d, float n) {
    const float by = fmaxf((st.m - ref) * c, kLow), f = ex2(by);
    st.n = fmaf(f, fmaf(by, st.d, st.n), n);
    st.d = fmaf(f, st.d, d);
    st.m = ref;
  }
};

// The values before the token in its own chunk, one a lane (-infinity past them), and how
// many of them equal x_t (a warp).
template <int DT>
__device__ __forceinline__ bool own_chunk(const Cut<DT>& cut, int t, float& x) {
  constexpr int E = DType<DT>::E, W = 16 / E;
  const int lane = threadIdx.x & 31;
  x = -INFINITY;
  if (t < cut.head || t >= cut.cols - cut.tail) return false;  // (the ragged ones are exact)
  const int first = cut.head + (t - cut.head) / W * W;
  if (first + lane < t) x = ld_elem_cached<DT>(cut.row + (int64_t)(first + lane) * E);
  return first + lane < t;
}
__device__ __forceinline__ int ties(bool is, float x, float xt) {
  return __popc(__ballot_sync(0xffffffffu, is && x == xt));
}

// ----------------------------------------------------------- a row's outputs ---
// A row whose token is ignored (a warp).
__device__ __forceinline__ void put_ignored(const LogprobParams& p, int64_t r) {
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
    p.logprob[r] = 0.f;
    if (p.entropy) p.entropy[r] = 0.f;
    if (p.row_max) p.row_max[r] = 0.f;
    if (p.log_sum) p.log_sum[r] = 0.f;
    if (p.rank) p.rank[r] = -1;
  }
  for (int i = lane; i < p.k; i += 32) {
    p.top_index[r * p.k + i] = -1;
    p.top_logprob[r * p.k + i] = 0.f;
  }
}
__device__ __forceinline__ bool is_bad(const Stat& st) {  // a NaN or an infinity
  return !(st.d >= 0.f && st.m < INFINITY);
}
// A row's numbers, written where `mine`; returns log_sum.
__device__ __forceinline__ float put_row(const LogprobParams& p, int64_t r, const Stat& st,
                                         bool good, float xt, int rank, bool mine) {
  const float nan = __int_as_float(0x7fc00000);
  const bool bad = is_bad(st), none = st.d == 0.f;  // (nothing but -infinity)
  const float log_sum = bad ? nan : none ? 0.f : logf(st.d);
  if (mine) {
    if (!good && p.bad) atomicAdd(p.bad, 1);
    p.logprob[r] = bad || !good ? nan : none ? 0.f : (xt - st.m) / p.temperature - log_sum;
    if (p.entropy) p.entropy[r] = bad ? nan : none ? 0.f : log_sum - st.n / st.d * kLn2;
    if (p.row_max) p.row_max[r] = bad ? nan : none ? -INFINITY : st.m;
    if (p.log_sum) p.log_sum[r] = log_sum;
    if (p.rank) p.rank[r] = bad || !good ? -1 : rank;
  }
  return log_sum;
}
// Place `at` of a row's list (v 0: no column there).
__device__ __forceinline__ void put_top(const LogprobParams& p, int64_t r, int at,
                                        unsigned long long v, const Stat& st, float log_sum) {
  const bool bad = is_bad(st);
  p.top_index[r * p.k + at] = bad || v == 0 ? -1 : (int32_t)~(uint32_t)v;
  p.top_logprob[r * p.k + at] =
      bad ? __int_as_float(0x7fc00000)
          : v == 0 ? -INFINITY : (unorder((uint32_t)(v >> 32)) - st.m) / p.temperature - log_sum;
}

// Many rows: a row a block at a time.  Four warps stream rows one after the other, each thread
// through a ring of asynchronous copies of its own (64 bytes a stage, four ahead, into the
// next row too).  They do not meet at a row's end: a warp leaves its statistics and its
// threads' maxima (of their whole part of the row, and of its pieces) in shared memory.  Two
// more warps finish every other row each: they read the candidates again and write the row's
// outputs.  The handovers are named barriers: arrivals that do not wait, and waits that take
// no issue slots, as polls would (3 of 12 instructions an element).  Each wait ends: a
// finisher waits for rows being streamed only, and a streaming warp for a row two before.
constexpr int kMainWarps = 4, kMain = 32 * kMainWarps;
constexpr int kFinish = 2;   // warps that finish rows, and rows not yet finished
constexpr int kStages = 4;   // a thread's batches in flight
constexpr int kBlocks = 4;   // an SM
constexpr int kSeg = 32 * kU;                 // chunks of a stage
constexpr int kBatch = kSeg * kMainWarps;     // of all warps' stages
constexpr int kGroups = 16;  // pieces of a thread's part of a row whose maxima are kept
constexpr int kRowCand = 384;
constexpr int kAgain = 128;  // chunks read again at a time
struct RowsShared {
  uint4 ring[kMainWarps][kStages][kSeg];
  Stat stat[kFinish][kMainWarps];
  int rank[kFinish][kMainWarps];
  uint32_t key[kFinish][kMain];
  unsigned short piece[kFinish][kGroups][kMain];  // bf16, rounded up
  unsigned short owner[kFinish][kMain], piece_of[kFinish][kMain * 2];
  unsigned long long cand[kFinish][kRowCand];
  uint4 again[kFinish][kAgain];
  int column[kFinish][kAgain];
};
__device__ __forceinline__ void bar_arrive(int id, int count) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}
// Row of slot f streamed: the four warps arrive, the finisher waits.  Row of slot f finished:
// the finisher arrives, warp w waits.
constexpr int kStreamed = kMain + 32, kFinished = 64;
__device__ __forceinline__ int streamed_id(int f) { return 1 + f; }
__device__ __forceinline__ int finished_id(int f, int w) { return 1 + kFinish + f * kMainWarps + w; }
static_assert(1 + kFinish + kFinish * kMainWarps <= 16, "named barriers");
// log2 of a piece's batches: at most kGroups pieces a thread.
__device__ __forceinline__ int piece_shift(int chunks) {
  int s = 0;
  while ((chunks - 1) / (kBatch << s) >= kGroups) ++s;
  return s;
}
__device__ __forceinline__ unsigned short bf16_up(float x) {
  unsigned short h;
  asm("cvt.rp.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
  return h;
}

// The k largest of a row, by one warp: candidates into sh.cand, their number (long ties: k of
// them, in order).
template <int DT>
__device__ __forceinline__ int find_largest(RowsShared& sh, int slot, const Cut<DT>& cut, int k,
                                            float greatest) {
  constexpr int E = DType<DT>::E, W = 16 / E, NW = kMain / 32;
  const int lane = threadIdx.x & 31, n = (int)cut.chunks;
  const uint32_t below = (1u << lane) - 1u;
  unsigned short *owner = sh.owner[slot], *piece_of = sh.piece_of[slot];
  unsigned long long* cand = sh.cand[slot];
  uint32_t mine[NW];
#pragma unroll
  for (int w = 0; w < NW; ++w) mine[w] = sh.key[slot][w * 32 + lane];
  // a lower bound of the k-th largest logit: the k-th largest of the lanes' maxima, as long
  // as not many more logits than k can be expected above it (some 44 for k = 24), or a value
  // that at least k, and not many more, of the pieces' maxima reach (bisection of the bits; a
  // maximum rounded up to T is above the bf16 before T).  Ranks and k = 20, 24, 25, 28 of 16384 x
  // 50304 bf16 by the first 367, 392, 398, 446 us, by the second 396, 405, 407, 413; 8192 rows
  // fp32 with 20 and 24 306 and 319, 298 and 300.
  const int shift = piece_shift(n);
  const int groups = (n - 1) / (kBatch << shift) + 1;
  uint32_t lo = order(-INFINITY) + 1u;
  if (k <= 24) {
    uint32_t top = mine[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) top = max(top, mine[w]);
    int before = 0;
#pragma unroll 4
    for (int w = 0; w < 32; ++w) {
      const uint32_t o = __shfl_sync(0xffffffffu, top, w);
      before += o > top || (o == top && w < lane);
    }
    const uint32_t who = __ballot_sync(0xffffffffu, before == k - 1);
    lo = max(lo, __shfl_sync(0xffffffffu, top, __ffs(who) - 1));
  } else {
    const uint32_t* maxima = reinterpret_cast<const uint32_t*>(sh.piece[slot]);
    uint32_t a = lo >> 16, b = (order(greatest) >> 16) + 2u;  // bf16, ordered
    while (b - a > 1) {
      const uint32_t mid = a + (b - a) / 2;
      const __nv_bfloat162 x2 = bf162_of((__float_as_uint(unorder(mid << 16)) >> 16) * 0x10001u);
      __nv_bfloat162 count = __float2bfloat162_rn(0.f);  // (at most 32 a half: exact)
#pragma unroll 4
      for (int i = lane; i < groups * (kMain / 2); i += 32)
        count = __hadd2(count, __hge2(bf162_of(maxima[i]), x2));
      const int cnt = __reduce_add_sync(0xffffffffu,
                                        (int)(__low2float(count) + __high2float(count)));
      if (cnt < k) {
        b = mid;
      } else {
        a = mid;
        if (cnt <= k + k / 4) break;
      }
    }
    lo = max(lo, DT == kBF16 ? a << 16 : (a - 1u) << 16);
  }
  const float least = unorder(lo);
  int owners = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const uint32_t has = __ballot_sync(0xffffffffu, mine[w] >= lo);
    if (mine[w] >= lo) owner[owners + __popc(has & below)] = (unsigned short)(w * 32 + lane);
    owners += __popc(has);
  }
  __syncwarp();
  // of those threads, the pieces whose maximum reaches it: their elements are read again (a
  // sixteenth or less of a thread's part of the row, where the row itself may have left L2)
  const int wide = groups > 8 ? 4 : 3;  // (log2, at least, of groups)
  int pieces = 0;
  constexpr int kMost = kMain * 2;
  for (int o = lane; o < (owners << wide) + lane; o += 32) {
    bool has = false;
    int code = 0;
    if (o < owners << wide) {
      const int who = owner[o >> wide], g = o & ((1 << wide) - 1);
      code = g * 512 + who;
      has = g < groups && bf16_bits_to_f32(sh.piece[slot][g][who]) >= least;
    }
    const uint32_t all = __ballot_sync(0xffffffffu, has);
    const int at = pieces + __popc(all & below);
    if (has && at < kMost) piece_of[at] = (unsigned short)code;
    pieces += __popc(all);
  }
  __syncwarp();
  int found = 0;
  auto put = [&](bool has, float x, int j) {  // (all lanes)
    const uint32_t all = __ballot_sync(0xffffffffu, has);
    if (all == 0) return;
    const int at = found + __popc(all & below);
    if (has && at < kRowCand)
      cand[at] = ((unsigned long long)order(x) << 32) | (uint32_t)~(uint32_t)j;
    found += __popc(all);
  };
  // (by way of shared memory, so that a lane has several loads in flight and the code is short:
  // the streaming warps share the instruction cache)
  const int all = pieces > kMost ? 0 : pieces << (shift + 2);
  static_assert(kU == 4, "a piece's chunks are counted in fours");
  for (int o = 0; o < all; o += kAgain) {
#pragma unroll
    for (int u = 0; u < kAgain; u += 32) {
      const int i = o + u + lane;
      int at = n;
      if (i < all) {
        const int code = piece_of[i >> (shift + 2)], q = i & ((4 << shift) - 1), who = code & 511;
        at = (((code >> 9) << shift) + (q >> 2)) * kBatch + (who >> 5) * kSeg + (q & 3) * 32 +
             (who & 31);
      }
      sh.column[slot][u + lane] = at < n ? cut.head + at * W : -1;
      if (at < n) cp_async16(&sh.again[slot][u + lane], cut.chunk(at));
    }
    cp_async_commit();
    cp_async_wait<0>();
#pragma unroll 1
    for (int u = lane; u < min(kAgain, all - o) + lane; u += 32) {
      const int j = sh.column[slot][u];
      const uint4 v = j < 0 ? chunk_fill<DT>(-INFINITY) : sh.again[slot][u];
#pragma unroll
      for (int e = 0; e < W; ++e) {
        const float x = chunk_get<DT>(v, e);
        put(x >= least, x, j + e);
      }
    }
    __syncwarp();
  }
  auto ragged = [&](auto f) {
    const int j = (int)cut.cols - cut.tail + lane;
    f(lane < cut.head, lane < cut.head ? ld_elem_cached<DT>(cut.row + lane * E) : -INFINITY, lane);
    f(lane < cut.tail, lane < cut.tail ? ld_elem_cached<DT>(cut.row + (int64_t)j * E) : -INFINITY, j);
  };
  ragged([&](bool is, float x, int j) { put(is && x >= least, x, j); });
  __syncwarp();
  if (pieces <= kMost && found <= kRowCand) return found;
  // too many columns reach the bound: the largest below the last, k times
  unsigned long long last = ~0ull;
  for (int at = 0; at < k; ++at) {
    unsigned long long best = 0;
    auto look = [&](bool is, float x, int j) {
      const unsigned long long v = ((unsigned long long)order(x) << 32) | (uint32_t)~(uint32_t)j;
      if (is && v < last && v > best) best = v;
    };
#pragma unroll 4
    for (int q = lane; q < n; q += 32) {
      const uint4 v = ld_chunk_cached(cut.chunk(q));
#pragma unroll
      for (int e = 0; e < W; ++e) look(true, chunk_get<DT>(v, e), cut.head + q * W + e);
    }
    ragged(look);
    for (int off = 16; off >= 1; off >>= 1)
      best = max(best, __shfl_xor_sync(0xffffffffu, best, off));
    last = best;
    if (lane == 0) cand[at] = best;
  }
  __syncwarp();
  return k;
}

template <int DT, bool kRank>
__global__ void __launch_bounds__(kMain + 32 * kFinish, kBlocks)
    logprob_rows_kernel(const LogprobParams p) {
  constexpr int E = DType<DT>::E, W = 16 / E, NW = kMainWarps;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  RowsShared& sh = *reinterpret_cast<RowsShared*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // tokens are read two rows ahead, their logits one
  const int64_t g = gridDim.x;
  auto token = [&](int64_t r) { return r < p.rows ? __ldg(p.tokens + r) : p.ignore; };
  auto logit = [&](int64_t r, int t) {
    return t >= 0 && t < p.cols && r < p.rows
               ? ld_elem_cached<DT>(p.x + (r * p.stride + t) * E)
               : 0.f;
  };
  auto row_at = [&](int64_t r) { return Cut<DT>(p.x + r * p.stride * E, p.cols); };
  int64_t r = blockIdx.x;
  int t1 = token(r), t2 = token(r + g), i = 0;  // i: rows taken (ignored ones do not count)
  if (warp < NW) {
    // the copies ahead: chunks of row rc, from `src` on, `left` of them from this warp's next
    // segment to the row's end (every call is one group of copies, the last ones empty)
    int64_t rc = blockIdx.x;
    int c1 = t1, c2 = t2, left = 0, put_at = 0, get_at = 0;
    const char* src = nullptr;
    bool begun = false;
    auto advance = [&]() {  // to the next row that has a segment for this warp
      do {
        if (begun) {
          rc += g;
          c1 = c2;
          c2 = token(rc + g);
        }
        begun = true;
        if (rc >= p.rows) return;
        const Cut<DT> cut = row_at(rc);
        left = c1 != p.ignore ? (int)cut.chunks - warp * kSeg : 0;
        src = cut.chunk(warp * kSeg + lane);
      } while (left <= 0);
    };
    auto ask = [&]() {
      if (left <= 0 && rc < p.rows) advance();
      uint4* dst = &sh.ring[warp][put_at][lane];
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (32 * u + lane < left) cp_async16(dst + 32 * u, src + 512 * u);
      cp_async_commit();
      src += kBatch * 16;
      left -= kBatch;
      put_at = put_at + 1 == kStages ? 0 : put_at + 1;
    };
    for (int k = 0; k < kStages; ++k) ask();
    float x1 = kRank ? logit(r, t1) : 0.f;
    for (; r < p.rows; r += g) {
      const int t = t1;
      const float xt = x1;
      t1 = t2;
      t2 = token(r + 2 * g);
      if (kRank) x1 = logit(r + g, t1);
      if (t == p.ignore) continue;
      const Cut<DT> cut = row_at(r);
      // (ragged elements are asked for now and taken at the row's end)
      float xh = 0.f, xl = 0.f;
      if (tid < cut.head) xh = ld_elem_cached<DT>(cut.row + tid * E);
      const int jl = (int)cut.cols - cut.tail + tid;
      if (tid < cut.tail) xl = ld_elem_cached<DT>(cut.row + (int64_t)jl * E);
      Pass<DT, kRank, 32> pass(p.c, xt, t);
      const int f = i % kFinish;
      if (i >= kFinish) named_bar(finished_id(f, warp), kFinished);
      const int n = (int)cut.chunks, per = 1 << piece_shift(n);
      int batch = 0, piece = 0;
      float most = -INFINITY;  // of the piece at hand
      for (int at = warp * kSeg; at < n; at += kBatch) {
        cp_async_wait<kStages - 1>();
        uint4 v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) v[u] = sh.ring[warp][get_at][32 * u + lane];
        if (at + kSeg > n)
#pragma unroll
          for (int u = 0; u < kU; ++u)
            if (at + 32 * u + lane >= n) v[u] = chunk_fill<DT>(-INFINITY);
        get_at = get_at + 1 == kStages ? 0 : get_at + 1;
        ask();  // into the stage just read
        const float m = pass.template take<kU>(v, cut.head + (at + lane) * W);
        if (p.k > 0) {
          most = fmaxf(most, m);
          if (++batch == per) {
            sh.piece[f][piece++][tid] = bf16_up(most);
            batch = 0;
            most = -INFINITY;
          }
        }
      }
      if (p.k > 0 && piece < kGroups) sh.piece[f][piece][tid] = bf16_up(most);
      if (tid < cut.head) pass.take1(xh, tid);
      if (tid < cut.tail) pass.take1(xl, jl);
      Stat st = pass.st;
      sh.key[f][tid] = order(st.m);
      for (int off = 16; off >= 1; off >>= 1) {
        const Stat o = shfl_xor(st, off);
        st = (lane & off) ? merge(o, st, p.c) : merge(st, o, p.c);
      }
      const int rank = kRank ? __reduce_add_sync(0xffffffffu, pass.rank) : 0;
      if (lane == 0) {
        sh.stat[f][warp] = st;
        sh.rank[f][warp] = rank;
      }
      __syncwarp();
      bar_arrive(streamed_id(f), kStreamed);
      ++i;
    }
    for (int k = max(i - kFinish, 0); k < i; ++k) named_bar(finished_id(k % kFinish, warp), kFinished);
    cp_async_wait<0>();
  } else {
    const int f = warp - NW;
    for (; r < p.rows; r += g) {
      const int t = t1;
      t1 = t2;
      t2 = token(r + 2 * g);
      if (t == p.ignore) {
        if (f == 0) put_ignored(p, r);
        continue;
      }
      if (i++ % kFinish != f) continue;
      const Cut<DT> cut = row_at(r);
      const bool good = t >= 0 && t < p.cols;
      const float xt = logit(r, t);
      float before;
      const bool own = kRank && good && own_chunk(cut, t, before);
      named_bar(streamed_id(f), kStreamed);
      Stat st = sh.stat[f][lane % NW];
      int rank = kRank ? __reduce_add_sync(0xffffffffu, lane < NW ? sh.rank[f][lane] : 0) : 0;
#pragma unroll
      for (int off = 1; off < NW; off <<= 1) {
        const Stat o = shfl_xor(st, off);
        st = (lane & off) ? merge(o, st, p.c) : merge(st, o, p.c);
      }
      if (kRank) rank += ties(own, before, xt);
      const float log_sum = put_row(p, r, st, good, xt, rank, lane == 0);
      if (p.k > 0) {
        int found = 0;
        if (st.d != 0.f) found = find_largest<DT>(sh, f, cut, p.k, st.m);
        // each candidate's place is the number of greater ones
        const unsigned long long* cand = sh.cand[f];
        for (int q = lane; q < found; q += 64) {
          const unsigned long long v = cand[q], v2 = q + 32 < found ? cand[q + 32] : 0;
          int at = 0, at2 = 0;
#pragma unroll 4
          for (int w = 0; w < found; ++w) {
            const unsigned long long o = cand[w];
            at += o > v;
            at2 += o > v2;
          }
          if (at < p.k) put_top(p, r, at, v, st, log_sum);
          if (v2 != 0 && at2 < p.k) put_top(p, r, at2, v2, st, log_sum);
        }
        for (int q = found + lane; q < p.k; q += 32) put_top(p, r, q, 0, st, log_sum);
      }
      __syncwarp();
      for (int w = 0; w < NW; ++w) bar_arrive(finished_id(f, w), kFinished);
    }
  }
}

// Few rows: a row a cluster, whose blocks take a slice each, all of their warps at every
// step, and hand their statistics and their k largest to the first.
template <int DT, bool kRank>
__global__ void __launch_bounds__(kT, 4) logprob_cluster_kernel(const LogprobParams p) {
  constexpr int E = DType<DT>::E, W = 16 / E, NW = kT / 32;
  constexpr int kMost = 8;  // blocks of a cluster
  __shared__ Stat s_stat[NW];
  __shared__ int s_rank[NW], s_count, s_owners;
  __shared__ uint32_t s_key[kT], s_thr;
  __shared__ unsigned short s_owner[kT];
  __shared__ unsigned long long s_cand[kCand];
  __shared__ float4 s_part[kMost];
  static_assert(alignof(decltype(s_part)) >= 16, "written 16 bytes at a time by other blocks");
  __shared__ unsigned long long s_list[kMost * kLogprobMaxK];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = (int)cluster_nrank(), me = (int)cluster_rank();
  // (the first block's shared memory is written once all have started)
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  const int64_t r = blockIdx.x / K;
  const int t = __ldg(p.tokens + r);
  if (t == p.ignore) {
    if (me == 0 && warp == 0) put_ignored(p, r);
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    return;
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
  Pass<DT, kRank, kT> pass(p.c, xt, t);
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
  if (kRank && good && me == 0) {
    float before;
    const bool own = own_chunk(cut, t, before);
    ranks = ties(own, before, xt);
  }
  if (kRank)
#pragma unroll
    for (int w = 0; w < NW; ++w) ranks += s_rank[w];
  // the slice's k largest: candidates in s_cand, or (long ties) one after the other
  int found = 0;
  const bool listed = p.k > 0 && st.d != 0.f;
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
  {
    // to the first block: statistics, and the k largest in order (0: no column)
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (tid == 0)
      st_cluster_f32x4(map_to_rank(&s_part[me], 0), st.m, st.d, st.n, __int_as_float(ranks));
    const uint32_t list = map_to_rank(s_list, 0) + me * p.k * 8;
    for (int q = found + tid; q < p.k; q += kT) st_cluster_u64(list + q * 8, 0ull);
    for (int q = tid; q < found; q += kT) {
      const unsigned long long v = s_cand[q];
      int at = 0;
      for (int w = 0; w < found; ++w) at += s_cand[w] > v;
      if (at < p.k) st_cluster_u64(list + at * 8, v);
    }
    cluster_sync();
    if (me != 0) return;
    st = Stat{s_part[0].x, s_part[0].y, s_part[0].z};
    ranks = __float_as_int(s_part[0].w);
    for (int w = 1; w < K; ++w) {
      st = merge(st, Stat{s_part[w].x, s_part[w].y, s_part[w].z}, c);
      ranks += __float_as_int(s_part[w].w);
    }
    found = K * p.k;
  }
  const float log_sum = put_row(p, r, st, good, xt, ranks, tid == 0);
  if (p.k > 0) {
    // each candidate's place is the number of greater ones
    int live = 0;
    for (int q = 0; q < found; ++q) live += s_list[q] != 0;
    for (int q = tid; q < found; q += kT) {
      const unsigned long long v = s_list[q];
      if (v == 0) continue;
      int at = 0;
      for (int w = 0; w < found; ++w) at += s_list[w] > v;
      if (at < p.k) put_top(p, r, at, v, st, log_sum);
    }
    for (int q = live + tid; q < p.k; q += kT) put_top(p, r, q, 0, st, log_sum);
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
  // (1 / T comes last: at a low temperature A and B over T may overflow where p is 0)
  const float A = -(g + h * ent), B = -h * kLn2;
  const float ls = __ldg(p.log_sum + r) * kLog2e;
  // of two neighbours' logits, in place
  auto grad = [&](float& x0, float& x1, int64_t j) {
    if (zero) {
      x0 = x1 = 0.f;
      return;
    }
    float a0, a1, v0, v1;
    add2(a0, a1, x0, x1, -m, -m);
    fma2(a0, a1, a0, a1, c, c, -ls, -ls);
    a0 = max_nan(a0, kLow), a1 = max_nan(a1, kLow);
    fma2(v0, v1, a0, a1, B, B, A, A);
    mul2(v0, v1, v0, v1, ex2(a0), ex2(a1));
    if (j == t) v0 += g;
    if (j + 1 == t) v1 += g;
    mul2(x0, x1, v0, v1, inv, inv);
  };
  auto grad1 = [&](float x, int64_t j) {
    float none = m;
    grad(x, none, j);
    return x;
  };
  if constexpr (kV) {
    for (int u = 0; u < kU; ++u) {
      const int64_t i = ((int64_t)seg * kU + u) * kT + tid;
      if (i >= cut.chunks) break;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (!zero) v = ld_chunk_stream(cut.chunk(i));
      float f[W];
#pragma unroll
      for (int e = 0; e < W; e += 2) {
        f[e] = chunk_get<DT>(v, e);
        f[e + 1] = chunk_get<DT>(v, e + 1);
        grad(f[e], f[e + 1], cut.head + i * W + e);
      }
      st_chunk_stream(out + (int64_t)cut.head * E + i * 16, chunk_pack<DT>(f));
    }
    if (seg == 0)
      each_ragged<DT>(cut, tid, [&](float x, int64_t j) { st_elem<DT>(out + j * E, grad1(x, j)); });
  } else {
    for (int u = 0; u < kU * W; ++u) {
      const int64_t j = ((int64_t)seg * kU * W + u) * kT + tid;
      if (j >= p.cols) break;
      st_elem<DT>(out + j * E, grad1(zero ? 0.f : ld_elem<DT>(cut.row + j * E), j));
    }
  }
}

}  // namespace

template <int DT>
static LogprobKernels kernels_of() {
  return LogprobKernels{
      {(const void*)logprob_rows_kernel<DT, false>, (const void*)logprob_rows_kernel<DT, true>},
      {(const void*)logprob_cluster_kernel<DT, false>, (const void*)logprob_cluster_kernel<DT, true>},
      {(const void*)logprob_bwd_kernel<DT, false>, (const void*)logprob_bwd_kernel<DT, true>},
      kT,
      kMain + 32 * kFinish,
      (int)sizeof(RowsShared),
      kT * kU * 16};
}
LogprobKernels logprob_kernels(int dtype) {
  return dtype == kF32 ? kernels_of<kF32>() : kernels_of<kBF16>();
}

}  // namespace rr
