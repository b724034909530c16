// k_rope.cu -- norms of queries and keys, head by head, with the position rotation in
// the same pass, and its gradient.
//
// A row is one head of one token, D elements.  With x its values, w the weight that all
// heads share and (c, s) the cosine and sine of the token's angle for a pair (a, b):
//   r = 1 / sqrt(sum x^2 / D + eps),  u = x r w,
//   y_a = c u_a - s u_b,  y_b = s u_a + c u_b   (elements behind the rotated ones: y = u),
// and backward, with g = the pair turned back by its angle:
//   dw = sum over rows of g x r,  h = g w,  dx = r (h - x r mean(h x r)).
// Nothing is saved between the two: the row is in registers anyway when r is needed.
//
// A lane owns a slot of a row: two chunks of W elements that hold W whole pairs (halves:
// chunk j and the one R / 2 elements on; neighbours: two adjacent chunks), so the rotation
// needs no exchange and the row's one sum is a butterfly over its D / 2W lanes.  A warp
// takes 32 / G heads of one token at a time and walks over the token's queries (or keys)
// with the token's cosines and sines in registers.
#include <cstdint>

#include "rr_device.cuh"
#include "rr_kernels.h"

namespace rr {
namespace {

constexpr int kThreads = 256;
// Row groups in flight a warp, and blocks an SM.  Memory bounds both kernels (the forward reads
// and writes each row once, the backward reads two and writes one); what they lack is bytes
// under way, which cost registers.  16384 tokens, bf16, 32 + 8 heads of 128 read and written by
// the forward: 60 us with 2 and 3, 5690 GB/s (2 and 4: 70, 3 and 3: 66, 1 and 5: 87; each row's
// loads issued before the one before it is worked on, 83); backward 103 us, 4960 GB/s, with 2
// and 2 (2 and 3: 137, 3 and 2: 113; likewise 149).  The bf16 kernels as they are keep 44 and 58
// bytes a thread in local memory; copies into shared memory were not tried.
constexpr int kFwdU = 2, kBwdU = 2, kFwdBlocks = 3, kBwdBlocks = 2;

// What a lane keeps of the row's layout: element offsets of its slots.
template <int W, int NS>
struct Slots {
  int ea[NS], eb[NS], ang[NS];
  bool on[NS], rot[NS];
  __device__ __forceinline__ Slots(int gl, const RopeParams& p) {
    const int n2 = p.dim / (2 * W), nrot = p.rot / (2 * W);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int s = gl + i * p.group;
      on[i] = s < n2;
      rot[i] = s < nrot;
      ang[i] = s * W;
      if (p.interleaved) {
        ea[i] = 2 * s * W;
        eb[i] = ea[i] + W;
      } else if (rot[i]) {
        ea[i] = s * W;
        eb[i] = p.rot / 2 + s * W;
      } else {
        ea[i] = p.rot + 2 * (s - nrot) * W;
        eb[i] = ea[i] + W;
      }
    }
  }
};

template <int DT, int W>
__device__ __forceinline__ void load_cached(float (&f)[W], const char* p) {
  if constexpr (W == 1) {
    f[0] = ld_elem_cached<DT>(p);
  } else {
    const uint4 c = ld_chunk_cached(p);
#pragma unroll
    for (int i = 0; i < W; ++i) f[i] = chunk_get<DT>(c, i);
  }
}
template <int DT, int W>
__device__ __forceinline__ void store(char* p, const float (&f)[W]) {
  if constexpr (W == 1)
    st_elem<DT>(p, f[0]);
  else
    *reinterpret_cast<uint4*>(p) = chunk_pack<DT>(f);
}

// Element by element, two at a time where there are two (half of the kernels' instructions
// are these): x *= y, x *= f, d += the sum of x y, d += x y, d += x f.
template <int W>
__device__ __forceinline__ void times(float (&x)[W], const float (&y)[W]) {
  if constexpr (W == 1) {
    x[0] *= y[0];
  } else {
#pragma unroll
    for (int e = 0; e < W; e += 2) mul2(x[e], x[e + 1], x[e], x[e + 1], y[e], y[e + 1]);
  }
}
template <int W>
__device__ __forceinline__ void times(float (&x)[W], float f) {
  if constexpr (W == 1) {
    x[0] *= f;
  } else {
#pragma unroll
    for (int e = 0; e < W; e += 2) mul2(x[e], x[e + 1], x[e], x[e + 1], f, f);
  }
}
template <int W>
__device__ __forceinline__ void add_to(float (&d)[2], const float (&x)[W], const float (&y)[W]) {
  if constexpr (W == 1) {
    d[0] += x[0] * y[0];
  } else {
#pragma unroll
    for (int e = 0; e < W; e += 2)
      fma2(d[0], d[1], x[e], x[e + 1], y[e], y[e + 1], d[0], d[1]);
  }
}
template <int W>
__device__ __forceinline__ void add_each(float (&d)[W], const float (&x)[W], const float (&y)[W]) {
  if constexpr (W == 1) {
    d[0] += x[0] * y[0];
  } else {
#pragma unroll
    for (int e = 0; e < W; e += 2)
      fma2(d[e], d[e + 1], x[e], x[e + 1], y[e], y[e + 1], d[e], d[e + 1]);
  }
}
template <int W>
__device__ __forceinline__ void plus(float (&d)[W], const float (&x)[W], float f) {
  if constexpr (W == 1) {
    d[0] += x[0] * f;
  } else {
#pragma unroll
    for (int e = 0; e < W; e += 2) fma2(d[e], d[e + 1], x[e], x[e + 1], f, f, d[e], d[e + 1]);
  }
}

// Turns the slot's pairs by (c, s).
template <int W>
__device__ __forceinline__ void turn(float (&a)[W], float (&b)[W], const float (&c)[W],
                                     const float (&s)[W], bool neighbours) {
  if (W > 1 && neighbours) {
    float u[2 * W];
#pragma unroll
    for (int i = 0; i < W; ++i) u[i] = a[i], u[W + i] = b[i];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float x = u[2 * i], y = u[2 * i + 1];
      u[2 * i] = c[i] * x - s[i] * y;
      u[2 * i + 1] = s[i] * x + c[i] * y;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) a[i] = u[i], b[i] = u[W + i];
  } else if constexpr (W == 1) {
    const float x = a[0], y = b[0];
    a[0] = c[0] * x - s[0] * y;
    b[0] = s[0] * x + c[0] * y;
  } else {
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      float t0, t1, u0, u1;
      mul2(t0, t1, s[i], s[i + 1], b[i], b[i + 1]);
      mul2(u0, u1, s[i], s[i + 1], a[i], a[i + 1]);
      fma2(a[i], a[i + 1], c[i], c[i + 1], a[i], a[i + 1], -t0, -t1);
      fma2(b[i], b[i + 1], c[i], c[i + 1], b[i], b[i + 1], u0, u1);
    }
  }
}

__device__ __forceinline__ float group_sum(float v, int group) {
  for (int off = group >> 1; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The token's angles for this lane's slots; out of the table: NaN, counted once a token.
template <int W, int NS>
__device__ __forceinline__ void angles(float (&c)[NS][W], float (&s)[NS][W],
                                       const Slots<W, NS>& sl, const RopeParams& p, int pos) {
#pragma unroll
  for (int i = 0; i < NS; ++i) {
#pragma unroll
    for (int e = 0; e < W; ++e) c[i][e] = 1.f, s[i][e] = 0.f;
    if (!sl.rot[i]) continue;
    if (pos < 0 || pos >= p.positions_n) {
#pragma unroll
      for (int e = 0; e < W; ++e) c[i][e] = s[i][e] = __int_as_float(0x7fc00000);
    } else {
      const int64_t at = (int64_t)pos * (p.rot / 2) + sl.ang[i];
      if constexpr (W == 1) {
        c[i][0] = __ldg(p.cos + at);
        s[i][0] = __ldg(p.sin + at);
      } else {
#pragma unroll
        for (int e = 0; e < W; e += 4) {
          const float4 cv = __ldg(reinterpret_cast<const float4*>(p.cos + at + e));
          const float4 sv = __ldg(reinterpret_cast<const float4*>(p.sin + at + e));
          c[i][e] = cv.x, c[i][e + 1] = cv.y, c[i][e + 2] = cv.z, c[i][e + 3] = cv.w;
          s[i][e] = sv.x, s[i][e + 1] = sv.y, s[i][e + 2] = sv.z, s[i][e + 3] = sv.w;
        }
      }
    }
  }
}

// A warp's share of the work: units of rows of one kind (all queries' units, then the keys'),
// each a token's rows [first, last) of that kind.  Units of a warp are gridDim x warps apart.
struct Unit {
  int64_t t;
  int first, last;
  bool isq;
};
__device__ __forceinline__ Unit unit_of(const RopeParams& p, int64_t u) {
  Unit x;
  const int64_t nq = p.tokens * p.q_segs;
  x.isq = u < nq;
  const int segs = x.isq ? p.q_segs : p.k_segs, rows = x.isq ? p.q_rows : p.k_rows;
  const int64_t v = x.isq ? u : u - nq;
  x.t = v <= 0xffffffffll ? (uint32_t)v / (uint32_t)segs : v / segs;
  x.first = (int)(v - x.t * segs) * rows;
  x.last = min(x.isq ? p.heads : p.kv_heads, x.first + rows);
  return x;
}
__device__ __forceinline__ int position_of(const RopeParams& p, int64_t t) {
  return p.positions ? __ldg(p.positions + t) : (int)t;
}
__device__ __forceinline__ void count_bad(const RopeParams& p, const Unit& x, int pos) {
  if (p.bad && pos >= p.positions_n && x.isq && x.first == 0 && (threadIdx.x & 31) == 0)
    atomicAdd(p.bad, 1);
}

// A slot's two chunks as they are stored.
template <int DT, int W>
struct Raw {
  uint4 a, b;
  __device__ __forceinline__ void load(const char* x, int ea, int eb) {
    constexpr int E = DType<DT>::E;
    if constexpr (W == 1) {
      a.x = ld_elem_bits<DT>(x + ea * E);
      b.x = ld_elem_bits<DT>(x + eb * E);
    } else {
      a = ld_chunk_stream(x + ea * E);
      b = ld_chunk_stream(x + eb * E);
    }
  }
  __device__ __forceinline__ void get(float (&fa)[W], float (&fb)[W]) const {
#pragma unroll
    for (int e = 0; e < W; ++e) {
      fa[e] = W == 1 ? bits_to_f32<DT>(a.x) : chunk_get<DT>(a, e);
      fb[e] = W == 1 ? bits_to_f32<DT>(b.x) : chunk_get<DT>(b, e);
    }
  }
};

// U row groups' loads are issued before the first is needed: what bounds the kernel is how
// many bytes are under way.
template <int DT, int W, int NS, int U>
__global__ void __launch_bounds__(kThreads, kFwdBlocks) rope_fwd_kernel(const RopeParams p) {
  constexpr int E = DType<DT>::E;
  const int lane = threadIdx.x & 31;
  const int gl = lane & (p.group - 1), sub = lane / p.group, per = 32 / p.group;
  const Slots<W, NS> sl(gl, p);
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  const int64_t units = p.tokens * (p.q_segs + p.k_segs);
  int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (u >= units) return;
  Unit x = unit_of(p, u);
  int pos = position_of(p, x.t);
  while (true) {
    const Unit now = x;
    const int at = pos;
    u += warps;
    if (u < units) {
      x = unit_of(p, u);
      pos = position_of(p, x.t);
    }
    const char* in = (now.isq ? p.q + now.t * p.q_stride * E : p.k + now.t * p.k_stride * E);
    char* out = (now.isq ? p.qo + now.t * p.qo_stride * E : p.ko + now.t * p.ko_stride * E);
    const char* w = now.isq ? p.qw : p.kw;
    count_bad(p, now, at);
    float c[NS][W], s[NS][W];
    for (int r0 = now.first; r0 < now.last; r0 += U * per) {
      Raw<DT, W> raw[U][NS];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int h = r0 + k * per + sub;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          raw[k][i].a = raw[k][i].b = make_uint4(0, 0, 0, 0);
          if (h < now.last && sl.on[i]) raw[k][i].load(in + (int64_t)h * p.dim * E, sl.ea[i], sl.eb[i]);
        }
      }
      if (r0 == now.first) angles<W, NS>(c, s, sl, p, at);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int h = r0 + k * per + sub;
        if (r0 + k * per >= now.last) break;
        float a[NS][W], b[NS][W], ss[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          raw[k][i].get(a[i], b[i]);
          add_to<W>(ss, a[i], a[i]);
          add_to<W>(ss, b[i], b[i]);
        }
        const float ms = group_sum(ss[0] + ss[1], p.group) * p.inv_dim;
        const bool keep = at >= 0 && ms <= 3.402823466e38f && ms + p.eps > 0.f;
        const float r = keep ? rsqrtf(ms + p.eps) : 0.f;
        if (h >= now.last) continue;
        char* y = out + (int64_t)h * p.dim * E;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          if (!sl.on[i]) continue;
          if (keep) {
            times<W>(a[i], r);
            times<W>(b[i], r);
            if (w) {
              float wi[W];
              load_cached<DT, W>(wi, w + sl.ea[i] * E);
              times<W>(a[i], wi);
              load_cached<DT, W>(wi, w + sl.eb[i] * E);
              times<W>(b[i], wi);
            }
            turn<W>(a[i], b[i], c[i], s[i], p.interleaved);
          } else {
#pragma unroll
            for (int e = 0; e < W; ++e) a[i][e] = b[i][e] = 0.f;
          }
          store<DT, W>(y + sl.ea[i] * E, a[i]);
          store<DT, W>(y + sl.eb[i] * E, b[i]);
        }
      }
    }
    if (u >= units) return;
  }
}

// dx of every row, and this block's sums over its rows of g x r for the two weights, in
// workspace row blockIdx.x ([2][D] floats), which rope_join_kernel adds up.  A warp's rows
// are queries first, then keys: one set of sums, put aside between the two.
template <int DT, int W, int NS, int U>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) rope_bwd_kernel(const RopeParams p) {
  constexpr int E = DType<DT>::E;
  extern __shared__ float part[];  // [warps][2][D]
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // (the join may come)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gl = lane & (p.group - 1), sub = lane / p.group, per = 32 / p.group;
  const Slots<W, NS> sl(gl, p);
  float acc[NS][2][W];
#pragma unroll
  for (int i = 0; i < NS * 2 * W; ++i) (&acc[0][0][0])[i] = 0.f;
  // the warp's row groups, in a fixed order, to its place for queries (0) or keys (1)
  auto put_aside = [&](int kind) {
#pragma unroll
    for (int i = 0; i < NS * 2 * W; ++i) {
      float v = (&acc[0][0][0])[i];
      for (int off = p.group; off < 32; off <<= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
      (&acc[0][0][0])[i] = v;
    }
    if (sub == 0)
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (sl.on[i])
#pragma unroll
          for (int e = 0; e < W; ++e) {
            part[(warp * 2 + kind) * p.dim + sl.ea[i] + e] = acc[i][0][e];
            part[(warp * 2 + kind) * p.dim + sl.eb[i] + e] = acc[i][1][e];
          }
#pragma unroll
    for (int i = 0; i < NS * 2 * W; ++i) (&acc[0][0][0])[i] = 0.f;
  };
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  const int64_t units = p.tokens * (p.q_segs + p.k_segs);
  int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + warp;
  bool queries = true;
  Unit x = unit_of(p, u < units ? u : 0);
  int pos = position_of(p, x.t);
  while (u < units) {
    const Unit now = x;
    const int at = pos;
    u += warps;
    if (u < units) {
      x = unit_of(p, u);
      pos = position_of(p, x.t);
    }
    if (queries && !now.isq) {
      if (p.ws) put_aside(0);
      queries = false;
    }
    const char* in = (now.isq ? p.q + now.t * p.q_stride * E : p.k + now.t * p.k_stride * E);
    const char* gin = (now.isq ? p.dyq + now.t * p.dyq_stride * E : p.dyk + now.t * p.dyk_stride * E);
    char* out = (now.isq ? p.qo + now.t * p.qo_stride * E : p.ko + now.t * p.ko_stride * E);
    const char* w = now.isq ? p.qw : p.kw;
    count_bad(p, now, at);
    float c[NS][W], s[NS][W];
    for (int r0 = now.first; r0 < now.last; r0 += U * per) {
      Raw<DT, W> rx[U][NS], rg[U][NS];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int h = r0 + k * per + sub;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          rx[k][i].a = rx[k][i].b = rg[k][i].a = rg[k][i].b = make_uint4(0, 0, 0, 0);
          if (h < now.last && sl.on[i]) {
            rx[k][i].load(in + (int64_t)h * p.dim * E, sl.ea[i], sl.eb[i]);
            rg[k][i].load(gin + (int64_t)h * p.dim * E, sl.ea[i], sl.eb[i]);
          }
        }
      }
      if (r0 == now.first) {
        angles<W, NS>(c, s, sl, p, at);
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int e = 0; e < W; ++e) s[i][e] = -s[i][e];  // the turn back
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int h = r0 + k * per + sub;
        if (r0 + k * per >= now.last) break;
        const bool live = h < now.last;
        float a[NS][W], b[NS][W], ga[NS][W], gb[NS][W], ss[2] = {0.f, 0.f}, dot[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          rx[k][i].get(a[i], b[i]);
          add_to<W>(ss, a[i], a[i]);
          add_to<W>(ss, b[i], b[i]);
        }
        const float ms = group_sum(ss[0] + ss[1], p.group) * p.inv_dim;
        const bool keep = at >= 0 && ms <= 3.402823466e38f && ms + p.eps > 0.f;
        const float r = keep ? rsqrtf(ms + p.eps) : 0.f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          rg[k][i].get(ga[i], gb[i]);
          turn<W>(ga[i], gb[i], c[i], s[i], p.interleaved);
          float wa[W], wb[W];
#pragma unroll
          for (int e = 0; e < W; ++e) wa[e] = wb[e] = 1.f;
          if (w && sl.on[i]) {
            load_cached<DT, W>(wa, w + sl.ea[i] * E);
            load_cached<DT, W>(wb, w + sl.eb[i] * E);
          }
          times<W>(a[i], r);
          times<W>(b[i], r);
          if (keep && live) {
            add_each<W>(acc[i][0], ga[i], a[i]);
            add_each<W>(acc[i][1], gb[i], b[i]);
          }
          times<W>(ga[i], wa);
          times<W>(gb[i], wb);
          add_to<W>(dot, ga[i], a[i]);
          add_to<W>(dot, gb[i], b[i]);
        }
        const float mean = group_sum(dot[0] + dot[1], p.group) * p.inv_dim;
        if (!live) continue;
        char* dx = out + (int64_t)h * p.dim * E;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          if (!sl.on[i]) continue;
          if (keep) {
            plus<W>(ga[i], a[i], -mean);
            plus<W>(gb[i], b[i], -mean);
            times<W>(ga[i], r);
            times<W>(gb[i], r);
          } else {
#pragma unroll
            for (int e = 0; e < W; ++e) ga[i][e] = gb[i][e] = 0.f;
          }
          store<DT, W>(dx + sl.ea[i] * E, ga[i]);
          store<DT, W>(dx + sl.eb[i] * E, gb[i]);
        }
      }
    }
  }
  if (p.ws == nullptr) return;
  put_aside(queries ? 0 : 1);
  if (queries) put_aside(1);  // (no keys: zeros)
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * p.dim; i += kThreads) {
    float v = 0.f;
    for (int wv = 0; wv < kThreads / 32; ++wv) v += part[wv * 2 * p.dim + i];
    p.ws[(int64_t)blockIdx.x * 2 * p.dim + i] = v;
  }
}

// The weights' gradients: column k of the `rows` sums, a warp a slice of the rows for 32
// columns, the slices in order.  Launched beside the kernel above, whose end it waits for (1999
// tokens, fp32, 16 + 4 heads of 64: 10.9 us in all; 12.0 as a launch after it).
template <int DT>
__global__ void __launch_bounds__(1024) rope_join_kernel(const float* ws, int rows, int dim,
                                                         char* dqw, char* dkw) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5, k = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float s = 0.f;
  if (k < 2 * dim) {
    int r = slice;
    for (; r + 128 < rows; r += 160) {
      float a[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) a[i] = __ldcs(ws + (int64_t)(r + 32 * i) * 2 * dim + k);
#pragma unroll
      for (int i = 0; i < 5; ++i) s += a[i];
    }
    for (; r < rows; r += 32) s += __ldcs(ws + (int64_t)r * 2 * dim + k);
  }
  part[slice][lane] = s;
  __syncthreads();
  if (slice > 0 || k >= 2 * dim) return;
  float t = part[0][lane];
  for (int i = 1; i < 32; ++i) t += part[i][lane];
  st_elem<DT>((k < dim ? dqw : dkw - (int64_t)dim * DType<DT>::E) + (int64_t)k * DType<DT>::E, t);
}

}  // namespace

template <int DT, int W>
static RopeKernels kernels_of(bool vec) {
  return vec ? RopeKernels{(const void*)rope_fwd_kernel<DT, W, 1, kFwdU>,
                           (const void*)rope_bwd_kernel<DT, W, 1, kBwdU>,
                           (const void*)rope_join_kernel<DT>, kThreads}
             : RopeKernels{(const void*)rope_fwd_kernel<DT, 1, 4, 1>,
                           (const void*)rope_bwd_kernel<DT, 1, 4, 1>,
                           (const void*)rope_join_kernel<DT>, kThreads};
}
RopeKernels rope_kernels(int dtype, bool vec) {
  return dtype == kF32 ? kernels_of<kF32, 4>(vec) : kernels_of<kBF16, 8>(vec);
}

}  // namespace rr
