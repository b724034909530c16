// k_packed.cu -- causal attention over packed sequences with grouped heads, and its
// gradient, for the types and head dimensions that the tensor-core kernels
// (k_packed_tc.cu) do not take: float32 and bf16, any head dimension up to 256 in whole
// 16-byte chunks.
//
// A warp owns one query row (forward, dq) or one key row of a key head (dk, dv).  It takes
// 32 positions of the other side at a time: first each lane the whole products of one
// position (s = q . k, backward also dO . v), then all lanes the D columns of the sums, 32
// positions one after the other.  Sums, weights and statistics are float32.
//   o = sum_j p_j v_j,  p_j = e^{s_j - lse};   delta = dO . o,  ds_j = p_j (dO . v_j - delta),
//   dq = scale sum_j ds_j k_j,  dk = scale sum_i ds_i q_i,  dv = sum_i p_i dO_i
// (the last two over the rows i that see the key, of every head of its group, in order).
#include <cstdint>

#include "rr_device.cuh"
#include "rr_kernels.h"

namespace rr {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// The sequence that holds token t: [begin, end) with begin <= t < end, or false.
__device__ __forceinline__ bool sequence_of(const PackedParams& p, int64_t t, int64_t& begin,
                                            int64_t& end) {
  int64_t lo = 0, hi = p.batch;  // the last b < batch with cu[b] <= t is in [lo - 1, hi)
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (__ldg(p.cu + mid) <= t) lo = mid + 1; else hi = mid;
  }
  if (lo == 0) return false;
  begin = max(__ldg(p.cu + lo - 1), 0);
  end = min((int64_t)__ldg(p.cu + lo), p.tokens);
  return t < end;
}

template <int DT>
__device__ __forceinline__ float dot(const float* a, const char* b, int dim) {
  constexpr int W = 16 / DType<DT>::E;
  float s = 0.f;
  for (int c = 0; c < dim; c += W) {
    const uint4 v = ld_chunk_cached(b + c * DType<DT>::E);
#pragma unroll
    for (int e = 0; e < W; ++e) s += a[c + e] * chunk_get<DT>(v, e);
  }
  return s;
}

template <int DT>
__device__ __forceinline__ const char* at(const char* base, int64_t t, int64_t stride, int head,
                                          int dim) {
  return base + (t * stride + (int64_t)head * dim) * DType<DT>::E;
}

// acc[i] += f row[lane + 32 i]
template <int DT>
__device__ __forceinline__ void axpy(float (&acc)[8], float f, const char* row, int dim, int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int d = lane + 32 * i;
    if (d < dim) acc[i] += f * ld_elem_cached<DT>(row + d * DType<DT>::E);
  }
}
template <int DT>
__device__ __forceinline__ void put(char* row, const float (&acc)[8], float f, int dim, int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int d = lane + 32 * i;
    if (d < dim) st_elem<DT>(row + d * DType<DT>::E, acc[i] * f);
  }
}

template <int DT>
__global__ void __launch_bounds__(32 * kWarps) packed_fwd_rows(const PackedParams p) {
  __shared__ float sq[kWarps][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t t = item / p.heads;
  const int h = (int)(item - t * p.heads), kv = h / (p.heads / p.kv_heads);
  int64_t begin, end;
  if (t >= p.tokens || !sequence_of(p, t, begin, end)) return;
  for (int d = lane; d < p.dim; d += 32)
    sq[warp][d] = ld_elem_cached<DT>(at<DT>(p.q, t, p.sq, h, p.dim) + d * DType<DT>::E);
  __syncwarp();
  float acc[8] = {}, m = -INFINITY, l = 0.f;
  for (int64_t j0 = begin; j0 <= t; j0 += 32) {
    const int64_t j = j0 + lane;
    float s = -INFINITY;
    if (j <= t) s = dot<DT>(sq[warp], at<DT>(p.k, j, p.sk, kv, p.dim), p.dim) * p.scale_log2;
    float mn = s;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
    mn = fmaxf(m, mn);
    const float ref = mn == -INFINITY ? 0.f : mn, f = ex2(m - ref), w = ex2(s - ref);
    l = l * f + warp_sum(w);
    m = mn;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] *= f;
    const int n = (int)min((int64_t)32, t - j0 + 1);
    for (int i = 0; i < n; ++i)
      axpy<DT>(acc, __shfl_sync(0xffffffffu, w, i), at<DT>(p.v, j0 + i, p.sv, kv, p.dim), p.dim,
               lane);
  }
  put<DT>(const_cast<char*>(at<DT>(p.o, t, p.so, h, p.dim)), acc, 1.f / l, p.dim, lane);
  if (p.lse && lane == 0) p.lse[(int64_t)h * p.tokens + t] = (m + __log2f(l)) * kLn2;
}

template <int DT>
__global__ void __launch_bounds__(32 * kWarps) packed_dq_rows(const PackedParams p) {
  __shared__ float sq[kWarps][256], sg[kWarps][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t t = item / p.heads;
  const int h = (int)(item - t * p.heads), kv = h / (p.heads / p.kv_heads);
  int64_t begin, end;
  if (t >= p.tokens || !sequence_of(p, t, begin, end)) return;
  float delta = 0.f;
  for (int d = lane; d < p.dim; d += 32) {
    sq[warp][d] = ld_elem_cached<DT>(at<DT>(p.q, t, p.sq, h, p.dim) + d * DType<DT>::E);
    sg[warp][d] = ld_elem_cached<DT>(at<DT>(p.dout, t, p.sdo, h, p.dim) + d * DType<DT>::E);
    delta += sg[warp][d] * ld_elem_cached<DT>(at<DT>(p.o, t, p.so, h, p.dim) + d * DType<DT>::E);
  }
  delta = warp_sum(delta);
  __syncwarp();
  const int64_t row = (int64_t)h * p.tokens + t;
  if (lane == 0) p.delta[row] = delta;
  const float lse = p.lse[row] * kLog2e;
  float acc[8] = {};
  for (int64_t j0 = begin; j0 <= t; j0 += 32) {
    const int64_t j = j0 + lane;
    float ds = 0.f;
    if (j <= t) {
      const float s = dot<DT>(sq[warp], at<DT>(p.k, j, p.sk, kv, p.dim), p.dim);
      const float dp = dot<DT>(sg[warp], at<DT>(p.v, j, p.sv, kv, p.dim), p.dim);
      ds = ex2(s * p.scale_log2 - lse) * (dp - delta);
    }
    const int n = (int)min((int64_t)32, t - j0 + 1);
    for (int i = 0; i < n; ++i)
      axpy<DT>(acc, __shfl_sync(0xffffffffu, ds, i), at<DT>(p.k, j0 + i, p.sk, kv, p.dim), p.dim,
               lane);
  }
  put<DT>(const_cast<char*>(at<DT>(p.dq, t, p.sdq, h, p.dim)), acc, p.scale, p.dim, lane);
}

template <int DT>
__global__ void __launch_bounds__(32 * kWarps) packed_dkv_rows(const PackedParams p) {
  __shared__ float sk[kWarps][256], sv[kWarps][256];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kWarps + warp;
  const int64_t t = item / p.kv_heads;
  const int kv = (int)(item - t * p.kv_heads), group = p.heads / p.kv_heads;
  int64_t begin, end;
  if (t >= p.tokens || !sequence_of(p, t, begin, end)) return;
  for (int d = lane; d < p.dim; d += 32) {
    sk[warp][d] = ld_elem_cached<DT>(at<DT>(p.k, t, p.sk, kv, p.dim) + d * DType<DT>::E);
    sv[warp][d] = ld_elem_cached<DT>(at<DT>(p.v, t, p.sv, kv, p.dim) + d * DType<DT>::E);
  }
  __syncwarp();
  float ak[8] = {}, av[8] = {};
  for (int h = kv * group; h < (kv + 1) * group; ++h)
    for (int64_t i0 = t; i0 < end; i0 += 32) {
      const int64_t i = i0 + lane;
      float w = 0.f, ds = 0.f;
      if (i < end) {
        const int64_t row = (int64_t)h * p.tokens + i;
        const float s = dot<DT>(sk[warp], at<DT>(p.q, i, p.sq, h, p.dim), p.dim);
        const float dp = dot<DT>(sv[warp], at<DT>(p.dout, i, p.sdo, h, p.dim), p.dim);
        w = ex2(s * p.scale_log2 - p.lse[row] * kLog2e);
        ds = w * (dp - p.delta[row]);
      }
      const int n = (int)min((int64_t)32, end - i0);
      for (int e = 0; e < n; ++e) {
        axpy<DT>(av, __shfl_sync(0xffffffffu, w, e), at<DT>(p.dout, i0 + e, p.sdo, h, p.dim),
                 p.dim, lane);
        axpy<DT>(ak, __shfl_sync(0xffffffffu, ds, e), at<DT>(p.q, i0 + e, p.sq, h, p.dim), p.dim,
                 lane);
      }
    }
  put<DT>(const_cast<char*>(at<DT>(p.dk, t, p.sdk, kv, p.dim)), ak, p.scale, p.dim, lane);
  put<DT>(const_cast<char*>(at<DT>(p.dv, t, p.sdv, kv, p.dim)), av, 1.f, p.dim, lane);
}

}  // namespace

PackedRowKernels packed_row_kernels(int dtype) {
  if (dtype == kF32)
    return PackedRowKernels{(const void*)packed_fwd_rows<kF32>, (const void*)packed_dq_rows<kF32>,
                            (const void*)packed_dkv_rows<kF32>, kWarps};
  return PackedRowKernels{(const void*)packed_fwd_rows<kBF16>, (const void*)packed_dq_rows<kBF16>,
                          (const void*)packed_dkv_rows<kBF16>, kWarps};
}

}  // namespace rr
