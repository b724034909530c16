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
// M = sum t + tt.  Zt is summed over the unlisted columns themselves: Z less
// the listed terms would lose every digit when the list holds nearly all of
// the student's mass.
//
// A bit filter of up to 2^16 bits in shared memory holds (column mod its size)
// of the listed columns; a column whose bit is clear is unlisted, one whose bit
// is set is looked up in the list (only rows longer than the filter ever find
// it is not there).  Listed columns are stored again after the row's sweep, by
// the one thread whose entry is the first with that column.
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

// One block per row, single-element accesses: any alignment, any length.
template <int DT>
__global__ void __launch_bounds__(kDistT) distill_rows_kernel(const DistillParams p) {
  constexpr int E = DType<DT>::E;
  extern __shared__ __align__(16) unsigned char smem[];
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
        any = 1;
        vm = fmaxf(vm, v);
        tx[i] = ld_elem<DT>(x + (int64_t)j * E);
        const uint32_t b = (uint32_t)j & fmask;
        if (atomicOr(&filter[b >> 5], 1u << (b & 31)) & (1u << (b & 31))) s_dup = 1;
      }
    }
    any = __syncthreads_or(any);
    vm = block_max(vm, red);
    const bool live = any && (p.tail || vm != -INFINITY);
    // the row's maximum and sums (online, per thread, then merged)
    float m = -INFINITY, d = 0.f, dt = 0.f;
    if (live) {
      for (int64_t j = tid; j < p.cols; j += kDistT) {
        const float v = ld_elem<DT>(x + j * E);
        if (v > m) {
          const float a = ex2((m - v) * p.c);
          d *= a;
          dt *= a;
          m = v;
        }
        const float e = v == -INFINITY ? 0.f : ex2((v - m) * p.c);
        d += e;
        if (p.tail) {
          const uint32_t b = (uint32_t)j & fmask;
          bool listed = (filter[b >> 5] >> (b & 31)) & 1;
          if (listed && p.filter_bits < p.cols) {
            listed = false;
            for (int i = 0; i < p.k; ++i) listed = listed || tidx[i] == (int)j;
          }
          if (!listed) dt += e;
        }
      }
    }
    const float M = block_max(m, red);
    const float a = m == -INFINITY ? 0.f : ex2((m - M) * p.c);
    const float Z = block_sum(d * a, red);
    const float Zt = p.tail ? block_sum(dt * a, red) : 0.f;
    const float g = p.temperature * (p.grad != nullptr ? p.grad[r] : 1.f);
    if (!live || M == -INFINITY) {  // no teacher, or nothing to learn from: zeros
      if (tid == 0) p.loss[r] = 0.f;
      if (y != nullptr)
        for (int64_t j = tid; j < p.cols; j += kDistT) st_elem<DT>(y + j * E, 0.f);
    } else {
      // t_k and the loss
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
        if (t > 0.f) l += t * (lt - ((tx[i] - M) * p.inv_t - lnZ));
        else if (t != t) l = t;
        st += t;
        tval[i] = t;
      }
      l = block_sum(l, red);
      float mass = 1.f, tt = 0.f;
      if (p.tail) {
        st = block_sum(st, red);
        tt = Zt > 0.f ? fmaxf(1.f - st, 0.f) : 0.f;
        mass = st + tt;
        if (tt > 0.f) l += tt * (logf(tt) - (logf(Zt) - lnZ));
      }
      if (tid == 0) p.loss[r] = p.temperature * p.temperature * l;
      if (y != nullptr) {
        const float A = g * (mass / Z), B = tt > 0.f ? g * (tt / Zt) : 0.f;
        for (int64_t j = tid; j < p.cols; j += kDistT) {
          const float v = ld_elem<DT>(x + j * E);
          const float e = v == -INFINITY ? 0.f : ex2((v - M) * p.c);
          st_elem<DT>(y + j * E, e * (A - B));
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

}  // namespace

DistillKernel distill_kernel(int dtype) {
  return {dtype == kBF16 ? (const void*)distill_rows_kernel<kBF16>
                         : (const void*)distill_rows_kernel<kF32>,
          kDistT};
}

}  // namespace rr
