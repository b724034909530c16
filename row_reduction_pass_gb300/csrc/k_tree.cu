// k_tree.cu -- attention of a tree of new tokens over a paged cache, any page
// size: one warp per query row, online softmax over its keys (the fallback for
// page sizes that the tensor-core kernel cannot tile).
#include <cstdint>

#include "rr_device.cuh"
#include "rr_kernels.h"

namespace rr {
namespace {

constexpr int kTreeT = 128;

template <int D>
__global__ void __launch_bounds__(kTreeT) tree_rows_kernel_t(const TreeParams p) {
  constexpr int C = D / 32;  // values a lane holds of the row
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (kTreeT / 32) + (threadIdx.x >> 5);
  if (row >= p.batch * p.nodes * p.heads) return;
  const int h = (int)(row % p.heads);
  const int i = (int)(row / p.heads % p.nodes);
  const int64_t b = row / p.heads / p.nodes;
  const int kvh = h / (p.heads / p.kv_heads);
  // lane w holds word w of the bits of the nodes that node i sees
  uint32_t bits = 0;
  bool present = true;
  if (p.parents != nullptr) {
    const int32_t* par = p.parents + b * p.nodes;
    for (int a = i; a >= 0;) {
      if ((a >> 5) == lane) bits |= 1u << (a & 31);
      const int up = par[a];
      if (up < -1 || up >= a) present = false;
      if (!present) break;
      a = up;
    }
  }
  float q[C], o[C];
  const char* qp = p.q + row * D * 2 + lane * C * 2;
#pragma unroll
  for (int t = 0; t < C; ++t) {
    q[t] = ld_elem<kBF16>(qp + 2 * t);
    o[t] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int64_t ctx = max(p.length[b], 0);
  const int64_t end =
      present ? min(ctx + (p.parents != nullptr ? p.nodes : i + 1), p.width * p.page) : 0;
  for (int64_t pos = 0; pos < end; ++pos) {
    if (pos >= ctx && p.parents != nullptr) {
      const int j = (int)(pos - ctx);
      if (!((__shfl_sync(0xffffffffu, bits, j >> 5) >> (j & 31)) & 1)) continue;
    }
    const int64_t page = p.table[b * p.width + pos / p.page];
    if (page < 0 || page >= p.pages) continue;
    const int64_t at = (((page * p.page + pos % p.page) * p.kv_heads + kvh) * D + lane * C) * 2;
    float s = 0.f;
#pragma unroll
    for (int t = 0; t < C; ++t) s = fmaf(q[t], ld_elem_cached<kBF16>(p.k + at + 2 * t), s);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s);
    const float a = mn == -INFINITY ? 1.f : ex2(m - mn), w = mn == -INFINITY ? 0.f : ex2(s - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int t = 0; t < C; ++t)
      o[t] = fmaf(w, ld_elem_cached<kBF16>(p.v + at + 2 * t), o[t] * a);
  }
  char* op = p.o + row * D * 2 + lane * C * 2;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int t = 0; t < C; ++t) st_elem<kBF16>(op + 2 * t, o[t] * inv);
  if (lane == 0 && p.lse != nullptr)
    p.lse[row] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

}  // namespace

const void* tree_rows_kernel(int d) {
  return d == 64    ? (const void*)tree_rows_kernel_t<64>
         : d == 128 ? (const void*)tree_rows_kernel_t<128>
                    : nullptr;
}

}  // namespace rr
