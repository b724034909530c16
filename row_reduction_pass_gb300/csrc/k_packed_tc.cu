// k_packed_tc.cu -- causal attention over packed sequences with grouped heads on the
// 5th-generation tensor cores (bf16, head dimension 64 or 128).
//
// Forward.  A block, one per SM, works on two tiles of 128 query rows at once that attend
// to the same keys (halves 0 and 1): two heads of a key head's group over the same tokens,
// or, where the group is odd, two neighbouring tiles of one head.  Key and value tiles of
// 128 tokens are loaded once for both.  Per half and key tile: S = Q K^T into TMEM, a
// softmax warpgroup of four warps (thread t owns row t, TMEM lane t) turns it into bf16
// weights in TMEM with the running maximum and sum of the online softmax, O += P V.
// While one half is in its softmax the tensor cores work for the other.
//   head_dim 128: a half's 256 TMEM columns are S (128), whose first half P overwrites, and
//     O (128); S of the next tile follows O += P V of this one.
//   head_dim 64: S (128), P (64) and O (64); S of the next tile as soon as S has been read.
// Roles: warps 0-3 and 4-7 the halves' softmax, warp 8 loads (TMA), warps 9 and 10 issue the
// halves' products.
//
// Work.  An item is a level of a sequence (a tile of 128 queries, or two where the group is
// odd) with one pair of a key head; its cost is the level.  Sequence lengths are known on the
// device only, so each block sorts the (at most 128) sequences by their length and finds its
// items in the list of all levels, longest first, that the blocks are dealt in a zigzag.
// More sequences are taken in their own order.
//
// A tile's rows beyond its sequence (the next one's, or past the buffer, which read as zero)
// are not stored, and keys beyond a row's own are masked in S.  Their V has weight 0, which a
// NaN or infinity there would turn into NaN: a row that ends with one is computed again from
// the keys that it sees (repair_row).
#include <algorithm>
#include <cstdint>

#include "rr_device.cuh"
#include "rr_kernels.h"
#include "rr_tc.cuh"

namespace rr {
namespace {

constexpr int kTile = 128;           // query rows and keys of a tile
constexpr int kBox = kTile * 128;    // bytes of 128 rows x 64 columns
constexpr int kSorted = 128;         // sequences that a block sorts

// TMA box [128 tokens x 1 head x 64 columns] at {column, head, token}.
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, int col, int head,
                                         int token, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(head), "r"(token), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void store_box(const CUtensorMap* map, const void* src, int col,
                                          int head, int token) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(col), "r"(head), "r"(token), "r"(smem_addr(src))
      : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void stores_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void stores_done() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// A block's items: entry u of the list of levels, longest first, with part p of `parts`.
struct Item {
  int beg, len;   // the sequence
  int level, part;
  bool ok;
};
struct Sequences {
  int2* seq;       // shared: (begin, length) of the live sequences, longest first
  const int* cu;
  int n, batch, tokens, rows, parts, entries;
  int lv[kSorted / 32];  // levels of sequences lane, lane + 32, ...
  bool sorted;

  __device__ __forceinline__ int2 bounds(int b) const {
    const int a = min(max(__ldg(cu + b), 0), tokens), e = min(max(__ldg(cu + b + 1), 0), tokens);
    return make_int2(a, max(e - a, 0));
  }
  // All threads of the block; `tmp` is shared room for kSorted int2.
  __device__ __forceinline__ void init(int2* s, int2* tmp, const PackedParams& p, int rows_,
                                       int parts_) {
    seq = s;
    cu = p.cu;
    batch = (int)p.batch;
    tokens = (int)p.tokens;
    rows = rows_;
    parts = parts_;
    sorted = batch <= kSorted;
    const int tid = threadIdx.x, lane = tid & 31;
    int2 mine = make_int2(0, 0);
    if (sorted && tid < batch) tmp[tid] = mine = bounds(tid);
    n = __syncthreads_count(mine.y > 0);
    if (sorted && mine.y > 0) {
      const int l = (mine.y + rows - 1) / rows;
      int at = 0;
      for (int b = 0; b < batch; ++b) {
        const int o = (tmp[b].y + rows - 1) / rows;
        at += o > l || (o == l && b < tid);
      }
      seq[at] = mine;
    }
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int k = 0; k < kSorted / 32; ++k) {
      const int b = lane + 32 * k;
      lv[k] = sorted && b < n ? (seq[b].y + rows - 1) / rows : 0;
      sum += lv[k];
    }
    // unsorted: entry floor(begin / rows) + b + level, some of which are none
    entries = sorted ? __reduce_add_sync(0xffffffffu, sum) : tokens / rows + batch;
  }
  // levels at or above l, over all sequences
  __device__ __forceinline__ int above(int l) const {
    int s = 0;
#pragma unroll
    for (int k = 0; k < kSorted / 32; ++k) s += max(lv[k] - l, 0);
    return __reduce_add_sync(0xffffffffu, s);
  }
  // The r-th item of this block (all lanes of a warp); more: whether r is within the list.
  __device__ __forceinline__ Item get(int r, bool& more) const {
    const int nb = (int)gridDim.x, me = (int)blockIdx.x;
    const int64_t i = (int64_t)r * nb + ((r & 1) ? nb - 1 - me : me);
    const int64_t u64 = i / parts;
    Item it{0, 0, 0, (int)(i - u64 * parts), false};
    more = u64 < entries;
    if (!more) return it;
    const int u = (int)u64;
    if (sorted) {
      int lo = 0, hi = (seq[0].y + rows - 1) / rows;  // above(lo) > u >= above(hi)
      int at_hi = 0;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1, f = above(mid);
        if (f > u) {
          lo = mid;
        } else {
          hi = mid;
          at_hi = f;
        }
      }
      const int2 s = seq[u - at_hi];
      it.beg = s.x, it.len = s.y, it.level = lo, it.ok = true;
    } else {
      int lo = 0, hi = batch - 1;  // the last sequence whose first entry is at or before u
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (bounds(mid).x / rows + mid <= u) lo = mid; else hi = mid - 1;
      }
      const int2 s = bounds(lo);
      it.beg = s.x, it.len = s.y, it.level = u - s.x / rows - lo;
      it.ok = it.level >= 0 && it.level * rows < it.len;
    }
    return it;
  }
};

template <int D>
struct Fwd {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBoxes * kBox;
  static constexpr int kOffK = 2 * kTileBytes, kOffV = 4 * kTileBytes;
  static constexpr int kOffStage = 6 * kTileBytes;       // 8 warps' output boxes
  static constexpr int kStage = 32 * 128;
  static constexpr int kOffBar = kOffStage + 8 * kStage;
  static constexpr int kOffSeq = kOffBar + 256;
  static constexpr int kSmem = kOffSeq + kSorted * 8 + 1024;
  static constexpr uint32_t kColP = D == 128 ? 0 : 128, kColO = 256 - D;
  static constexpr uint32_t kIdescS = attn_idesc(kTile, kTile, false);
  static constexpr uint32_t kIdescO = attn_idesc(kTile, D, true);
};

// Row t of head h again, in float32, from the keys that it sees: the warp's lanes take 32
// keys' scores, then all the D columns.  sq: shared room for D floats.
template <int D>
__device__ __noinline__ void repair_row(const PackedParams& p, int64_t begin, int64_t t, int h,
                                        float* sq) {
  const int lane = threadIdx.x & 31, kv = h / (p.heads / p.kv_heads);
  const char* q = p.q + (t * p.sq + (int64_t)h * D) * 2;
  __syncwarp();
  for (int d = lane; d < D; d += 32) sq[d] = ld_elem_cached<kBF16>(q + 2 * d);
  __syncwarp();
  float acc[D / 32] = {}, m = -INFINITY, l = 0.f;
  for (int64_t j0 = begin; j0 <= t; j0 += 32) {
    float s = -INFINITY;
    if (j0 + lane <= t) {
      const char* k = p.k + ((j0 + lane) * p.sk + (int64_t)kv * D) * 2;
      s = 0.f;
      for (int c = 0; c < D; c += 8) {
        const uint4 v = ld_chunk_cached(k + 2 * c);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += sq[c + e] * chunk_get<kBF16>(v, e);
      }
      s *= p.scale_log2;
    }
    float mn = s;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
    mn = fmaxf(m, mn);
    const float ref = mn == -INFINITY ? 0.f : mn, f = ex2(m - ref), w = ex2(s - ref);
    float sum = w;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    l = l * f + sum;
    m = mn;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] *= f;
    const int n = (int)min((int64_t)32, t - j0 + 1);
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const char* v = p.v + ((j0 + i) * p.sv + (int64_t)kv * D) * 2;
#pragma unroll
      for (int e = 0; e < D / 32; ++e)
        acc[e] += wi * ld_elem_cached<kBF16>(v + 2 * (lane + 32 * e));
    }
  }
  char* o = const_cast<char*>(p.o) + (t * p.so + (int64_t)h * D) * 2;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) st_elem<kBF16>(o + 2 * (lane + 32 * i), acc[i] / l);
}

// A half's query tile of an item: its first row in the sequence, head and key tiles (0: none).
struct Half {
  int row0, head, tiles;
};
__device__ __forceinline__ Half half_of(const Item& it, int h, int group, bool even) {
  Half x;
  const int pairs = even ? group / 2 : group;
  const int kv = it.part / pairs, pair = it.part - kv * pairs;
  const int tile = even ? it.level : 2 * it.level + h;
  x.head = kv * group + (even ? 2 * pair + h : pair);
  x.row0 = tile * kTile;
  x.tiles = it.ok && x.row0 < it.len ? tile + 1 : 0;
  return x;
}

template <int D>
__global__ void __launch_bounds__(352, 1)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to,
                      const PackedParams p) {
  using C = Fwd<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = p.heads / p.kv_heads;
  const bool even = group % 2 == 0;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* bar_q = bars;           // [half] Q landed
  uint64_t* bar_qfree = bars + 2;   // [half] the item's last S done
  uint64_t* bar_s = bars + 4;       // [half] S done
  uint64_t* bar_sfree = bars + 6;   // [half] S read (head_dim 64), 128 arrivals
  uint64_t* bar_p = bars + 8;       // [half] P written, 128 arrivals
  uint64_t* bar_o = bars + 10;      // [half] O += P V done
  uint64_t* bar_ofree = bars + 12;  // [half] O read, 128 arrivals
  uint64_t* bar_kfull = bars + 14;  // [stage]
  uint64_t* bar_vfull = bars + 16;
  uint64_t* bar_kempty = bars + 18; // [stage] both halves' S done
  uint64_t* bar_vempty = bars + 20; // [stage] both halves' O += P V done
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 22);

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tslot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 32 * 8) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_q[i], 1);
      mbar_init(&bar_qfree[i], 1);
      mbar_init(&bar_s[i], 1);
      mbar_init(&bar_sfree[i], 128);
      mbar_init(&bar_p[i], 128);
      mbar_init(&bar_o[i], 1);
      mbar_init(&bar_ofree[i], 128);
      mbar_init(&bar_kfull[i], 1);
      mbar_init(&bar_vfull[i], 1);
      mbar_init(&bar_kempty[i], 2);
      mbar_init(&bar_vempty[i], 2);
    }
    fence_mbar_init();
  }
  Sequences list;
  list.init(reinterpret_cast<int2*>(smem + C::kOffSeq), reinterpret_cast<int2*>(smem + C::kOffStage),
            p, even ? kTile : 2 * kTile, (even ? group / 2 : group) * p.kv_heads);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  bool dead = false, more;

  // A role whose wait gave up asks for nothing more, and what it has asked for ends before
  // the block does.
  if (warp == 8) {
    // ------------------------------------------------------------ loads
    int nk = 0, nv = 0, qn[2] = {0, 0};
    for (int r = 0;; ++r) {
      const Item it = list.get(r, more);
      if (!more) break;
      if (!it.ok || lane != 0) continue;
      const int kv = it.part / (even ? group / 2 : group);
      int n = 0;
      for (int h = 0; h < 2; ++h) {
        const Half x = half_of(it, h, group, even);
        if (x.tiles == 0) continue;
        n = max(n, x.tiles);
        if (qn[h] > 0) wait_spin(&bar_qfree[h], (uint32_t)((qn[h] - 1) & 1), dead, p.err);
        if (dead) break;
        ++qn[h];
        mbar_arrive_expect_tx(&bar_q[h], C::kTileBytes);
        for (int b = 0; b < C::kBoxes; ++b)
          load_box(smem + h * C::kTileBytes + b * kBox, &tq, 64 * b, x.head, it.beg + x.row0,
                   &bar_q[h]);
      }
      for (int t = 0; t < n; ++t) {
        const int s = nk & 1;
        const uint32_t ph = (uint32_t)(((nk >> 1) - 1) & 1);
        if (nk >= 2) wait_spin(&bar_kempty[s], ph, dead, p.err);
        if (dead) break;
        ++nk;
        mbar_arrive_expect_tx(&bar_kfull[s], C::kTileBytes);
        for (int b = 0; b < C::kBoxes; ++b)
          load_box(smem + C::kOffK + s * C::kTileBytes + b * kBox, &tk, 64 * b, kv,
                   it.beg + t * kTile, &bar_kfull[s]);
        if (nv >= 2) wait_spin(&bar_vempty[s], ph, dead, p.err);
        if (dead) break;
        ++nv;
        mbar_arrive_expect_tx(&bar_vfull[s], C::kTileBytes);
        for (int b = 0; b < C::kBoxes; ++b)
          load_box(smem + C::kOffV + s * C::kTileBytes + b * kBox, &tv, 64 * b, kv,
                   it.beg + t * kTile, &bar_vfull[s]);
      }
    }
    for (int n = max(nk - 2, 0); n < nk; ++n)
      mbar_wait_bounded(&bar_kfull[n & 1], (uint32_t)((n >> 1) & 1), p.err);
    for (int n = max(nv - 2, 0); n < nv; ++n)
      mbar_wait_bounded(&bar_vfull[n & 1], (uint32_t)((n >> 1) & 1), p.err);
    for (int h = 0; h < 2; ++h)
      if (qn[h] > 0) mbar_wait_bounded(&bar_q[h], (uint32_t)((qn[h] - 1) & 1), p.err);
  } else if (warp >= 9) {
    // --------------------------------------------------- a half's products
    const int h = warp - 9;
    const uint32_t tm = tmem + 256u * h;
    const uint32_t q_addr = smem_addr(smem + h * C::kTileBytes);
    int kc = 0, ns = 0, no = 0, items = 0;  // key tiles loaded, products issued, items
    auto stage = [&](int t) { return (kc + t) & 1; };
    auto phase = [&](int t) { return (uint32_t)(((kc + t) >> 1) & 1); };
    auto issue_s = [&](int t, bool last) {
      const uint32_t k_addr = smem_addr(smem + C::kOffK + stage(t) * C::kTileBytes);
      wait_spin(&bar_kfull[stage(t)], phase(t), dead, p.err);
      if (dead) return;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (uint32_t)((kk >> 2) * kBox + (kk & 3) * 32);
        mma_ss(tm, sw128_desc(q_addr + off, 16, 1024), sw128_desc(k_addr + off, 16, 1024),
               C::kIdescS, kk > 0 ? 1u : 0u);
      }
      ++ns;
      mma_commit(&bar_s[h]);
      mma_commit(&bar_kempty[stage(t)]);
      if (last) mma_commit(&bar_qfree[h]);
    };
    auto issue_pv = [&](int t) {
      const uint32_t v_addr = smem_addr(smem + C::kOffV + stage(t) * C::kTileBytes);
      wait_spin(&bar_vfull[stage(t)], phase(t), dead, p.err);
      if (dead) return;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < kTile / 16; ++kk)
        mma_ts(tm + C::kColO, tm + C::kColP + 8 * kk, sw128_desc(v_addr + kk * 2048, kBox, 1024),
               C::kIdescO, (t > 0 || kk > 0) ? 1u : 0u);
      ++no;
      mma_commit(&bar_o[h]);
      mma_commit(&bar_vempty[stage(t)]);
    };
    for (int r = 0;; ++r) {
      const Item it = list.get(r, more);
      if (!more) break;
      if (!it.ok) continue;
      const int nh = half_of(it, h, group, even).tiles;
      const int n = max(nh, half_of(it, 1 - h, group, even).tiles);
      if (lane == 0) {
        if (nh > 0) {
          wait_spin(&bar_q[h], (uint32_t)(items & 1), dead, p.err);
          if (D == 64) {
            if (ns > 0) wait_spin(&bar_sfree[h], (uint32_t)((ns - 1) & 1), dead, p.err);
            issue_s(0, nh == 1);
          }
        }
        for (int t = 0; t < nh && !dead; ++t) {
          if (D == 128) {
            // P of the tile before stands where S goes
            if (no > 0) wait_spin(&bar_o[h], (uint32_t)((no - 1) & 1), dead, p.err);
            issue_s(t, t == nh - 1);
          } else if (t + 1 < nh) {
            wait_spin(&bar_sfree[h], (uint32_t)(no & 1), dead, p.err);
            issue_s(t + 1, t + 1 == nh - 1);
          }
          wait_spin(&bar_p[h], (uint32_t)(no & 1), dead, p.err);
          if (t == 0 && items > 0)
            wait_spin(&bar_ofree[h], (uint32_t)((items - 1) & 1), dead, p.err);
          issue_pv(t);
        }
        // the other half's tiles: a stage is given back once it has landed, so that its
        // barrier's phases keep their order
        for (int t = nh; t < n && !dead; ++t) {
          wait_spin(&bar_kfull[stage(t)], phase(t), dead, p.err);
          if (!dead) mbar_arrive(&bar_kempty[stage(t)]);
          wait_spin(&bar_vfull[stage(t)], phase(t), dead, p.err);
          if (!dead) mbar_arrive(&bar_vempty[stage(t)]);
        }
      }
      kc += n;
      items += nh > 0;
    }
    if (ns > 0) mbar_wait_bounded(&bar_s[h], (uint32_t)((ns - 1) & 1), p.err);
    if (no > 0) mbar_wait_bounded(&bar_o[h], (uint32_t)((no - 1) & 1), p.err);
  } else {
    // ------------------------------------------------- a half's softmax
    const int h = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 256u * h + lanes, tP = tS + C::kColP, tO = tS + C::kColO;
    const float sc = p.scale_log2;
    unsigned char* box = smem + C::kOffStage + warp * C::kStage;
    int th = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!dead) dead = !mbar_wait_bounded(bar, parity, p.err);
    };
    for (int r = 0;; ++r) {
      const Item it = list.get(r, more);
      if (!more) break;
      const Half x = half_of(it, h, group, even);
      if (x.tiles == 0) continue;
      float m = -INFINITY, l = 0.f;
      for (int t = 0; t < x.tiles; ++t, ++th) {
        wait(&bar_s[h], (uint32_t)(th & 1));
        tc_fence_after();
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_nowait(tS + 32 * c, v[c]);
        tmem_ld_wait();
        if (D == 64) {
          tc_fence_before();
          mbar_arrive(&bar_sfree[h]);
        }
        if (t == x.tiles - 1) {  // the diagonal: keys after the row
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i > row) v[c][i] = __float_as_uint(-INFINITY);
        }
        float mx[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) mx[i & 7] = fmaxf(mx[i & 7], __uint_as_float(v[c][i]));
        const float mx0 = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const float mx1 = fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]));
        // m moves only when the tile's maximum exceeds it by more than 2^8 (P stays below
        // 2^8 otherwise, exact in its sum's float32), so O is rarely rescaled
        const float mt = fmaxf(mx0, mx1) * sc;
        const float mn = mt > m + 8.f ? mt : m;
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float alpha = ex2(m - ref);
        float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
        uint32_t pk[4][16];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            float t0, t1, t2, t3;
            fma2(t0, t1, __uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1]), sc, sc, -ref, -ref);
            fma2(t2, t3, __uint_as_float(v[c][i + 2]), __uint_as_float(v[c][i + 3]), sc, sc, -ref,
                 -ref);
            const float p0 = ex2(t0), p1 = ex2(t1), p2 = ex2(t2), p3 = ex2(t3);
            add2(l0, l1, l0, l1, p0, p1);
            add2(l2, l3, l2, l3, p2, p3);
            pk[c][i >> 1] = pack_bf16(p0, p1);
            pk[c][(i >> 1) + 1] = pack_bf16(p2, p3);
          }
        l = l * alpha + ((l0 + l1) + (l2 + l3));
        m = mn;
        if (D == 64 && th > 0) {  // the product before is done with P and O
          wait(&bar_o[h], (uint32_t)((th - 1) & 1));
          tc_fence_after();
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_st16(tP + 16 * c, pk[c]);
        if (t > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          uint32_t o[D / 32][32];
#pragma unroll
          for (int c = 0; c < D / 32; ++c) tmem_ld32_nowait(tO + 32 * c, o[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float a0, a1;
              mul2(a0, a1, __uint_as_float(o[c][i]), __uint_as_float(o[c][i + 1]), alpha, alpha);
              o[c][i] = __float_as_uint(a0);
              o[c][i + 1] = __float_as_uint(a1);
            }
            tmem_st32(tO + 32 * c, o[c]);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar_p[h]);
      }
      // O / l and lse
      wait(&bar_o[h], (uint32_t)((th - 1) & 1));
      tc_fence_after();
      uint32_t o[D / 32][32];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) tmem_ld32_nowait(tO + 32 * c, o[c]);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(&bar_ofree[h]);
      const float inv = 1.f / l;
      const bool live = x.row0 + row < it.len;
      const int64_t at = (int64_t)it.beg + x.row0 + row;
      if (p.lse != nullptr && live) p.lse[(int64_t)x.head * p.tokens + at] = (m + __log2f(l)) * kLn2;
      float f0 = 0.f, f1 = 0.f;  // NaN if any value is NaN or infinite
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int i = 0; i < 32; i += 2)
          fma2(f0, f1, __uint_as_float(o[c][i]), __uint_as_float(o[c][i + 1]), 0.f, 0.f, f0, f1);
      const bool fine = f0 + f1 == 0.f;
      const bool whole = __all_sync(0xffffffffu, live && fine);
      char* out = const_cast<char*>(p.o) + (at * p.so + (int64_t)x.head * D) * 2;
#pragma unroll
      for (int b = 0; b < C::kBoxes; ++b) {
        if (whole) {
          if (lane == 0) stores_read();  // the box's last store has read it
          __syncwarp();
        }
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            const uint32_t* oc = o[2 * b + c2];
            const uint4 q4 = make_uint4(
                pack_bf16(__uint_as_float(oc[i]) * inv, __uint_as_float(oc[i + 1]) * inv),
                pack_bf16(__uint_as_float(oc[i + 2]) * inv, __uint_as_float(oc[i + 3]) * inv),
                pack_bf16(__uint_as_float(oc[i + 4]) * inv, __uint_as_float(oc[i + 5]) * inv),
                pack_bf16(__uint_as_float(oc[i + 6]) * inv, __uint_as_float(oc[i + 7]) * inv));
            const int ch = 4 * c2 + (i >> 3);  // 16-byte chunk of the 128-byte row
            if (whole)
              *reinterpret_cast<uint4*>(box + lane * 128 + ((ch ^ (lane & 7)) << 4)) = q4;
            else if (live && fine)
              *reinterpret_cast<uint4*>(out + 128 * b + 16 * ch) = q4;
          }
        if (whole) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) store_box(&to, box, 64 * b, x.head, (int)at);
        }
      }
      uint32_t broken = __ballot_sync(0xffffffffu, live && !fine);
      if (broken) {
        if (lane == 0) stores_read();
        __syncwarp();
        while (broken) {
          const int who = __ffs(broken) - 1;
          broken &= broken - 1;
          repair_row<D>(p, it.beg, __shfl_sync(0xffffffffu, at, who), x.head,
                        reinterpret_cast<float*>(box));
        }
      }
    }
    if (lane == 0) stores_done();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
}

// [tokens][heads][d] bf16, tokens `stride` elements apart, in boxes of `rows` tokens x 1 head
// x 64 columns, 128-byte swizzled.
bool encode_map(CUtensorMap* map, const char* base, int64_t tokens, int heads, int d,
                int64_t stride, int rows) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows}, es[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<char*>(base), dims, strides,
                box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

}  // namespace

PackedTcKernels packed_tc_kernels(int d) {
  if (d == 64) return PackedTcKernels{(const void*)packed_fwd_kernel<64>, Fwd<64>::kSmem};
  if (d == 128) return PackedTcKernels{(const void*)packed_fwd_kernel<128>, Fwd<128>::kSmem};
  return PackedTcKernels{nullptr, 0};
}

const char* packed_tc_fwd_launch(const PackedParams& p, int sms, cudaStream_t stream) {
  const PackedTcKernels k = packed_tc_kernels(p.dim);
  CUtensorMap maps[4];
  if (!encode_map(&maps[0], p.q, p.tokens, p.heads, p.dim, p.sq, kTile) ||
      !encode_map(&maps[1], p.k, p.tokens, p.kv_heads, p.dim, p.sk, kTile) ||
      !encode_map(&maps[2], p.v, p.tokens, p.kv_heads, p.dim, p.sv, kTile) ||
      !encode_map(&maps[3], p.o, p.tokens, p.heads, p.dim, p.so, 32))
    return "tensor map encoding failed";
  const int group = p.heads / p.kv_heads;
  const int64_t rows = group % 2 == 0 ? kTile : 2 * kTile;
  const int64_t parts = (int64_t)(group % 2 == 0 ? group / 2 : group) * p.kv_heads;
  const int64_t items = (p.tokens / rows + p.batch) * parts;
  PackedParams pc = p;
  void* args[] = {&maps[0], &maps[1], &maps[2], &maps[3], &pc};
  if (cudaLaunchKernel(k.fwd, dim3((unsigned)std::min<int64_t>(sms, items)), dim3(352), args,
                       (size_t)k.fwd_smem, stream) != cudaSuccess)
    return "launch failed";
  return nullptr;
}

}  // namespace rr
