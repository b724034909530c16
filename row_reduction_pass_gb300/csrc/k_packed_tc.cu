// k_packed_tc.cu -- causal attention over packed sequences with grouped heads on the
// 5th-generation tensor cores (bf16, head dimension 64 or 128).
//
// Forward.  A block, one per SM, works on one tile of 128 query rows of a head at a time:
// S = Q K^T of a key tile into one of three TMEM buffers, eight softmax warps (two threads a
// row, 64 keys each, which trade their maxima) turn it into bf16 weights in the same buffer
// with the running maximum and sum of the online softmax, O += P V.  With S two tiles ahead
// the softmax always finds its next tile, and the tensor cores have two products that do not
// depend on each other: a product of 128 x 128 x 16 takes 85 to 130 cycles alone and 66 beside
// another.  Sequences of 5117, 0, 1 and 4077 tokens, 32 heads on 8, head_dim 128: 247 us, 1420
// TFLOP/s; head_dim 64 243.  (Two tiles of 128 rows a block, which share the loaded keys but leave TMEM for one S
// each, took 384 us, S, softmax and O += P V one after the other; with their scores in two
// buffers of 64 keys 344 us: an S of 64 keys takes as long as one of 128.)
//   TMEM: S (3 x 128 columns, P over the first half of each half) and O (D columns).
// Roles: warps 0-7 softmax (two to a quarter of the lanes), warp 8 loads Q and K (TMA), warp 11
// loads V, warps 9 and 10 issue S and O += P V.
//
// Work.  An item is a level of a sequence (a tile of 128 queries) with one head; its cost is the
// level.  Sequence lengths are known on the device only, so each block sorts the (at most 128 live)
// sequences by their length and finds its items in the list of all levels, longest first, that
// the blocks are dealt in a zigzag.  More are taken in their own order, each item found by a
// search of the bounds in global memory: 128 sequences of 50 tokens 79 us, with one of one token
// more 110 (gradient 265, 310); of 8 to 1200 tokens 261 and 325 (904, 1320); 120 of 60 before 8 of
// 3000 558 and 597 (2046, 2259); 32 heads on 8, head_dim 128, flushed caches.  Batches of up to 128
// sequences have kernels of their own, without that search (247 instead of 253 us above).  Batches
// padded with empty ones: the live ones among up to kLooked are gathered and sorted (10 of 200
// tokens 26 us, with 1000 empty ones 30, with 4000 34; by skipping them 37 to 42 and 38 to 48, with
// 16000 40 to 56), else a lookup that finds none goes on over half or more of those that follow
// (60000: 42 to 56; one lookup each: 16000).
//
// A tile's rows beyond its sequence (the next one's, or past the buffer, which read as zero)
// are not stored, and keys beyond a row's own are masked in S.  Their V has weight 0, which a
// NaN or infinity there would turn into NaN.  V's rows behind a sequence are set to zero in shared
// memory before their product.  Those of the sequence's own later tokens are not looked at
// (testing the one tile an item that has some took the long prompts from 255 to 270 us or more):
// a block notes the items in which a row ended as NaN or infinite, and when all its roles have
// ended it reads their last tiles of V and computes the rows again that an unseen value reached
// (repair_items).  A value that a row does see stays, and costs the reading of that tile.
#include <algorithm>
#include <cstdint>

#include "rr_device.cuh"
#include "rr_kernels.h"
#include "rr_tc.cuh"

namespace rr {
namespace {

constexpr int kTile = 128;           // query rows and keys of a tile
constexpr int kBox = kTile * 128;    // bytes of 128 rows x 64 columns
constexpr int kSorted = 128;         // live sequences that a block sorts
constexpr int kLooked = 8192;        // sequences among which it looks for them

// TMA box [128 tokens x 1 head x 64 columns] at {column, head, token}.
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* map, int col, int head,
                                         int token, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(head), "r"(token), "r"(smem_addr(bar))
      : "memory");
}
// The same box on its way into L2.
__device__ __forceinline__ void prefetch_box(const CUtensorMap* map, int col, int head,
                                             int token) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(col), "r"(head), "r"(token)
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
// kMany: more than kSorted sequences, some of which may be empty.
template <bool kMany>
struct Sequences {
  int2* seq;       // shared: (begin, length) of the live sequences, longest first
  const int* cu;
  int n, batch, tokens, rows, parts, entries, me;
  int lv[kSorted / 32];  // levels of sequences lane, lane + 32, ...
  bool sorted_;

  __device__ __forceinline__ bool sorted() const { return !kMany || sorted_; }
  __device__ __forceinline__ int2 bounds(int b) const {
    const int a = min(max(__ldg(cu + b), 0), tokens), e = min(max(__ldg(cu + b + 1), 0), tokens);
    return make_int2(a, max(e - a, 0));
  }
  // All threads of the block; `tmp` is shared room for kSorted int2 and a word a warp.
  __device__ __forceinline__ void init(int2* s, int2* tmp, const PackedParams& p, int rows_,
                                       int parts_) {
    seq = s;
    cu = p.cu;
    batch = (int)p.batch;
    tokens = (int)p.tokens;
    rows = rows_;
    parts = parts_;
    me = (int)blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31;
    int2 mine = make_int2(0, 0);
    int room = batch;  // of tmp
    if constexpr (!kMany) {
      if (tid < batch) tmp[tid] = mine = bounds(tid);
      n = __syncthreads_count(mine.y > 0);
    } else if (batch <= kLooked) {  // the live ones, in order, as long as there is room
      int* counts = reinterpret_cast<int*>(tmp + kSorted);
      n = 0;
      for (int b0 = 0; b0 < batch && n <= kSorted; b0 += (int)blockDim.x) {
        const int2 s = b0 + tid < batch ? bounds(b0 + tid) : make_int2(0, 0);
        const uint32_t live = __ballot_sync(0xffffffffu, s.y > 0);
        if (lane == 0) counts[tid >> 5] = __popc(live);
        __syncthreads();
        int at = n + __popc(live & ((1u << lane) - 1u));
        for (int w = 0; w < (int)blockDim.x / 32; ++w) {
          const int c = counts[w];
          at += w < tid >> 5 ? c : 0;
          n += c;
        }
        if (s.y > 0 && at < kSorted) tmp[at] = s;
        __syncthreads();
      }
      room = n;
      if (tid < min(n, kSorted)) mine = tmp[tid];
    } else {
      n = kSorted + 1;
    }
    sorted_ = n <= kSorted;
    if (sorted() && mine.y > 0) {
      const int l = (mine.y + rows - 1) / rows;
      int at = 0;
      for (int b = 0; b < room; ++b) {
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
      lv[k] = sorted() && b < n ? (seq[b].y + rows - 1) / rows : 0;
      sum += lv[k];
    }
    // unsorted: entry floor(begin / rows) + b + level, some of which are none
    // (not more than 2^31 items, which 32 bits count: of bounds that decrease there could be)
    entries = sorted() ? (int)min((uint32_t)__reduce_add_sync(0xffffffffu, sum),
                                  0x80000000u / (uint32_t)p.heads)
                       : tokens / rows + batch;
  }
  // levels at or above l, over all sequences
  __device__ __forceinline__ int above(int l) const {
    int s = 0;
#pragma unroll
    for (int k = 0; k < kSorted / 32; ++k) s += max(lv[k] - l, 0);
    return __reduce_add_sync(0xffffffffu, s);
  }
  // The r-th item of this block (all lanes of a warp); more: whether r is within the list.  Where it
  // is none (unsorted only), the next one is not before place `part`.
  __device__ __forceinline__ Item get(int r, bool& more) const {
    const uint32_t nb = gridDim.x, i = r * nb + ((r & 1) ? nb - 1 - me : me);
    const int u = (int)(i / (uint32_t)parts);
    Item it{0, 0, 0, (int)(i - (uint32_t)u * parts), false};
    more = u < entries;
    if (!more) return it;
    if (sorted()) {
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
      if (!it.ok) {
        // none: on over half or more of the empty sequences that follow (those before a bound that
        // is this one's end), a lane looking 2^lane of them ahead
        const int b = min(lo + 1 + (1 << min((int)threadIdx.x & 31, 21)), batch);  // (batch <= 2^20)
        const bool same = min(max(__ldg(cu + b), 0), tokens) <= s.x + s.y;
        const int far = __popc(__ballot_sync(0xffffffffu, same));
        const int next = min(lo + 1 + (far ? 1 << min(far - 1, 21) : 0), batch);
        it.part = (int)((uint32_t)((s.x + s.y) / rows + next) * parts / nb);
      }
    }
    return it;
  }
};

// A block's items that have a row which is not finite: a bit for each of the first kFlagged - 1,
// one for all others.  flags[kFlagged / 32]: whether there are any.
constexpr int kFlagged = 4096;

template <int D>
struct Fwd {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBoxes * kBox;       // Q, then two stages of K and of V
  static constexpr int kOffK = kTileBytes, kOffV = 3 * kTileBytes;
  static constexpr int kOffStage = 5 * kTileBytes;       // 8 warps' output boxes
  static constexpr int kStage = 32 * 128;
  static constexpr int kOffTrade = kOffStage + 8 * kStage;  // [2][half][128] floats
  static constexpr int kOffBar = kOffTrade + 2048;
  static constexpr int kOffSeq = kOffBar + 256;
  static constexpr int kOffFlags = kOffSeq + kSorted * 8;
  static constexpr int kSmem = kOffFlags + kFlagged / 8 + 16 + 1024;
  static constexpr uint32_t kColO = 384;
  static constexpr uint32_t kIdescS = attn_idesc(kTile, kTile, false);
  static constexpr uint32_t kIdescO = attn_idesc(kTile, D, true);
};

// 64 columns of a warp's 32 rows (lane = row, lo and hi 32 columns each) times f as bf16: as
// one TMA store of whole lines from `box` where every row is stored, else row by row.
__device__ __forceinline__ void put_box(const uint32_t (&lo)[32], const uint32_t (&hi)[32], float f,
                                        unsigned char* box, const CUtensorMap* map, int col,
                                        int head, int token, char* out, bool whole, bool mine) {
  const int lane = threadIdx.x & 31;
  if (whole) {
    if (lane == 0) stores_read();  // the box's last store has read it
    __syncwarp();
  }
#pragma unroll
  for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
    for (int i = 0; i < 32; i += 8) {
      const uint32_t* oc = c2 ? hi : lo;
      const uint4 q4 = make_uint4(
          pack_bf16(__uint_as_float(oc[i]) * f, __uint_as_float(oc[i + 1]) * f),
          pack_bf16(__uint_as_float(oc[i + 2]) * f, __uint_as_float(oc[i + 3]) * f),
          pack_bf16(__uint_as_float(oc[i + 4]) * f, __uint_as_float(oc[i + 5]) * f),
          pack_bf16(__uint_as_float(oc[i + 6]) * f, __uint_as_float(oc[i + 7]) * f));
      const int ch = 4 * c2 + (i >> 3);  // 16-byte chunk of the 128-byte row
      if (whole)
        *reinterpret_cast<uint4*>(box + lane * 128 + ((ch ^ (lane & 7)) << 4)) = q4;
      else if (mine)
        *reinterpret_cast<uint4*>(out + 16 * ch) = q4;
    }
  if (whole) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) store_box(map, box, col, head, token);
  }
}

// 64 columns of a warp's 32 rows (lane = row, lo and hi 32 columns each) times f as bf16, for
// the rows of `rows` (a bit each).  Eight lanes trade their 16-byte chunks, so that each of
// them stores one chunk of eight rows and a store covers whole lines of 128 bytes.  out: this
// column of the warp's first row, rows `stride` bytes apart.
__device__ __forceinline__ void put_rows(const uint32_t (&lo)[32], const uint32_t (&hi)[32],
                                         float f, char* out, int64_t stride, uint32_t rows) {
  const int lane = threadIdx.x & 31, at = lane & 7;
  uint32_t x[8][4];
#pragma unroll
  for (int c = 0; c < 8; ++c)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t* o = (c < 4 ? lo : hi) + 8 * (c & 3) + 2 * k;
      x[c][k] = pack_bf16(__uint_as_float(o[0]) * f, __uint_as_float(o[1]) * f);
    }
#pragma unroll
  for (int bit = 1; bit < 8; bit *= 2)
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if ((c & bit) == 0)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool up = (at & bit) != 0;
          const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? x[c][k] : x[c | bit][k], bit);
          (up ? x[c][k] : x[c | bit][k]) = got;
        }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const int row = (lane & ~7) + c;
    if (rows >> row & 1)
      *reinterpret_cast<uint4*>(out + row * stride + 16 * at) =
          make_uint4(x[c][0], x[c][1], x[c][2], x[c][3]);
  }
}

// Zeros in `bytes` of shared memory, by one thread (visible to later tensor products of it).
__device__ __forceinline__ void zero_smem(void* at, int bytes) {
  asm volatile("st.bulk.weak.shared::cta [%0], %1, 0;" ::"r"(smem_addr(at)), "l"((int64_t)bytes)
               : "memory");
}

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

// How many of an item's rows, its first ones, a NaN or infinity of V reached that they do not see
// (a warp; D / 32 columns a lane).  In a column, the rows before its last such value, but from
// its first NaN on a row is NaN by what it sees.
template <int D>
__device__ __forceinline__ int reached_rows(const PackedParams& p, const Item& it) {
  const int lane = threadIdx.x & 31, q0 = it.level * kTile, n = min(kTile, it.len - q0);
  const char* v = p.v + ((int64_t)(it.beg + q0) * p.sv +
                         (int64_t)(it.part / (p.heads / p.kv_heads)) * D + lane * (D / 32)) * 2;
  int last[D / 32] = {}, nan[D / 32];
#pragma unroll
  for (int c = 0; c < D / 32; ++c) nan[c] = kTile;
#pragma unroll 1
  for (int j0 = 0; j0 < n; j0 += 32) {
    uint32_t x[32][D / 64], odd = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j)
#pragma unroll
      for (int k = 0; k < D / 64; ++k)
        x[j][k] = j0 + j < n
                      ? __ldg(reinterpret_cast<const uint32_t*>(v + (j0 + j) * p.sv * 2) + k) : 0u;
#pragma unroll
    for (int j = 0; j < 32; ++j)
#pragma unroll
      for (int k = 0; k < D / 64; ++k) odd |= (x[j][k] & 0x7f807f80u) + 0x00800080u;
    if ((odd & 0x80008000u) == 0) continue;  // no exponent of ones
#pragma unroll
    for (int j = 0; j < 32; ++j)
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const uint32_t bits = (x[j][c >> 1] >> 16 * (c & 1)) & 0x7fffu;
        if (bits >= 0x7f80u) last[c] = j0 + j;
        if (bits > 0x7f80u) nan[c] = min(nan[c], j0 + j);
      }
  }
  int rows = 0;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) rows = max(rows, min(last[c], nan[c]));
  return __reduce_max_sync(0xffffffffu, rows);
}

// All threads of the block, when its roles have ended and what they stored is in place.
template <int D, bool kMany>
__device__ __noinline__ void repair_items(const PackedParams& p, const uint32_t* flags,
                                          unsigned char* smem) {
  constexpr int NW = 12;
  __shared__ int rows[NW];
  const int warp = threadIdx.x >> 5;
  float* sq = reinterpret_cast<float*>(smem) + warp * D;
  Sequences<kMany> list;
  list.init(reinterpret_cast<int2*>(smem + NW * D * 4),
            reinterpret_cast<int2*>(smem + NW * D * 4) + kSorted, p, kTile, p.heads);
  for (int r0 = 0;; r0 += NW) {  // a warp an item
    bool more;
    const int bit = min(r0 + warp, kFlagged - 1);
    const Item mine = list.get(r0 + warp, more);
    const bool last = warp == NW - 1 && !more;
    rows[warp] = mine.ok && (flags[bit >> 5] >> (bit & 31) & 1) ? reached_rows<D>(p, mine) : 0;
    __syncthreads();
    for (int k = 0; k < NW; ++k) {  // then all warps the rows of each
      if (rows[k] == 0) continue;
      bool is;
      const Item it = list.get(r0 + k, is);
      const int64_t first = (int64_t)it.beg + it.level * kTile;
      for (int i = warp; i < rows[k]; i += NW) repair_row<D>(p, it.beg, first + i, it.part, sq);
    }
    if (__syncthreads_or(last)) return;
  }
}

// Bits n to 31 (all for n <= 0, none for n >= 32).
__device__ __forceinline__ uint32_t bits_from(int n) {
  return n >= 32 ? 0u : 0xffffffffu << max(n, 0);
}

// D (+)= A B^T of two tiles in shared memory, A [128 x D], B [128 x D].
template <int D>
__device__ __forceinline__ void issue_tiles(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = (uint32_t)((kk >> 2) * kBox + (kk & 3) * 32);
    mma_ss(d, sw128_desc(a + off, 16, 1024), sw128_desc(b + off, 16, 1024), idesc, kk > 0 ? 1u : 0u);
  }
}
template <int D, bool kMany>
__global__ void __launch_bounds__(384, 1)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                      const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to,
                      const PackedParams p) {
  using C = Fwd<D>;
  constexpr int T = C::kTileBytes;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* bar_q = bars;           // Q landed
  uint64_t* bar_qfree = bars + 1;   // the item's last S done
  uint64_t* bar_ofree = bars + 2;   // O read, 256 arrivals
  uint64_t* bar_kfull = bars + 3;   // [stage]
  uint64_t* bar_vfull = bars + 5;
  uint64_t* bar_kempty = bars + 7;
  uint64_t* bar_vempty = bars + 9;
  uint64_t* bar_s = bars + 11;      // [buffer] S done
  uint64_t* bar_o = bars + 14;      // [buffer] O += P V done
  uint64_t* bar_p = bars + 17;      // [buffer] P written, 256 arrivals
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 20);

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tslot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 32 * 8) {
    for (int i = 0; i < 17; ++i) mbar_init(bars + i, i == 2 ? 256 : 1);
    for (int i = 17; i < 20; ++i) mbar_init(bars + i, 256);
    fence_mbar_init();
  }
  uint32_t* flags = reinterpret_cast<uint32_t*>(smem + C::kOffFlags);
  if (tid <= kFlagged / 32) flags[tid] = 0;
  Sequences<kMany> list;
  list.init(reinterpret_cast<int2*>(smem + C::kOffSeq), reinterpret_cast<int2*>(smem + C::kOffStage),
            p, kTile, p.heads);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const int group = p.heads / p.kv_heads;
  bool dead = false, more;
  int b = 0;        // the tile's S buffer
  uint32_t ph = 0;  // and how often all have been used (parity)
  auto next_buffer = [&]() {
    if (++b == 3) b = 0, ph ^= 1;
  };

  // A role whose wait gave up asks for nothing more, and what it has asked for ends before
  // the block does.
  if (warp == 8 || warp == 11) {
    // --------------------------------------------------- loads: Q and K, or V
    const bool keys = warp == 8;
    const CUtensorMap* map = keys ? &tk : &tv;
    uint64_t *full = keys ? bar_kfull : bar_vfull, *empty = keys ? bar_kempty : bar_vempty;
    unsigned char* stages = smem + (keys ? C::kOffK : C::kOffV);
    int n = 0, items = 0;
    for (int r = 0;; ++r) {
      const Item it = list.get(r, more);
      if (!more) break;
      if (!it.ok) r = max(r, it.part - 1);
      if (!it.ok || lane != 0) continue;
      const int h = it.part;
      if (keys) {
        if (items > 0) wait_spin(bar_qfree, (uint32_t)((items - 1) & 1), dead, p.err);
        if (!dead) {
          ++items;
          mbar_arrive_expect_tx(bar_q, T);
          for (int x = 0; x < C::kBoxes; ++x)
            load_box(smem + x * kBox, &tq, 64 * x, h, it.beg + it.level * kTile, bar_q);
        }
      }
      for (int t = 0; t <= it.level; ++t) {
        const int s = n & 1;
        if (n >= 2) wait_spin(&empty[s], (uint32_t)(((n >> 1) - 1) & 1), dead, p.err);
        if (dead) break;
        ++n;
        mbar_arrive_expect_tx(&full[s], T);
        for (int x = 0; x < C::kBoxes; ++x)
          load_box(stages + s * T + x * kBox, map, 64 * x, h / group, it.beg + t * kTile, &full[s]);
      }
    }
    for (int i = max(n - 2, 0); i < n; ++i)
      mbar_wait_bounded(&full[i & 1], (uint32_t)((i >> 1) & 1), p.err);
    if (items > 0) mbar_wait_bounded(bar_q, (uint32_t)((items - 1) & 1), p.err);
  } else if (warp == 9) {
    // ----------------------------------------------------------- S = Q K^T
    int n = 0, items = 0;
    for (int r = 0;; ++r) {
      const Item it = list.get(r, more);
      if (!more) break;
      if (!it.ok) r = max(r, it.part - 1);
      if (!it.ok || lane != 0) continue;
      wait_spin(bar_q, (uint32_t)(items++ & 1), dead, p.err);
      for (int t = 0; t <= it.level; ++t) {
        const int s = n & 1;
        wait_spin(&bar_kfull[s], (uint32_t)((n >> 1) & 1), dead, p.err);
        // O += P V of three tiles ago is done with the buffer
        if (n >= 3) wait_spin(&bar_o[b], ph ^ 1, dead, p.err);
        if (dead) break;
        tc_fence_after();
        issue_tiles<D>(tmem + 128 * b, smem_addr(smem), smem_addr(smem + C::kOffK + s * T),
                       C::kIdescS);
        mma_commit(&bar_s[b]);
        mma_commit(&bar_kempty[s]);
        if (t == it.level) mma_commit(bar_qfree);
        ++n;
        next_buffer();
      }
    }
    if (n > 0) {  // (the last one's buffer, and its parity)
      const int last = b == 0 ? 2 : b - 1;
      mbar_wait_bounded(&bar_s[last], b == 0 ? ph ^ 1 : ph, p.err);
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ O += P V
    int n = 0, items = 0;
    for (int r = 0;; ++r) {
      const Item it = list.get(r, more);
      if (!more) break;
      if (!it.ok) r = max(r, it.part - 1);
      if (!it.ok || lane != 0) continue;
      for (int t = 0; t <= it.level; ++t) {
        const int s = n & 1;
        wait_spin(&bar_vfull[s], (uint32_t)((n >> 1) & 1), dead, p.err);
        const int rest = it.len - t * kTile;
        if (rest < kTile && !dead) {  // rows behind the sequence
          for (int x = 0; x < C::kBoxes; ++x)
            zero_smem(smem + C::kOffV + s * T + x * kBox + rest * 128, (kTile - rest) * 128);
          fence_proxy_async_smem();
        }
        if (t == 0 && items > 0) wait_spin(bar_ofree, (uint32_t)((items - 1) & 1), dead, p.err);
        wait_spin(&bar_p[b], ph, dead, p.err);
        if (dead) break;
        tc_fence_after();
        const uint32_t v_addr = smem_addr(smem + C::kOffV + s * T);
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          mma_ts(tmem + C::kColO, tmem + 128 * b + 8 * kk + (kk >= 4 ? 32 : 0),
                 sw128_desc(v_addr + kk * 2048, kBox, 1024), C::kIdescO,
                 (t > 0 || kk > 0) ? 1u : 0u);
        mma_commit(&bar_o[b]);
        mma_commit(&bar_vempty[s]);
        ++n;
        next_buffer();
      }
      ++items;
    }
    if (n > 0) {
      const int last = b == 0 ? 2 : b - 1;
      mbar_wait_bounded(&bar_o[last], b == 0 ? ph ^ 1 : ph, p.err);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int row = tid & 127, half = warp >> 2, col0 = 64 * half;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + col0, tO = tmem + lanes + C::kColO;
    const float sc = p.scale_log2;
    // the diagonal: a bit for each of this thread's keys that its row sees
    const uint32_t sees[2] = {~bits_from(row + 1 - col0), ~bits_from(row - 31 - col0)};
    unsigned char* box = smem + C::kOffStage + warp * C::kStage;
    float* trade = reinterpret_cast<float*>(smem + C::kOffTrade);
    int swaps = 0;
    // gives `x` to the row's other thread and takes its value
    auto swap = [&](float x) {
      float* at = trade + 256 * (swaps++ & 1);
      at[128 * half + row] = x;
      named_bar(1 + (warp & 3), 64);
      return at[128 * (half ^ 1) + row];
    };
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!dead) dead = !mbar_wait_bounded(bar, parity, p.err);
    };
    for (int r = 0;; ++r) {
      const Item it = list.get(r, more);
      if (!more) break;
      if (!it.ok) {
        r = max(r, it.part - 1);
        continue;
      }
      const int h = it.part, q0 = it.level * kTile;
      float m = -INFINITY, l = 0.f;  // for all keys; of this thread's
      for (int t = 0; t <= it.level; ++t) {
        wait(&bar_s[b], ph);
        tc_fence_after();
        uint32_t v[2][32];
        tmem_ld32_nowait(tS + 128 * b, v[0]);
        tmem_ld32_nowait(tS + 128 * b + 32, v[1]);
        tmem_ld_wait();
        if (t == it.level) {  // the diagonal: keys after the row
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(sees[c] >> i & 1)) v[c][i] = __float_as_uint(-INFINITY);
        }
        float mx[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = __uint_as_float(v[0][k]);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) mx[i & 7] = fmaxf(mx[i & 7], __uint_as_float(v[c][i]));
        const float mx0 = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const float mx1 = fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]));
        // m, the sums' reference, moves only when the tile's maximum exceeds it, and then to
        // 2^8 above, so O is rarely rescaled.  P is at most 1: O overflows only where a sum of
        // that many v does.
        const float mine = fmaxf(mx0, mx1);
        const float mt = fmaxf(mine, swap(mine)) * sc;
        const float mn = mt > m ? mt + 8.f : m;
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float alpha = ex2(m - ref);
        if (t > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          const int before = b == 0 ? 2 : b - 1;
          wait(&bar_o[before], b == 0 ? ph ^ 1 : ph);
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t o[32];
            const uint32_t at = tO + D / 2 * half + 32 * c;
            tmem_ld32_nowait(at, o);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float a0, a1;
              mul2(a0, a1, __uint_as_float(o[i]), __uint_as_float(o[i + 1]), alpha, alpha);
              o[i] = __float_as_uint(a0);
              o[i + 1] = __float_as_uint(a1);
            }
            tmem_st32(at, o);
          }
        }
        float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            float t0, t1, t2, t3;
            fma2(t0, t1, __uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1]), sc, sc, -ref, -ref);
            fma2(t2, t3, __uint_as_float(v[c][i + 2]), __uint_as_float(v[c][i + 3]), sc, sc, -ref,
                 -ref);
            const float p0 = ex2(t0), p1 = ex2(t1), p2 = ex2(t2), p3 = ex2(t3);
            add2(l0, l1, l0, l1, p0, p1);
            add2(l2, l3, l2, l3, p2, p3);
            pk[i >> 1] = pack_bf16(p0, p1);
            pk[(i >> 1) + 1] = pack_bf16(p2, p3);
          }
          tmem_st16(tS + 128 * b + 16 * c, pk);  // (over columns of its own)
        }
        l = l * alpha + ((l0 + l1) + (l2 + l3));
        m = mn;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar_p[b]);
        next_buffer();
      }
      // O / l and lse
      const int last = b == 0 ? 2 : b - 1;
      wait(&bar_o[last], b == 0 ? ph ^ 1 : ph);
      tc_fence_after();
      const int col = D == 128 ? col0 : 0;  // (head_dim 64: the first four warps store)
      uint32_t o[2][32];
      tmem_ld32_nowait(tO + col, o[0]);
      tmem_ld32_nowait(tO + col + 32, o[1]);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(bar_ofree);
      l += swap(l);
      const float inv = 1.f / l;
      const bool live = q0 + row < it.len;
      const int64_t at = (int64_t)it.beg + q0 + row;
      if (p.lse != nullptr && live && half == 0)
        p.lse[(int64_t)h * p.tokens + at] = (m + __log2f(l)) * kLn2;
      float f0 = 0.f, f1 = 0.f;  // NaN if any value is NaN or infinite
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 32; i += 2)
          fma2(f0, f1, __uint_as_float(o[c][i]), __uint_as_float(o[c][i + 1]), 0.f, 0.f, f0, f1);
      f0 += f1;
      const bool fine = f0 + swap(f0) == 0.f;
      char* out = const_cast<char*>(p.o) + (at * p.so + (int64_t)h * D + col) * 2;
      if (D == 128 || half == 0)
        put_box(o[0], o[1], inv, box, &to, col, h, (int)at, out,
                __all_sync(0xffffffffu, live), live);
      if (half == 0 && __any_sync(0xffffffffu, live && !fine) && lane == 0) {
        atomicOr(flags + (min(r, kFlagged - 1) >> 5), 1u << (min(r, kFlagged - 1) & 31));
        flags[kFlagged / 32] = 1;
      }
    }
    if (lane == 0) stores_done();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u)
                 : "memory");
  if (flags[kFlagged / 32]) repair_items<D, kMany>(p, flags, smem + C::kOffStage);
}

// ------------------------------------------------------------------ backward ---
// A kernel for delta = sum dO o of each row, then one whose blocks take tiles of dK and dV and
// then tiles of dQ (S and dP are computed for both, so that every sum has one owner and a fixed
// order).  dK and dV are computed transposed, so that all three are products of a weight matrix
// in TMEM with a tile in shared memory, as O = P V is.  Their items are long and uneven: blocks
// with the longest of them get the shortest of dQ's (in two kernels 296 instead of 293 us, and 53
// instead of 47 us for the second sizes below).
//
// A block has eight softmax warps, two to a quarter of the 128 TMEM lanes, with 64 of the
// tile's 128 columns each; warp 8 loads (V in dQ: warp 11), warps 9 and 10 issue.
//
// dQ, a query tile against key tiles t: S(t) = Q K^T, dP(t) = dO V^T, then
//   dS = P (dP - delta) as bf16 over S, dQ += dS K.  S has two buffers and K three stages, so
//   that S and dP of t + 1 run while the softmax works on t.  dQ is read and stored after the
//   next item's first tile, while which its last product runs.
// dK and dV, a key tile against the query tiles of all heads of its group, in two TMEM buffers
//   X and Y that change places with each tile: S^T = K Q^T in X, dP^T = V dO^T in Y; P^T and
//   dS^T, bf16, over S^T in X; dV += P^T dO, dK += dS^T Q.  Y is free once dP^T is read, so S^T
//   of the next tile and dV run while the softmax goes on to dS^T; the next dP^T, into X, while
//   it works on the next P^T.
//
// What bounds them: the chain from one tile's weights over the product that reads them to the
// next tile's scores.  A product of 128 x 128 x 128 takes 690 cycles with both operands in
// shared memory and 1090 with one in TMEM when it runs alone, 530 in company; the two parts
// come to 2450 and 3200 cycles a tile of three and four products.  Sequences of 2414, 0, 1,
// 1924 and 639 tokens, 32 heads on 8, head_dim 128: 16 us for delta and 277; twelve of 0 to 603
// tokens, 12 heads on 4, head_dim 64: 3 and 44 us.  Tried and no faster, as kernels of their own:
// delta inside dQ's, from a tile of o (144 us instead of 24 + 110); lse and delta as further
// terms of the products instead of 32 loads from shared memory a tile (201 instead of 190 us for
// dK, dV then); sixteen softmax warps (172 of 171); a buffer more for dP^T with head_dim 64 (32
// of 33 us).
//
// Rows of a tile beyond its sequence are masked, and where such a row is summed over (K in
// dQ; Q and dO in dK, dV) it is set to zero in shared memory before the product, so that no
// other sequence's NaN takes part.
template <int D>
struct Bwd {
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBoxes * kBox;
  static constexpr int kOffStat = 6 * kTileBytes;     // dK, dV: [stage][-lse, -delta][128]
  static constexpr int kOffTrade = 7 * kTileBytes;    // dQ: [128] floats
  static constexpr int kOffBarQ = kOffTrade + 512, kOffBarK = kOffBarQ + 256;
  static constexpr int kStage = 32 * 128;
  static constexpr int kOffSeq = kOffBarK + 256;
  static constexpr int kSmem = kOffSeq + kSorted * 8 + 1024;
  static constexpr uint32_t kIdescS = attn_idesc(kTile, kTile, false);
  static constexpr uint32_t kIdescG = attn_idesc(kTile, D, true);
};

// The tensor maps of the backward kernel: 128-row boxes of q, k, v and dO, 32-row boxes of dK and
// dV (dQ is stored row by row).
struct BwdMaps {
  CUtensorMap q, k, v, g, dk, dv;
};

// Rows [from, 128) of a tile in shared memory become zero (all lanes of a warp).
template <int D>
__device__ __forceinline__ void clear_rows(unsigned char* tile, int from) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  for (int b = 0; b < D / 64; ++b)
    for (int i = from * 8 + lane; i < kTile * 8; i += 32)
      *reinterpret_cast<uint4*>(tile + b * kBox + i * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

// delta of the rows within the sequences: a warp a token, D / 8 lanes a head, four heads of
// each under way.
template <int D>
__global__ void __launch_bounds__(256) packed_delta_kernel(const PackedParams p) {
  constexpr int G = D / 8, R = 32 / G, U = 4;
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= p.tokens || t < __ldg(p.cu) || t >= __ldg(p.cu + p.batch)) return;
  const char* g = p.dout + (t * p.sdo + lane % G * 8) * 2;
  const char* o = p.o + (t * p.so + lane % G * 8) * 2;
  for (int h0 = lane / G; h0 - lane / G < p.heads; h0 += R * U) {
    uint4 a[U], b[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int h = min(h0 + k * R, p.heads - 1);
      a[k] = ld_chunk_cached(g + (int64_t)h * D * 2);
      b[k] = ld_chunk_cached(o + (int64_t)h * D * 2);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s += chunk_get<kBF16>(a[k], e) * chunk_get<kBF16>(b[k], e);
#pragma unroll
      for (int off = G / 2; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      const int h = h0 + k * R;
      if (h < p.heads && lane % G == 0) p.delta[(int64_t)h * p.tokens + t] = s;
    }
  }
}

template <int D, class List>
__device__ __forceinline__ void dq_part(const BwdMaps& maps, const PackedParams& p,
                                        const List& list, unsigned char* smem,
                                        uint32_t tmem) {
  using C = Bwd<D>;
  constexpr int T = C::kTileBytes;
  constexpr uint32_t kColP = 256, kColG = 384;  // dP, dQ after S's two buffers
  unsigned char *sq = smem, *sg = smem + T;
  auto sk = [&](int s) { return smem + (2 + s) * T; };
  auto sv = [&](int s) { return smem + (5 + s) * T; };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBarQ);
  uint64_t* bar_q = bars;           // Q and dO landed
  uint64_t* bar_qfree = bars + 1;   // the item's last S and dP done
  uint64_t* bar_dp = bars + 2;
  uint64_t* bar_read = bars + 3;    // dP read, 256 arrivals
  uint64_t* bar_gfree = bars + 4;   // dQ read, 256 arrivals
  uint64_t* bar_ds = bars + 5;      // [buffer] dS written, 256 arrivals
  uint64_t* bar_s = bars + 7;       // [buffer] S done
  uint64_t* bar_g = bars + 9;       // [buffer] dQ += dS K done
  uint64_t* bar_kfull = bars + 11;  // [stage of 3]
  uint64_t* bar_kempty = bars + 14;
  uint64_t* bar_vfull = bars + 17;  // [stage of 2]
  uint64_t* bar_vempty = bars + 19;
  const int group = p.heads / p.kv_heads;
  bool dead = false, more;

  if (warp == 8 || warp == 11) {
    // ------------------------------------------ loads: Q, dO and K, or V
    const bool keys = warp == 8;
    const CUtensorMap* map = keys ? &maps.k : &maps.v;
    uint64_t *full = keys ? bar_kfull : bar_vfull, *empty = keys ? bar_kempty : bar_vempty;
    const int ring = keys ? 3 : 2;
    int s = 0, n = 0, items = 0;
    uint32_t ph = 0;
    Item nx = list.get(0, more);
    for (int r = 1; more; ++r) {
      const Item it = nx;
      nx = list.get(r, more);
      if (!it.ok) r = max(r, it.part - 1);
      if (!it.ok || lane != 0) continue;
      const int h = it.part;
      if (keys) {
        if (items > 0) wait_spin(bar_qfree, (uint32_t)((items - 1) & 1), dead, p.err);
        if (!dead) {
          ++items;
          mbar_arrive_expect_tx(bar_q, 2 * T);
          for (int b = 0; b < C::kBoxes; ++b) {
            load_box(sq + b * kBox, &maps.q, 64 * b, h, it.beg + it.level * kTile, bar_q);
            load_box(sg + b * kBox, &maps.g, 64 * b, h, it.beg + it.level * kTile, bar_q);
          }
          if (nx.ok)  // (the next item's are loaded only when this one's last S and dP are done)
            for (int b = 0; b < C::kBoxes; ++b) {
              prefetch_box(&maps.q, 64 * b, nx.part, nx.beg + nx.level * kTile);
              prefetch_box(&maps.g, 64 * b, nx.part, nx.beg + nx.level * kTile);
            }
        }
      }
      for (int t = 0; t <= it.level; ++t) {
        if (n >= ring) wait_spin(&empty[s], ph ^ 1, dead, p.err);
        if (dead) break;
        ++n;
        mbar_arrive_expect_tx(&full[s], T);
        for (int b = 0; b < C::kBoxes; ++b)
          load_box((keys ? sk(s) : sv(s)) + b * kBox, map, 64 * b, h / group, it.beg + t * kTile,
                   &full[s]);
        if (++s == ring) s = 0, ph ^= 1;
      }
    }
    for (int i = min(n, ring); i > 0; --i) {
      if (--s < 0) s = ring - 1, ph ^= 1;
      mbar_wait_bounded(&full[s], ph, p.err);
    }
    if (items > 0) mbar_wait_bounded(bar_q, (uint32_t)((items - 1) & 1), p.err);
  } else if (warp == 9) {
    // ----------------------------------------------------------- S and dP
    int ns = 0, n = 0, items = 0, ks = 0;
    uint32_t kph = 0;
    Item nx = list.get(0, more);
    for (int r = 1; more; ++r) {
      const Item it = nx;
      nx = list.get(r, more);
      if (!it.ok) r = max(r, it.part - 1);
      if (!it.ok || lane != 0) continue;
      wait_spin(bar_q, (uint32_t)(items++ & 1), dead, p.err);
      for (int t = 0; t <= it.level; ++t) {
        const int s = n & 1;
        const uint32_t ph = (uint32_t)((n >> 1) & 1);
        wait_spin(&bar_kfull[ks], kph, dead, p.err);
        // dQ += dS K of two tiles ago is done with the buffer
        if (n >= 2) wait_spin(&bar_g[s], ph ^ 1, dead, p.err);
        if (dead) break;
        tc_fence_after();
        issue_tiles<D>(tmem + 128 * s, smem_addr(sq), smem_addr(sk(ks)), C::kIdescS);
        mma_commit(&bar_s[s]);
        ++ns;
        if (++ks == 3) ks = 0, kph ^= 1;
        wait_spin(&bar_vfull[s], ph, dead, p.err);
        if (n > 0) wait_spin(bar_read, (uint32_t)((n - 1) & 1), dead, p.err);
        if (dead) break;
        tc_fence_after();
        issue_tiles<D>(tmem + kColP, smem_addr(sg), smem_addr(sv(s)), C::kIdescS);
        mma_commit(bar_dp);
        mma_commit(&bar_vempty[s]);
        if (t == it.level) mma_commit(bar_qfree);
        ++n;
      }
    }
    if (ns > 0) mbar_wait_bounded(&bar_s[(ns - 1) & 1], (uint32_t)(((ns - 1) >> 1) & 1), p.err);
    if (n > 0) mbar_wait_bounded(bar_dp, (uint32_t)((n - 1) & 1), p.err);
  } else if (warp == 10) {
    // --------------------------------------------------------- dQ += dS K
    int n = 0, items = 0, ks = 0;
    uint32_t kph = 0;
    Item nx = list.get(0, more);
    for (int r = 1; more; ++r) {
      const Item it = nx;
      nx = list.get(r, more);
      if (!it.ok) {
        r = max(r, it.part - 1);
        continue;
      }
      for (int t = 0; t <= it.level; ++t) {
        const int s = n & 1, rest = it.len - t * kTile;
        if (lane == 0) wait_spin(&bar_kfull[ks], kph, dead, p.err);
        if (rest < kTile) {
          // (S may be reading them: the columns that they give are masked)
          dead = __shfl_sync(0xffffffffu, (int)dead, 0) != 0;
          if (dead) break;
          clear_rows<D>(sk(ks), rest);
        }
        if (lane == 0) {
          wait_spin(&bar_ds[s], (uint32_t)((n >> 1) & 1), dead, p.err);
          if (t == 0 && items > 0) wait_spin(bar_gfree, (uint32_t)((items - 1) & 1), dead, p.err);
        }
        dead = __shfl_sync(0xffffffffu, (int)dead, 0) != 0;
        if (dead) break;
        if (lane == 0) {
          tc_fence_after();
          const uint32_t k_addr = smem_addr(sk(ks));
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_ts(tmem + kColG, tmem + 128 * s + 8 * kk + (kk >= 4 ? 32 : 0),
                   sw128_desc(k_addr + kk * 2048, kBox, 1024), C::kIdescG,
                   (t > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&bar_g[s]);
          mma_commit(&bar_kempty[ks]);
        }
        if (++ks == 3) ks = 0, kph ^= 1;
        ++n;
      }
      ++items;
    }
    if (lane == 0 && n > 0)
      mbar_wait_bounded(&bar_g[(n - 1) & 1], (uint32_t)(((n - 1) >> 1) & 1), p.err);
  } else {
    // ------------------------------------------------------------ softmax
    const int row = tid & 127, half = warp >> 2, col0 = 64 * half;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + col0, tG = tmem + lanes + kColG;
    const float sc = p.scale_log2;
    // the diagonal: a bit for each of this thread's keys that its row sees
    const uint32_t sees[2] = {~bits_from(row + 1 - col0), ~bits_from(row - 31 - col0)};
    float* trade = reinterpret_cast<float*>(smem + C::kOffTrade);
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!dead) dead = !mbar_wait_bounded(bar, parity, p.err);
    };
    int n = 0;
    // An item's dQ is read and stored after the next one's first tile, during which its last
    // product runs.
    int old_first = 0, old_rows = 0, old_head = 0;  // of this warp's rows: the first, how many
    auto store = [&]() {
      const int last = n - 1;  // (called before the next tile is counted)
      wait(&bar_g[last & 1], (uint32_t)((last >> 1) & 1));
      tc_fence_after();
      const int col = D == 128 ? col0 : 0;  // (head_dim 64: the first four warps store)
      uint32_t o[2][32];
      tmem_ld32_nowait(tG + col, o[0]);
      tmem_ld32_nowait(tG + col + 32, o[1]);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive(bar_gfree);
      if (D == 128 || half == 0)
        put_rows(o[0], o[1], p.scale,
                 const_cast<char*>(p.dq) +
                     ((int64_t)old_first * p.sdq + (int64_t)old_head * D + col) * 2,
                 p.sdq * 2, __ballot_sync(0xffffffffu, lane < old_rows));
    };
    float nl_next = 0.f, nd_next = 0.f;
    auto load_stats = [&](const Item& it) {
      const int q = it.level * kTile + row;
      const int64_t stat = (int64_t)it.part * p.tokens + it.beg + q;
      const bool live = it.ok && q < it.len;
      nl_next = live ? -p.lse[stat] * kLog2e : 0.f;
      nd_next = live ? -p.delta[stat] : 0.f;
    };
    Item nx = list.get(0, more);
    load_stats(nx);
    for (int r = 1; more; ++r) {
      const Item it = nx;
      const float nl = nl_next;
      float nd = nd_next;
      nx = list.get(r, more);
      load_stats(nx);
      if (!it.ok) {
        r = max(r, it.part - 1);
        continue;
      }
      for (int t = 0; t <= it.level; ++t, ++n) {
        uint32_t v[2][32], w[2][32];
        const int s = n & 1;
        const uint32_t tB = tS + 128 * s;
        wait(&bar_s[s], (uint32_t)((n >> 1) & 1));
        tc_fence_after();
        tmem_ld32_nowait(tB, v[0]);
        tmem_ld32_nowait(tB + 32, v[1]);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float t0, t1;
            fma2(t0, t1, __uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1]), sc, sc, nl, nl);
            v[c][i] = __float_as_uint(ex2(t0));
            v[c][i + 1] = __float_as_uint(ex2(t1));
          }
        wait(bar_dp, (uint32_t)(n & 1));
        tc_fence_after();
        tmem_ld32_nowait(tS + kColP, w[0]);
        tmem_ld32_nowait(tS + kColP + 32, w[1]);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(bar_read);
        if (it.level == 0) {
          // One key tile: delta = sum P dP, without the rounding of o, is at hand.  It counts
          // most in these rows, whose few large weights all but cancel in dP - delta.
          float d = 0.f;
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (sees[c] >> i & 1)
                d = fmaf(__uint_as_float(v[c][i]), __uint_as_float(w[c][i]), d);
          if (half == 1) trade[row] = d;
          named_bar(1 + (warp & 3), 64);
          if (half == 0) trade[row] = d += trade[row];
          named_bar(1 + (warp & 3), 64);
          if (half == 1) d = trade[row];
          nd = -d;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float t0, t1;
            add2(t0, t1, __uint_as_float(w[c][i]), __uint_as_float(w[c][i + 1]), nd, nd);
            mul2(t0, t1, t0, t1, __uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1]));
            w[c][i] = __float_as_uint(t0);
            w[c][i + 1] = __float_as_uint(t1);
          }
        if (t == it.level) {  // the diagonal: keys after the row
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(sees[c] >> i & 1)) w[c][i] = 0u;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            pk[i >> 1] = pack_bf16(__uint_as_float(w[c][i]), __uint_as_float(w[c][i + 1]));
          tmem_st16(tB + 16 * c, pk);  // (over columns of its own)
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar_ds[s]);
        if (t == 0 && n > 0) store();
      }
      old_first = it.beg + it.level * kTile + 32 * (warp & 3);
      old_rows = it.beg + it.len - old_first;
      old_head = it.part;
    }
    if (n > 0) store();
  }
}

template <int D, class List>
__device__ __forceinline__ void dkv_part(const BwdMaps& maps, const PackedParams& p,
                                         const List& list, unsigned char* smem,
                                         uint32_t tmem) {
  using C = Bwd<D>;
  constexpr int T = C::kTileBytes;
  constexpr uint32_t kColV = 256, kColK = 256 + D;  // dV, dK, after two buffers
  unsigned char *sk = smem, *sv = smem + T;
  auto sq = [&](int s) { return smem + (2 + s) * T; };
  auto sg = [&](int s) { return smem + (4 + s) * T; };
  auto stats = [&](int s) { return reinterpret_cast<float*>(smem + C::kOffStat) + 256 * s; };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBarK);
  uint64_t* bar_kv = bars;          // K and V landed
  uint64_t* bar_s = bars + 1;
  uint64_t* bar_dp = bars + 2;
  uint64_t* bar_g = bars + 3;       // dV += P^T dO and dK += dS^T Q done
  uint64_t* bar_qfull = bars + 4;   // [stage]
  uint64_t* bar_dofull = bars + 6;
  uint64_t* bar_stat = bars + 8;    // lse and delta written
  uint64_t* bar_empty = bars + 10;  // [stage] dV and dK are done with it
  uint64_t* bar_read = bars + 12;   // dP^T read, 256 arrivals
  uint64_t* bar_p = bars + 13;      // [buffer] P^T written, 256 arrivals
  uint64_t* bar_ds = bars + 15;     // dS^T written, 256 arrivals
  uint64_t* bar_gfree = bars + 16;  // dK and dV read, 256 arrivals
  uint64_t* bar_kvfree = bars + 17; // the output boxes (over K and V) are read, 8 arrivals
  const int group = p.heads / p.kv_heads;
  bool dead = false, more;
  // Item: key tile `first` of the sequence's nt, level + 1 query tiles of each head of `part`.
  auto first_of = [&](const Item& it) { return (it.len + kTile - 1) / kTile - 1 - it.level; };

  if (warp == 8) {
    // ------------------------------------------------------------ loads
    int n = 0, items = 0;
    for (int r = 0;; ++r) {
      const Item it = list.get(r, more);
      if (!more) break;
      if (!it.ok) {
        r = max(r, it.part - 1);
        continue;
      }
      const int first = first_of(it);
      if (lane == 0) {
        if (items > 0) wait_spin(bar_kvfree, (uint32_t)((items - 1) & 1), dead, p.err);
        if (!dead) {
          mbar_arrive_expect_tx(bar_kv, 2 * T);
          for (int b = 0; b < C::kBoxes; ++b) {
            load_box(sk + b * kBox, &maps.k, 64 * b, it.part, it.beg + first * kTile, bar_kv);
            load_box(sv + b * kBox, &maps.v, 64 * b, it.part, it.beg + first * kTile, bar_kv);
          }
          ++items;
        }
      }
      for (int h = it.part * group; h < (it.part + 1) * group; ++h)
        for (int i = first; i <= first + it.level; ++i) {
          const int s = n & 1;
          if (lane == 0) {
            if (n >= 2) wait_spin(&bar_empty[s], (uint32_t)(((n >> 1) - 1) & 1), dead, p.err);
            if (!dead) {
              mbar_arrive_expect_tx(&bar_qfull[s], T);
              for (int b = 0; b < C::kBoxes; ++b)
                load_box(sq(s) + b * kBox, &maps.q, 64 * b, h, it.beg + i * kTile, &bar_qfull[s]);
              mbar_arrive_expect_tx(&bar_dofull[s], T);
              for (int b = 0; b < C::kBoxes; ++b)
                load_box(sg(s) + b * kBox, &maps.g, 64 * b, h, it.beg + i * kTile, &bar_dofull[s]);
            }
          }
          dead = __shfl_sync(0xffffffffu, (int)dead, 0) != 0;
          if (dead) break;
          float* st = stats(s);
          float a[4], d[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = i * kTile + 32 * j + lane;
            const int64_t at = (int64_t)h * p.tokens + it.beg + row;
            a[j] = row < it.len ? -__ldg(p.lse + at) * kLog2e : 0.f;
            d[j] = row < it.len ? -p.delta[at] : 0.f;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            st[32 * j + lane] = a[j];
            st[128 + 32 * j + lane] = d[j];
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_stat[s]);
          ++n;
        }
    }
    if (lane == 0) {
      for (int i = max(n - 2, 0); i < n; ++i) {
        mbar_wait_bounded(&bar_qfull[i & 1], (uint32_t)((i >> 1) & 1), p.err);
        mbar_wait_bounded(&bar_dofull[i & 1], (uint32_t)((i >> 1) & 1), p.err);
      }
      if (items > 0) mbar_wait_bounded(bar_kv, (uint32_t)((items - 1) & 1), p.err);
    }
  } else if (warp == 9) {
    // ------------------------------------------- S^T = K Q^T, dP^T = V dO^T
    int ns = 0, n = 0, items = 0;
    for (int r = 0;; ++r) {
      const Item it = list.get(r, more);
      if (!more) break;
      if (!it.ok) r = max(r, it.part - 1);
      if (!it.ok || lane != 0) continue;
      const int tiles = group * (it.level + 1);
      wait_spin(bar_kv, (uint32_t)(items++ & 1), dead, p.err);
      for (int t = 0; t < tiles; ++t) {
        const int s = n & 1;
        const uint32_t ph = (uint32_t)((n >> 1) & 1), before = (uint32_t)((n - 1) & 1);
        wait_spin(&bar_qfull[s], ph, dead, p.err);
        if (n > 0) wait_spin(bar_read, before, dead, p.err);  // this buffer had dP^T
        if (dead) break;
        tc_fence_after();
        issue_tiles<D>(tmem + 128 * s, smem_addr(sk), smem_addr(sq(s)), C::kIdescS);
        mma_commit(bar_s);
        ++ns;
        wait_spin(&bar_dofull[s], ph, dead, p.err);
        if (n > 0) wait_spin(bar_g, before, dead, p.err);  // this one the weights
        if (dead) break;
        tc_fence_after();
        issue_tiles<D>(tmem + 128 * (s ^ 1), smem_addr(sv), smem_addr(sg(s)), C::kIdescS);
        mma_commit(bar_dp);
        ++n;
      }
    }
    if (ns > 0) mbar_wait_bounded(bar_s, (uint32_t)((ns - 1) & 1), p.err);
    if (n > 0) mbar_wait_bounded(bar_dp, (uint32_t)((n - 1) & 1), p.err);
  } else if (warp == 10) {
    // ---------------------------------------- dV += P^T dO, dK += dS^T Q
    int n = 0, items = 0;
    bool open = false;  // dV of a tile is issued, its dK is not
    for (int r = 0;; ++r) {
      const Item it = list.get(r, more);
      if (!more) break;
      if (!it.ok) {
        r = max(r, it.part - 1);
        continue;
      }
      const int first = first_of(it), tiles = group * (it.level + 1);
      for (int t = 0, i = first; t < tiles; ++t, i = i == first + it.level ? first : i + 1) {
        const int s = n & 1, rest = it.len - i * kTile;
        const uint32_t ph = (uint32_t)((n >> 1) & 1), tW = tmem + 128 * s;
        auto sum = [&](uint32_t to, uint32_t weights, const unsigned char* tile) {
          tc_fence_after();
          const uint32_t addr = smem_addr(tile);
#pragma unroll
          for (int kk = 0; kk < kTile / 16; ++kk)
            mma_ts(tmem + to, weights + 8 * kk + (kk >= 4 ? 32 : 0),
                   sw128_desc(addr + kk * 2048, kBox, 1024), C::kIdescG,
                   (t > 0 || kk > 0) ? 1u : 0u);
        };
        if (lane == 0) {
          wait_spin(&bar_dofull[s], ph, dead, p.err);
          wait_spin(&bar_qfull[s], ph, dead, p.err);
        }
        if (rest < kTile) {
          // (S^T and dP^T may be reading them: the columns that they give are masked)
          dead = __shfl_sync(0xffffffffu, (int)dead, 0) != 0;
          if (dead) break;
          clear_rows<D>(sg(s), rest);
          clear_rows<D>(sq(s), rest);
        }
        if (lane == 0) {
          wait_spin(&bar_p[s], ph, dead, p.err);
          if (t == 0 && items > 0) wait_spin(bar_gfree, (uint32_t)((items - 1) & 1), dead, p.err);
        }
        dead = __shfl_sync(0xffffffffu, (int)dead, 0) != 0;
        if (dead) break;
        open = true;
        if (lane == 0) {
          sum(kColV, tW, sg(s));
          wait_spin(bar_ds, (uint32_t)(n & 1), dead, p.err);
        }
        dead = __shfl_sync(0xffffffffu, (int)dead, 0) != 0;
        if (dead) break;
        if (lane == 0) {
          sum(kColK, tW + 32, sq(s));
          mma_commit(bar_g);
          mma_commit(&bar_empty[s]);
        }
        open = false;
        ++n;
      }
      ++items;
    }
    if (lane == 0) {
      if (open) {  // (nobody waits for it any more)
        mma_commit(bar_g);
        ++n;
      }
      if (n > 0) mbar_wait_bounded(bar_g, (uint32_t)((n - 1) & 1), p.err);
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax
    const int row = tid & 127, half = warp >> 2, col0 = 64 * half;  // key row, query columns
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + col0;
    const float sc = p.scale_log2;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!dead) dead = !mbar_wait_bounded(bar, parity, p.err);
    };
    int n = 0;
    for (int r = 0;; ++r) {
      const Item it = list.get(r, more);
      if (!more) break;
      if (!it.ok) {
        r = max(r, it.part - 1);
        continue;
      }
      const int first = first_of(it), tiles = group * (it.level + 1);
      for (int t = 0, i = first; t < tiles; ++t, ++n, i = i == first + it.level ? first : i + 1) {
        const int s = n & 1;
        const float4* nl = reinterpret_cast<const float4*>(stats(s) + col0);
        const float4* nd = nl + 32;
        const uint32_t tX = tS + 128 * s, tY = tS + 128 * (s ^ 1);
        uint32_t v[2][32], pk[16];
        // columns [lo, hi) of this thread's 64 see its key
        const int lo = i == first ? row - col0 : 0, hi = it.len - i * kTile - col0;
        const bool edge = i == first || it.len - i * kTile < kTile;
        uint32_t sees[2];  // a bit for each
#pragma unroll
        for (int c = 0; c < 2; ++c)
          sees[c] = bits_from(lo - 32 * c) & ~bits_from(hi - 32 * c);
        wait(&bar_stat[s], (uint32_t)((n >> 1) & 1));
        wait(bar_s, (uint32_t)(n & 1));
        tc_fence_after();
        tmem_ld32_nowait(tX, v[0]);
        tmem_ld32_nowait(tX + 32, v[1]);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 l = nl[8 * c + (j >> 2)];
            float t0, t1, t2, t3;
            fma2(t0, t1, __uint_as_float(v[c][j]), __uint_as_float(v[c][j + 1]), sc, sc, l.x, l.y);
            fma2(t2, t3, __uint_as_float(v[c][j + 2]), __uint_as_float(v[c][j + 3]), sc, sc, l.z,
                 l.w);
            v[c][j] = __float_as_uint(ex2(t0));
            v[c][j + 1] = __float_as_uint(ex2(t1));
            v[c][j + 2] = __float_as_uint(ex2(t2));
            v[c][j + 3] = __float_as_uint(ex2(t3));
          }
          if (edge) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(sees[c] >> j & 1)) v[c][j] = 0u;
          }
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            pk[j >> 1] = pack_bf16(__uint_as_float(v[c][j]), __uint_as_float(v[c][j + 1]));
          tmem_st16(tX + 16 * c, pk);  // (over columns of its own)
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bar_p[s]);
        wait(bar_dp, (uint32_t)(n & 1));
        tc_fence_after();
        if (first == 0 && i == 0) {
          // The sequence's first rows see this key tile alone: as in dQ, delta = sum P dP, over
          // a column's 32 lanes by halving, then over the four warps of the column.
          float* part = reinterpret_cast<float*>(smem + C::kOffStat + 2048);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t y[32];
            float x[32];
            tmem_ld32_nowait(tY + 32 * c, y);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j)
              x[j] = sees[c] >> j & 1 ? __uint_as_float(v[c][j]) * __uint_as_float(y[j]) : 0.f;
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1)
#pragma unroll
              for (int j = 0; j < off; ++j) {
                const bool up = (lane & off) != 0;
                const float give = up ? x[j] : x[j + off], keep = up ? x[j + off] : x[j];
                x[j] = keep + __shfl_xor_sync(0xffffffffu, give, off);
              }
            part[128 * (warp & 3) + col0 + 32 * c + lane] = x[0];
          }
          named_bar(5 + half, 128);
          if (row < 64) {
            const float* at = part + col0 + row;
            stats(s)[128 + col0 + row] = -((at[0] + at[128]) + (at[256] + at[384]));
          }
          named_bar(5 + half, 128);
        }
        uint32_t w[2][32];
        tmem_ld32_nowait(tY, w[0]);
        tmem_ld32_nowait(tY + 32, w[1]);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(bar_read);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 d = nd[8 * c + (j >> 2)];
            float t0, t1, t2, t3;
            add2(t0, t1, __uint_as_float(w[c][j]), __uint_as_float(w[c][j + 1]), d.x, d.y);
            add2(t2, t3, __uint_as_float(w[c][j + 2]), __uint_as_float(w[c][j + 3]), d.z, d.w);
            mul2(t0, t1, t0, t1, __uint_as_float(v[c][j]), __uint_as_float(v[c][j + 1]));
            mul2(t2, t3, t2, t3, __uint_as_float(v[c][j + 2]), __uint_as_float(v[c][j + 3]));
            w[c][j] = __float_as_uint(t0);
            w[c][j + 1] = __float_as_uint(t1);
            w[c][j + 2] = __float_as_uint(t2);
            w[c][j + 3] = __float_as_uint(t3);
          }
          if (edge) {  // (0 times a NaN)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(sees[c] >> j & 1)) w[c][j] = 0u;
          }
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            pk[j >> 1] = pack_bf16(__uint_as_float(w[c][j]), __uint_as_float(w[c][j + 1]));
          tmem_st16(tX + 32 + 16 * c, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar_ds);
      }
      wait(bar_g, (uint32_t)((n - 1) & 1));
      tc_fence_after();
      const bool live = first * kTile + row < it.len;
      const bool whole = __all_sync(0xffffffffu, live);
      const int64_t at = (int64_t)it.beg + first * kTile + row;
      const uint32_t tV = tmem + lanes + kColV, tK = tmem + lanes + kColK;
      char* dv = const_cast<char*>(p.dv) + (at * p.sdv + (int64_t)it.part * D) * 2;
      char* dk = const_cast<char*>(p.dk) + (at * p.sdk + (int64_t)it.part * D) * 2;
      uint32_t o[2][32];
      if constexpr (D == 128) {  // 64 columns of dV and of dK each
        uint32_t o2[2][32];
        tmem_ld32_nowait(tV + col0, o[0]);
        tmem_ld32_nowait(tV + col0 + 32, o[1]);
        tmem_ld32_nowait(tK + col0, o2[0]);
        tmem_ld32_nowait(tK + col0 + 32, o2[1]);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(bar_gfree);
        unsigned char* box = smem + warp * 2 * C::kStage;
        put_box(o[0], o[1], 1.f, box, &maps.dv, col0, it.part, (int)at, dv + 2 * col0, whole,
                live);
        put_box(o2[0], o2[1], p.scale, box + C::kStage, &maps.dk, col0, it.part, (int)at,
                dk + 2 * col0, whole, live);
      } else {  // dV for one half of the warps, dK for the other
        tmem_ld32_nowait(half ? tK : tV, o[0]);
        tmem_ld32_nowait((half ? tK : tV) + 32, o[1]);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(bar_gfree);
        put_box(o[0], o[1], half ? p.scale : 1.f, smem + warp * C::kStage,
                half ? &maps.dk : &maps.dv, 0, it.part, (int)at, half ? dk : dv, whole, live);
      }
      if (lane == 0) {
        stores_read();
        mbar_arrive(bar_kvfree);
      }
    }
    if (lane == 0) stores_done();
  }
}

template <int D, bool kMany>
__global__ void __launch_bounds__(384, 1)
    packed_bwd_kernel(const __grid_constant__ BwdMaps maps, const PackedParams p) {
  using C = Bwd<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5;
  uint64_t* bars_q = reinterpret_cast<uint64_t*>(smem + C::kOffBarQ);
  uint64_t* bars_k = reinterpret_cast<uint64_t*>(smem + C::kOffBarK);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars_k + 18);
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tslot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 32 * 8) {
    for (int i = 0; i < 18; ++i) mbar_init(bars_k + i, i < 12 ? 1 : i < 17 ? 256 : 8);
    for (int i = 0; i < 21; ++i) mbar_init(bars_q + i, i >= 3 && i < 7 ? 256 : 1);
    fence_mbar_init();
  }
  Sequences<kMany> list;
  list.init(reinterpret_cast<int2*>(smem + C::kOffSeq), reinterpret_cast<int2*>(smem), p, kTile,
            p.kv_heads);
  fence_proxy_async_smem();  // (the list's scratch lies where copies will land)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  dkv_part<D>(maps, p, list, smem, tmem);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  list.parts = p.heads;
  list.me = (int)(gridDim.x - 1 - blockIdx.x);  // (the first blocks had the longest items)
  dq_part<D>(maps, p, list, smem, tmem);
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

template <int D, bool kMany>
static PackedTcKernels tc_kernels() {
  return PackedTcKernels{(const void*)packed_fwd_kernel<D, kMany>,
                         (const void*)packed_delta_kernel<D>,
                         (const void*)packed_bwd_kernel<D, kMany>, Fwd<D>::kSmem, Bwd<D>::kSmem};
}
PackedTcKernels packed_tc_kernels(int d, int64_t batch) {
  const bool many = batch > kSorted;
  return d == 64    ? many ? tc_kernels<64, true>() : tc_kernels<64, false>()
         : d == 128 ? many ? tc_kernels<128, true>() : tc_kernels<128, false>()
                    : PackedTcKernels{};
}

const char* packed_tc_fwd_launch(const PackedParams& p, int sms, cudaStream_t stream) {
  const PackedTcKernels k = packed_tc_kernels(p.dim, p.batch);
  CUtensorMap maps[4];
  if (!encode_map(&maps[0], p.q, p.tokens, p.heads, p.dim, p.sq, kTile) ||
      !encode_map(&maps[1], p.k, p.tokens, p.kv_heads, p.dim, p.sk, kTile) ||
      !encode_map(&maps[2], p.v, p.tokens, p.kv_heads, p.dim, p.sv, kTile) ||
      !encode_map(&maps[3], p.o, p.tokens, p.heads, p.dim, p.so, 32))
    return "tensor map encoding failed";
  const int64_t items = (p.tokens / kTile + p.batch) * p.heads;
  PackedParams pc = p;
  void* args[] = {&maps[0], &maps[1], &maps[2], &maps[3], &pc};
  if (cudaLaunchKernel(k.fwd, dim3((unsigned)std::min<int64_t>(sms, items)), dim3(384), args,
                       (size_t)k.fwd_smem, stream) != cudaSuccess)
    return "launch failed";
  return nullptr;
}

const char* packed_tc_bwd_launch(const PackedParams& p, int sms, cudaStream_t stream) {
  const PackedTcKernels k = packed_tc_kernels(p.dim, p.batch);
  BwdMaps maps;
  if (!encode_map(&maps.q, p.q, p.tokens, p.heads, p.dim, p.sq, kTile) ||
      !encode_map(&maps.k, p.k, p.tokens, p.kv_heads, p.dim, p.sk, kTile) ||
      !encode_map(&maps.v, p.v, p.tokens, p.kv_heads, p.dim, p.sv, kTile) ||
      !encode_map(&maps.g, p.dout, p.tokens, p.heads, p.dim, p.sdo, kTile) ||
      !encode_map(&maps.dk, p.dk, p.tokens, p.kv_heads, p.dim, p.sdk, 32) ||
      !encode_map(&maps.dv, p.dv, p.tokens, p.kv_heads, p.dim, p.sdv, 32))
    return "tensor map encoding failed";
  PackedParams pc = p;
  void* dargs[] = {&pc};
  if (cudaLaunchKernel(k.delta, dim3((unsigned)((p.tokens + 7) / 8)), dim3(256), dargs, 0,
                       stream) != cudaSuccess)
    return "launch failed";
  const int64_t levels = p.tokens / kTile + p.batch;
  void* args[] = {&maps, &pc};
  if (cudaLaunchKernel(k.bwd, dim3((unsigned)std::min<int64_t>(sms, levels * p.heads)), dim3(384),
                       args, (size_t)k.bwd_smem, stream) != cudaSuccess)
    return "launch failed";
  return nullptr;
}

}  // namespace rr
