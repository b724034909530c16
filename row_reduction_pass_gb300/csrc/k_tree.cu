// k_tree.cu -- attention of a tree of new tokens over a paged cache (the online
// softmax of k_attn.cu, with the query rows of one key head as the tile, and the
// keys cut into shares).
//
// The n * G rows (node, head of the group) of one sequence and key head share
// its keys, so they are the rows of a tile: 128 at a time, thread t of a softmax
// warpgroup owning row t.  The work is counted in key tiles of BN keys over all
// (sequence, key head, row tile) items in order, and every pipeline (two per
// SM) takes an equal run of them, whatever the lengths, which the host does not
// know.  The runs are runs of groups of up to 16 pipelines side by side, which
// work on the row tiles of the same keys (so the keys come from DRAM once: with
// the row tiles one after the other 8 x 62 tokens x 64 heads read 1.7 GB for
// 0.54 GB of cache) and on key heads of the same positions (which lie side by side
// in the cache: decode batch 215 -> 200 us); an item is (sequence, block of heads,
// block of row tiles).  An item inside one run is finished there; of an item cut by runs every
// piece leaves its unscaled output, maximum and sum in the workspace, and a
// second kernel joins the pieces.
//
// Bound: a key tile is read once per row tile (HBM: 44.7 GB/s a SM, 0.73 us per
// 32 KB tile of keys and values), its two products cost 128 rows whatever the
// number that is alive (0.3 us), so up to 128 rows a key head are HBM-bound and
// more are bound by the products and the softmax, as in k_attn.cu.
//
// The keys come through the page table as tensor-map boxes of [64 head
// dimensions x R positions x 1 head x 1 page], R the largest power of two that
// divides the page size, at most BN.  Tiles that reach past the context take a
// mask of 32 bits per 32 keys: the ancestors of the row's node (bits found by
// walking the parents once a piece), or the nodes up to it.  The rows of V at
// positions that no row may see are cleared in shared memory before the product,
// and so are non-finite values at nodes (0 x inf would be NaN for rows that do not
// see the node); rows that do see such a node get the values added at the end.
//
// The softmax weights are rounded to bf16 before P V, since both operands of that
// product have V's type (their sum stays in fp32): o is 0.0023 off float64 (2-norm), its
// own rounding to bf16 alone is 0.0017.  A weight split into two bf16 would double the
// product.
//
// Measured (in a graph): 64 sequences of 500-8000 keys, one token, 32 heads over 8 of
// 128: 171 us, 96 % of the copy bandwidth; one such sequence of 4001: 14.5 us, a
// piece's latency and the join's; 16 trees of 30 nodes, 16 heads over 4 of 64, over
// 1000-4100 keys 24.8 us, the same; 8 trees of 62 nodes, 64 heads over 8, over
// 12000-20000 keys 225 us, 57 % of the bf16 rate (k_attn.cu's 54 % on long causal
// heads): the pipelines' tiles follow one another every 1570 cycles, of which the
// softmax works 1250, and the issuers of S and P V are held 870 and 480 by the tensor
// pipe's queue.  Tried and slower there: half of Q in TMEM for less shared memory
// traffic (239 -> 242 us), Q copied asynchronously and O written in whole lines (240 ->
// 246 us; a pipeline's prologue and epilogue are the other's tiles' time).
//
// Page sizes that are not a multiple of 16 go to a kernel of one warp per query
// row, a key at a time: the 64 sequences above take 9.9 ms with a page size of 1, 9.7
// with 5.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "rr_device.cuh"
#include "rr_kernels.h"
#include "rr_tc.cuh"

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

// ------------------------------------------------------------ tensor cores ---

// 4-D TMA tile load [dst] <- map at {c0, c1, c2, c3}, completing bytes on bar.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, int c3, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "r"(smem_addr(bar))
      : "memory");
}

// The wait for this thread's tcgen05.ld, as an operation on the registers loaded, so
// that no use of them can be moved before it.
__device__ __forceinline__ void tmem_ld_done(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]),
                 "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                 "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}

constexpr int kTM = 128;  // rows of a tile: MMA M, TMEM lanes
// Two softmax warpgroups, and for each pipeline w a warp that issues S (8 + w), one
// for O += P V (10 + w), one that loads K (12 + w) and one that loads V (14 + w): a
// load takes its warp about 650 cycles, an issue 500-1000, and in one warp they
// delayed one another (one loader for both pipelines: decode batch 200 -> 234 us).
constexpr int kTreeThreads = 512;
constexpr int kMaskStride = kTreeMaxNodes / 32 + 1;  // mask words of a row, one spare

// Tiles, stages, TMEM columns (256 a pipeline: S, P buffers, O) as in k_attn.cu.
template <int D>
struct TreePL {
  static constexpr int BN = D == 64 ? 128 : 64;
  static constexpr int NS = 2;
  static constexpr int NPB = D == 128 ? 2 : 1;
  static constexpr int kBoxes = D / 64;
  static constexpr int kQBox = kTM * 128;
  static constexpr int kQBytes = kBoxes * kQBox;
  static constexpr int kKVBox = BN * 128;
  static constexpr int kKVBytes = kBoxes * kKVBox;
  static constexpr int kPipe = kQBytes + NS * 2 * kKVBytes;
  static constexpr int kOffMask = 2 * kPipe;
  static constexpr int kOffPar = kOffMask + 2 * kTM * kMaskStride * 4;  // [2][256] parents
  static constexpr int kOffBar = kOffPar + 2 * kTreeMaxNodes * 4;
  static constexpr int kOffScan = kOffBar + 512;
  static constexpr int kSmem = kOffScan + 256 + 1024;
  static constexpr uint32_t kColS = 0, kColP = BN, kColO = 256 - D;
  static constexpr uint32_t kIdescS = attn_idesc(kTM, BN, false);
  static constexpr uint32_t kIdescO = attn_idesc(kTM, D, true);
};

// A piece: the key tiles [t0, t1) of an item, t1 - t0 of its T tiles.
struct TreeSeg {
  int left;   // tiles of the run from t0 on
  int b, hm, t0, t1, T;
  int ctx;    // keys before the nodes
  int vis;    // positions below it may be seen by some row of the tile
  int tiles;  // tiles to work on: those of [t0, t1) below vis
  int h, mt;  // key head and row tile of item hm
};

// keys before the nodes (nodes past the table are not seen wherever they are)
__device__ __forceinline__ int tree_context(const TreeParams& p, const TreeGeo& g, int b) {
  return min(max(__ldg(p.length + b), 0), g.cap);
}
// key tiles of a sequence
template <int BN>
__device__ __forceinline__ int tree_tiles(const TreeParams& p, const TreeGeo& g, int ctx) {
  return (min(ctx + p.nodes, g.cap) + BN - 1) / BN;
}
// position / page size, and the rest: a shift for the usual powers of two (a
// division costs an issuing warp about 300 cycles a tile)
__device__ __forceinline__ int tree_page(const TreeParams& p, const TreeGeo& g, int pos) {
  return g.page_shift >= 0 ? pos >> g.page_shift : pos / p.page;
}
__device__ __forceinline__ int tree_page_row(const TreeParams& p, const TreeGeo& g, int pos) {
  return g.page_shift >= 0 ? pos & (p.page - 1) : pos % p.page;
}

// How the tiles are cut into runs, one for each group of pipelines.
//   flat: run i is tiles [i share, (i + 1) share) of all, across items.
//   own (few items): every item is cut into pieces of at most `share` tiles of its
//     own, a piece a run.  No run then pays for a second piece (its own queries,
//     first products, output: about kTreePieceTiles tiles), so this is taken where
//     its longest run is at most that much longer than the flat one: 16 sequences of
//     1000-4100 keys, 30 nodes, head_dim 64: the slowest pipeline 42000 -> 24000
//     cycles.
struct TreePlan {
  int share;
  bool own;
};
constexpr int kTreePieceTiles = 3;
constexpr int kTreeWarpSeqs = 320;  // a warp plans up to these many; more are always flat

__device__ __forceinline__ int tree_cdiv(int a, int b) { return (a + b - 1) / b; }
__device__ __forceinline__ int warp_isum(int v) {
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

// Sequence b's tiles (0 past the last sequence).  The planning loops read the
// lengths again each time: they stay in the first-level cache, and rolled loops keep
// the code short, which is fetched once per call.
template <int BN>
__device__ __forceinline__ int tree_tiles_of(const TreeParams& p, const TreeGeo& g, int b) {
  return b < (int)p.batch ? tree_tiles<BN>(p, g, tree_context(p, g, b)) : 0;
}
template <int BN>
__device__ __forceinline__ TreePlan tree_plan(const TreeParams& p, const TreeGeo& g) {
  const int lane = threadIdx.x & 31, batch = (int)p.batch;
  int sum = 0, some = 0;
#pragma unroll 1
  for (int b = lane; b < batch; b += 32) {
    const int T = tree_tiles_of<BN>(p, g, b);
    sum += T;
    some += T > 0;
  }
  sum = warp_isum(sum) * g.KM;
  some = warp_isum(some) * g.KM;
  TreePlan plan{max(tree_cdiv(sum, g.groups), g.min_tiles), false};
  if (some > g.groups) return plan;
  // the least share, at most kTreePieceTiles above the flat one, whose pieces are no
  // more than the groups
#pragma unroll 1
  for (int share = plan.share; share <= plan.share + kTreePieceTiles; ++share) {
    int n = 0;
#pragma unroll 1
    for (int b = lane; b < batch; b += 32) n += tree_cdiv(tree_tiles_of<BN>(p, g, b), share);
    if (warp_isum(n) * g.KM <= g.groups) return TreePlan{share, true};
  }
  return plan;
}
// A sequence's units: the plan's runs if they are items' own, else its tiles.
template <int BN>
__device__ __forceinline__ int tree_units(const TreeParams& p, const TreeGeo& g,
                                          const TreePlan& plan, int b) {
  const int T = tree_tiles_of<BN>(p, g, b);
  return (plan.own ? tree_cdiv(T, plan.share) : T) * g.KM;
}
// The sequence that holds unit `at`, and how many are before it in *before; -1 past
// the end.
template <int BN>
__device__ __forceinline__ int tree_find(const TreeParams& p, const TreeGeo& g,
                                         const TreePlan& plan, int64_t at, int* before) {
  const int lane = threadIdx.x & 31;
  int base = 0;
#pragma unroll 1
  for (int b = 0; b < (int)p.batch; b += 32) {
    const int v = tree_units<BN>(p, g, plan, b + lane);
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, off);
      if (lane >= off) x += y;
    }
    const uint32_t m = __ballot_sync(0xffffffffu, base + x > at);
    if (m != 0) {
      const int l = __ffs(m) - 1;
      *before = base + __shfl_sync(0xffffffffu, x - v, l);
      return b + l;
    }
    base += __shfl_sync(0xffffffffu, x, 31);
  }
  return -1;
}

template <int D>
__device__ __forceinline__ void tree_seg_fill(TreeSeg& s, const TreeParams& p, const TreeGeo& g) {
  constexpr int BN = TreePL<D>::BN;
  s.t1 = min(s.T, s.t0 + s.left);
  int last = p.nodes - 1;  // the tile's last node
  if (p.parents == nullptr && g.MT > 1) last = min(last, (s.mt * kTM + kTM - 1) / g.G);
  s.vis = min(s.ctx + last + 1, g.cap);
  s.tiles = max(0, min(s.t1, (s.vis + BN - 1) / BN) - s.t0);
}
// A run's first piece, from its item hm: head, row tile, tiles.
template <int D>
__device__ __forceinline__ void tree_seg_place(TreeSeg& s, const TreeParams& p, const TreeGeo& g,
                                               int sub) {
  const int mb = g.MT / g.RB, hb = s.hm / mb;
  s.h = hb * g.HB + sub / g.RB;
  s.mt = (s.hm - hb * mb) * g.RB + sub % g.RB;
  tree_seg_fill<D>(s, p, g);
}
template <int D>
__device__ __forceinline__ bool tree_seg_next(TreeSeg& s, const TreeParams& p, const TreeGeo& g) {
  s.left -= s.t1 - s.t0;
  if (s.left <= 0) return false;
  s.t0 = 0;
  if ((s.mt += g.RB) >= g.MT) {
    s.mt -= g.MT;
    s.h += g.HB;
  }
  if (++s.hm == g.KM) {
    s.hm = 0;
    s.h -= p.kv_heads;
    do {  // (a sequence of no tiles has no items; tiles are left, so one comes)
      if (++s.b >= p.batch) return false;
      s.ctx = tree_context(p, g, s.b);
      s.T = tree_tiles<TreePL<D>::BN>(p, g, s.ctx);
    } while (s.T == 0);
  }
  tree_seg_fill<D>(s, p, g);
  return true;
}

// The sum over the block's threads before this one, and over all (in *total);
// scratch of 16 values.
__device__ __forceinline__ int tree_scan(int v, int* scratch, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll 4
  for (int i = 0; i < nw; ++i) {
    if (i < warp) before += scratch[i];
    all += scratch[i];
  }
  __syncthreads();
  *total = all;
  return before + x - v;
}

__device__ __forceinline__ bool odd_bf16x2(uint32_t w) {  // an infinity or NaN in the pair
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// The workspace: two pieces a pipeline (its run's first and last), a piece being
// [D / 4][rows] 16-byte chunks of the output (so that the rows of a warp write, and
// the joining threads read, whole lines), behind them the pieces' [rows] (maximum,
// sum), and behind those the plan: its share, whether the runs are items' own, and
// the units before each sequence.
template <int D>
__device__ __forceinline__ int32_t* tree_ws_plan(const TreeParams& p, const TreeGeo& g) {
  const int64_t rows = min(p.nodes * g.G, kTM);
  return reinterpret_cast<int32_t*>(p.ws + (int64_t)g.max_slots * 2 * rows * (D + 2));
}
template <int D>
__global__ void __launch_bounds__(kTreeThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                   const __grid_constant__ TreeParams p, const TreeGeo g) {
  using C = TreePL<D>;
  constexpr int BN = C::BN;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int w = warp < 8 ? warp >> 2 : warp & 1;  // this thread's pipeline
  unsigned char* pipe = smem + w * C::kPipe;
  unsigned char* sq = pipe;
  auto stage_k = [&](int s) { return pipe + C::kQBytes + (2 * s) * C::kKVBytes; };
  auto stage_v = [&](int s) { return pipe + C::kQBytes + (2 * s + 1) * C::kKVBytes; };
  uint32_t* masks = reinterpret_cast<uint32_t*>(smem + C::kOffMask) + w * kTM * kMaskStride;
  int32_t* spar = reinterpret_cast<int32_t*>(smem + C::kOffPar) + w * kTreeMaxNodes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + w * 16;
  uint64_t* bar_q = bars + 0;       // Q written, 128 arrivals
  uint64_t* bar_s = bars + 1;       // S done
  uint64_t* bar_sfree = bars + 2;   // S read, 128 arrivals
  uint64_t* bar_ofree = bars + 3;   // O read, 128 arrivals
  uint64_t* bar_p = bars + 4;       // [NPB] P written, 128 arrivals
  uint64_t* bar_o = bars + 6;       // [NPB] O += P V done with the P buffer
  uint64_t* bar_kfull = bars + 8;   // [2]
  uint64_t* bar_vfull = bars + 10;  // [2]
  uint64_t* bar_kempty = bars + 12; // [2] S done with the K stage
  uint64_t* bar_vempty = bars + 14; // [2] O += P V done with the V stage
  uint64_t* extra = reinterpret_cast<uint64_t*>(smem + C::kOffBar) + 40;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(extra);
  int* odd = reinterpret_cast<int*>(extra + 1) + w;  // the last piece with a non-finite V row
  TreeSeg* firsts = reinterpret_cast<TreeSeg*>(extra + 4);  // [2]
  int* scratch = reinterpret_cast<int*>(smem + C::kOffScan);

  const int slot0 = 2 * (int)blockIdx.x;
  // the joining grid may be set up now (it waits for this one before it reads)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tslot)),
                 "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if ((warp == 8 || warp == 9) && lane == 0) {
    mbar_init(bar_q, 128);
    mbar_init(bar_s, 1);
    mbar_init(bar_sfree, 128);
    mbar_init(bar_ofree, 128);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_p[i], 128);
      mbar_init(&bar_o[i], 1);
      mbar_init(&bar_kfull[i], 1);
      mbar_init(&bar_vfull[i], 1);
      mbar_init(&bar_kempty[i], 1);
      mbar_init(&bar_vempty[i], 1);
    }
    fence_mbar_init();
    *odd = 0;
  }
  // where the pipelines' runs begin: a loading warp of each plans (the others only
  // read the result: a plan in every warp cost the softmax loop registers)
  if (p.batch <= kTreeWarpSeqs) {
    if (warp == 12 || warp == 13) {
      TreeSeg sg;
      sg.left = 0;
      const int grp = (slot0 + w) / g.side;
      if (grp < g.groups) {
        int before = 0;
        const TreePlan plan = tree_plan<BN>(p, g);
        const int64_t at = plan.own ? grp : (int64_t)grp * plan.share;
        const int b = tree_find<BN>(p, g, plan, at, &before);
        if (b >= 0) {
          sg.b = b;
          sg.ctx = tree_context(p, g, b);
          sg.T = tree_tiles<BN>(p, g, sg.ctx);
          const int off = (int)at - before;
          if (plan.own) {
            const int n = tree_cdiv(sg.T, plan.share);
            sg.hm = off / n;
            sg.t0 = (off - sg.hm * n) * plan.share;
            sg.left = min(plan.share, sg.T - sg.t0);
          } else {
            sg.hm = off / sg.T;
            sg.t0 = off - sg.hm * sg.T;
            sg.left = plan.share;  // (the sequences end, or the run does)
          }
          tree_seg_place<D>(sg, p, g, slot0 + w - grp * g.side);
        }
      }
      if (lane == 0) firsts[w] = sg;
    }
  } else {
    // many sequences: each thread counts the tiles of some, and the one that holds a
    // run's first tile writes it down
    const int batch = (int)p.batch, per = (batch + kTreeThreads - 1) / kTreeThreads;
    const int b0 = tid * per, b1 = min(b0 + per, batch);
    int mine = 0, total;
    if (tid < 2) firsts[tid].left = 0;  // (before the scan's barriers)
    for (int b = b0; b < b1; ++b) mine += tree_tiles<BN>(p, g, tree_context(p, g, b)) * g.KM;
    const int at = tree_scan(mine, scratch, &total);
    const int share = max(tree_cdiv(total, g.groups), g.min_tiles);
    if (blockIdx.x == 0) {  // the plan, for the join
      int32_t* plan = tree_ws_plan<D>(p, g);
      if (tid == 0) plan[0] = share, plan[1] = 0;
      int before = at;
      for (int b = b0; b < b1; ++b) {
        plan[2 + b] = before;
        before += tree_tiles<BN>(p, g, tree_context(p, g, b)) * g.KM;
      }
    }
    for (int s = 0; s < 2; ++s) {
      const int gs = (slot0 + s) / g.side;
      const int64_t start = (int64_t)gs * share;
      if (gs >= g.groups || start < at || start >= (int64_t)at + mine) continue;
      int off = (int)start - at;
      for (int b = b0; b < b1; ++b) {
        TreeSeg sg;
        sg.ctx = tree_context(p, g, b);
        sg.T = tree_tiles<BN>(p, g, sg.ctx);
        const int n = sg.T * g.KM;
        if (off >= n) {
          off -= n;
          continue;
        }
        sg.left = share;
        sg.b = b;
        sg.hm = off / sg.T;
        sg.t0 = off - sg.hm * sg.T;
        tree_seg_place<D>(sg, p, g, slot0 + s - gs * g.side);
        firsts[s] = sg;
        break;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *tslot + 256u * w;
  const TreeSeg first = firsts[w];
  bool dead = false;  // a wait gave up: no further waits (the kernel still ends)
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!dead) dead = !mbar_wait_bounded(bar, parity, p.err);
  };
  // a pipeline's tiles in order: tile t0 + j of a piece
  struct Cur {
    TreeSeg s;
    int j;
    bool ok;
  };
  auto settle = [&](Cur& c) {  // to the next piece that has tiles
    while (c.ok && c.s.tiles == 0) c.ok = tree_seg_next<D>(c.s, p, g);
    c.j = 0;
  };
  auto advance = [&](Cur& c) {
    if (++c.j < c.s.tiles) return;
    c.ok = tree_seg_next<D>(c.s, p, g);
    settle(c);
  };
  auto begin = [&](const TreeSeg& s) {
    Cur c{s, 0, s.left > 0};
    settle(c);
    return c;
  };

  int copies = 0;  // tiles that this loader has asked for
  if (first.left <= 0) {
    // no run for this pipeline
  } else if (warp >= 12) {
    // ------------------------------------------------------ the loaders
    // Tiles of K or V through the page table: K(n) goes where S(n - 2) has read its
    // keys, V(n) where O += P V of n - 2 has.  Lane i loads box i, whose page it
    // looks up one tile ahead.
    const bool isv = warp >= 14;
    const CUtensorMap* map = isv ? &tv : &tk;
    uint64_t* full = isv ? bar_vfull : bar_kfull;
    uint64_t* empty = isv ? bar_vempty : bar_kempty;
    unsigned char* stage = isv ? stage_v(0) : stage_k(0);
    Cur c = begin(first);
    int page = 0;
    auto box_pos = [&]() { return (c.s.t0 + c.j) * BN + lane * g.box; };
    auto look_up = [&]() {
      if (!c.ok) return;
      const int pos = box_pos();
      if (lane * g.box < BN && pos < c.s.vis) {
        page = __ldg(p.table + (int64_t)c.s.b * p.width + tree_page(p, g, pos));
        if (page < 0 || page >= p.pages) page = (int)p.pages;  // out of range: zeros
      }
    };
    look_up();
    for (int n = 0; c.ok; ++n) {
      const int s = n & 1;
      if (n >= 2) wait_spin(&empty[s], (uint32_t)((n / 2 - 1) & 1), dead, p.err);
      if (__any_sync(0xffffffffu, dead)) break;
      const int key0 = (c.s.t0 + c.j) * BN, pos = box_pos();
      const int boxes = min(BN, c.s.vis - key0 + g.box - 1) >> g.box_shift;  // that hold keys
      if (lane == 0)
        mbar_arrive_expect_tx(&full[s], (uint32_t)(boxes * g.box * C::kBoxes * 128));
      __syncwarp();
      if (lane < boxes) {
        unsigned char* dst = stage + s * 2 * C::kKVBytes + lane * g.box * 128;
#pragma unroll
        for (int b = 0; b < C::kBoxes; ++b)
          tma_load_4d(dst + b * C::kKVBox, map, 64 * b, c.s.h, tree_page_row(p, g, pos), page,
                      &full[s]);
      }
      copies = n + 1;
      advance(c);
      look_up();
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------ the issuers
    if (lane == 0) {
      Cur c = begin(first);
      int pieces = 0;  // begun
      int issued = 0;
      // (the products end before the block does, also after a wait gave up)
      auto finish = [&](uint64_t* bar, uint32_t parity) {
        if (issued > 0) mbar_wait_bounded(bar, parity, p.err);
      };
      if (warp >= 10) {
        // O += P V as soon as P is written (the first of a piece, which overwrites
        // O, once the softmax has read it)
        for (int t = 0; c.ok && !dead; ++t) {
          if (c.j == 0 && pieces++ > 0) wait_spin(bar_ofree, (uint32_t)(pieces & 1), dead, p.err);
          wait_spin(&bar_p[t % C::NPB], (uint32_t)((t / C::NPB) & 1), dead, p.err);
          wait_spin(&bar_vfull[t & 1], (uint32_t)((t >> 1) & 1), dead, p.err);
          if (dead) break;
          const uint32_t v_addr = smem_addr(stage_v(t & 1));
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk)
            mma_ts(tm + C::kColO, tm + C::kColP + (t % C::NPB) * (BN / 2) + 8 * kk,
                   sw128_desc(v_addr + kk * 2048, C::kKVBox, 1024), C::kIdescO,
                   (c.j > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&bar_o[t % C::NPB]);
          mma_commit(&bar_vempty[t & 1]);
          issued = t + 1;
          advance(c);
        }
        finish(&bar_o[(issued + C::NPB - 1) % C::NPB], (uint32_t)(((issued - 1) / C::NPB) & 1));
      } else {
        // S = Q K^T as soon as the softmax has read the S before (a new piece's Q is
        // then there)
        for (int t = 0; c.ok && !dead; ++t) {
          wait_spin(&bar_kfull[t & 1], (uint32_t)((t >> 1) & 1), dead, p.err);
          if (c.j == 0) wait_spin(bar_q, (uint32_t)(pieces++ & 1), dead, p.err);
          if (t >= 1) wait_spin(bar_sfree, (uint32_t)((t - 1) & 1), dead, p.err);
          if (dead) break;
          const uint32_t q_addr = smem_addr(sq), k_addr = smem_addr(stage_k(t & 1));
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t qo = (uint32_t)((kk >> 2) * C::kQBox + (kk & 3) * 32);
            const uint32_t ko = (uint32_t)((kk >> 2) * C::kKVBox + (kk & 3) * 32);
            mma_ss(tm + C::kColS, sw128_desc(q_addr + qo, 16, 1024),
                   sw128_desc(k_addr + ko, 16, 1024), C::kIdescS, kk > 0 ? 1u : 0u);
          }
          mma_commit(bar_s);
          mma_commit(&bar_kempty[t & 1]);
          issued = t + 1;
          advance(c);
        }
        finish(bar_s, (uint32_t)((issued - 1) & 1));
      }
    }
  } else {
    // ------------------------------------------------ softmax warpgroup
    const int row = tid & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tm + lane_base + C::kColS;
    const uint32_t tO = tm + lane_base + C::kColO;
    const float sc = p.scale_log2;
    const int slot = slot0 + w;
    const int all_rows = p.nodes * g.G, ws_rows = min(all_rows, kTM);
    uint4* ws_o = reinterpret_cast<uint4*>(p.ws);
    float2* ws_ml = reinterpret_cast<float2*>(p.ws + (int64_t)g.max_slots * 2 * ws_rows * D);
    uint32_t* mask = masks + row * kMaskStride;
    TreeSeg s = first;
    int t = 0;        // tiles done by this pipeline
    int piece = 0;    // pieces seen
    bool more = true;
    for (; more; more = tree_seg_next<D>(s, p, g)) {
      const bool cut0 = piece == 0 && s.t0 > 0, cut1 = s.t1 < s.T;
      ++piece;
      const int h = s.h, mt = s.mt;
      const int R = mt * kTM + row;
      const bool live = R < all_rows;
      const bool wlive = mt * kTM + 32 * (warp & 3) < all_rows;  // some row of this warp
      const int node = live ? R / g.G : 0, head = h * g.G + (live ? R - node * g.G : 0);
      const int64_t out = ((int64_t)s.b * p.nodes + node) * p.heads + head;
      bool present = live;
      float m = -INFINITY, l = 0.f;
      if (s.tiles > 0) {
        // The piece's loads are asked for together: parents, Q, the table's entries.
        int up0 = 0, up1 = 0;
        if (p.parents != nullptr) {
          const int32_t* par = p.parents + (int64_t)s.b * p.nodes;
          if (row < p.nodes) up0 = __ldg(par + row);
          if (row + 128 < p.nodes) up1 = __ldg(par + row + 128);
        }
        // Q into the swizzled tile, a warp its 32 rows, whole rows at a time (a row per
        // lane would touch 32 lines an instruction); zeros for the rows of a live warp
        // beyond the last
        if (wlive) {
#pragma unroll 4
          for (int i = 0; i < D / 8; ++i) {
            const int at = i * 32 + lane, r = at / (D / 8), c = at % (D / 8);
            const int64_t from = __shfl_sync(0xffffffffu, out, r);
            const bool on = __shfl_sync(0xffffffffu, (int)live, r);
            const int qr = 32 * (warp & 3) + r;
            *reinterpret_cast<uint4*>(sq + (c >> 3) * C::kQBox + qr * 128 +
                                      (((c & 7) ^ (qr & 7)) << 4)) =
                on ? __ldg(reinterpret_cast<const uint4*>(p.q + from * D * 2) + c)
                   : make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(bar_q);
        // pages that do not exist: none in the pieces of a sound table
        bool holes = false;
        {
          const int last = min((s.t0 + s.tiles) * BN, s.vis) - 1;
          for (int i = tree_page(p, g, s.t0 * BN) + lane; i <= tree_page(p, g, last); i += 32) {
            const int page = __ldg(p.table + (int64_t)s.b * p.width + i);
            holes = holes || page < 0 || page >= p.pages;
          }
          holes = __any_sync(0xffffffffu, holes);
        }
        if (p.parents != nullptr) {
          // the bits of this row's node and its ancestors
          named_bar(1 + w, 128);  // (the parents of the piece before have been used)
          if (row < p.nodes) spar[row] = up0;
          if (row + 128 < p.nodes) spar[row + 128] = up1;
          for (int i = 0; i < kMaskStride; ++i) mask[i] = 0;
          named_bar(1 + w, 128);
          for (int a = node; a >= 0 && present;) {
            mask[a >> 5] |= 1u << (a & 31);
            const int up = spar[a];
            if (up < -1 || up >= a) present = false;
            a = up;
          }
        }
        // Tiles wholly inside the context go through a copy of the loop's body without
        // masks (a loop that carried them: large trees 235 -> 256 us).
        bool tail_seen = false;
        auto tile = [&](auto masked_c, int j) {
          constexpr bool masked = decltype(masked_c)::value;
          const int key0 = (s.t0 + j) * BN;
          const bool tail = masked && key0 + BN > min(s.ctx, s.vis);
          // which of the tile's keys this row sees, 32 to a word
          uint32_t seen[BN / 32];
          if constexpr (masked) {
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) {
              const int pos = key0 + 32 * c;  // of bit 0
              const int nb = pos - s.ctx;     // its node
              uint32_t bits = 0xffffffffu;
              if (p.parents != nullptr) {
                if (nb >= 0)
                  bits = nb >> 5 < kMaskStride - 1
                             ? __funnelshift_r(mask[nb >> 5], mask[(nb >> 5) + 1], nb & 31)
                             : 0u;
                else if (nb > -32)
                  bits = (mask[0] << -nb) | ((1u << -nb) - 1u);
              }
              const int lim = p.parents != nullptr ? s.vis : min(s.ctx + node + 1, s.vis);
              if (lim - pos <= 0) bits = 0;
              else if (lim - pos < 32) bits &= (1u << (lim - pos)) - 1u;
              if (holes) {
                for (int i = 0; i < 32; i += 16) {
                  if (pos + i >= s.vis) break;
                  const int page =
                      __ldg(p.table + (int64_t)s.b * p.width + tree_page(p, g, pos + i));
                  if (page < 0 || page >= p.pages) bits &= ~(0xffffu << i);
                }
              }
              seen[c] = bits;
            }
          }
          wait(bar_s, (uint32_t)(t & 1));
          tc_fence_after();
          if (wlive) {
            // S in halves of 64 columns: at BN = 128 the first is read again for its
            // exponentials (both at once are 128 registers, and spilled)
            uint32_t v[2][32];
            auto read_half = [&](int hf) {
#pragma unroll
              for (int c = 0; c < 2; ++c) tmem_ld32_nowait(tS + 64 * hf + 32 * c, v[c]);
              tmem_ld_done(v[0]);
              tmem_ld_done(v[1]);
              if constexpr (masked) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                  for (int i = 0; i < 32; ++i)
                    if (!((seen[2 * hf + c] >> i) & 1)) v[c][i] = __float_as_uint(-INFINITY);
              }
            };
            auto max_half = [&](float mx) {
              float x[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) x[k] = -INFINITY;
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i & 7] = fmaxf(x[i & 7], __uint_as_float(v[c][i]));
              return fmaxf(fmaxf(mx, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]))),
                           fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
            };
            float mx = -INFINITY;
            if constexpr (BN == 128) {
              read_half(0);
              mx = max_half(mx);
            }
            read_half(BN / 64 - 1);
            if constexpr (BN == 64) {
              tc_fence_before();
              mbar_arrive(bar_sfree);
            }
            mx = max_half(mx);
            // m moves only by more than 8 (k_attn.cu); a row that has seen no key
            // keeps m = -inf and takes its exponentials (all 0) from 0
            const float mt_ = mx * sc;
            const float m_new = mt_ > m + 8.f ? mt_ : m;
            const float alpha = m_new == m ? 1.f : ex2(m - m_new);
            const float mref = m_new == -INFINITY ? 0.f : m_new;
            float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
            const uint32_t tP = tm + lane_base + C::kColP + (t % C::NPB) * (BN / 2);
            bool p_free = t < C::NPB;
            auto exp_half = [&](int hf) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                  float t0, t1, t2, t3;
                  fma2(t0, t1, __uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1]), sc, sc,
                       -mref, -mref);
                  fma2(t2, t3, __uint_as_float(v[c][i + 2]), __uint_as_float(v[c][i + 3]), sc, sc,
                       -mref, -mref);
                  const float p0 = ex2(t0), p1 = ex2(t1), p2 = ex2(t2), p3 = ex2(t3);
                  add2(l0, l1, l0, l1, p0, p1);
                  add2(l2, l3, l2, l3, p2, p3);
                  pk[i >> 1] = pack_bf16(p0, p1);
                  pk[(i >> 1) + 1] = pack_bf16(p2, p3);
                }
                if (!p_free) {  // O += P V of tile t - NPB has read this P buffer
                  wait(&bar_o[t % C::NPB], (uint32_t)((t / C::NPB - 1) & 1));
                  tc_fence_after();
                  p_free = true;
                }
                tmem_st16(tP + 32 * hf + 16 * c, pk);
              }
            };
            exp_half(BN / 64 - 1);
            if constexpr (BN == 128) {
              read_half(0);
              tc_fence_before();
              mbar_arrive(bar_sfree);
              exp_half(0);
            }
            l = l * alpha + ((l0 + l1) + (l2 + l3));
            m = m_new;
            if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
              if constexpr (C::NPB > 1) {
                wait(&bar_o[(t - 1) % C::NPB], (uint32_t)(((t - 1) / C::NPB) & 1));
                tc_fence_after();
              }
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32_nowait(tO + 32 * c, o);
                tmem_ld_done(o);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  float a0, a1;
                  mul2(a0, a1, __uint_as_float(o[i]), __uint_as_float(o[i + 1]), alpha, alpha);
                  o[i] = __float_as_uint(a0);
                  o[i + 1] = __float_as_uint(a1);
                }
                tmem_st32(tO + 32 * c, o);
              }
            }
            tmem_st_wait();
          } else {
            tc_fence_before();
            mbar_arrive(bar_sfree);
            // a warp without rows keeps pace: its arrival below must not fall into
            // the P buffer's previous phase
            if (t >= C::NPB) wait(&bar_o[t % C::NPB], (uint32_t)((t / C::NPB - 1) & 1));
          }
          if (tail) {
            // V at positions nobody may see, and non-finite values at nodes: 0
            // (This barrier is not waited on at every tile, and the products may be two
            // tiles behind: V(t - 2) may not even have landed, and the wait for V(t)'s
            // phase would then be satisfied by the phase before V(t - 2)'s.  So first
            // the product that reads V(t - 2).)
            tail_seen = true;
            if (t >= 2) wait(&bar_vempty[t & 1], (uint32_t)(((t >> 1) - 1) & 1));
            wait(&bar_vfull[t & 1], (uint32_t)((t >> 1) & 1));
            const int vr = row % BN, pos = key0 + vr;
            if (pos >= s.ctx || pos >= s.vis) {
              uint4* vp =
                  reinterpret_cast<uint4*>(stage_v(t & 1) + row / BN * C::kKVBox + vr * 128);
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                uint4 x = vp[c];
                if (pos >= s.vis) {
                  vp[c] = make_uint4(0u, 0u, 0u, 0u);
                } else if (odd_bf16x2(x.x) || odd_bf16x2(x.y) || odd_bf16x2(x.z) ||
                           odd_bf16x2(x.w)) {
                  for (int i = 0; i < 4; ++i) {
                    uint32_t y = word_of(x, i);
                    if ((y & 0x7f80u) == 0x7f80u) y &= 0xffff0000u;
                    if ((y & 0x7f800000u) == 0x7f800000u) y &= 0xffffu;
                    set_word(x, i, y);
                  }
                  vp[c] = x;
                  *odd = piece;
                }
              }
            }
            fence_proxy_async_smem();
          }
          tc_fence_before();
          mbar_arrive(&bar_p[t % C::NPB]);
        };
        const int inside = holes ? 0 : min(s.tiles, max(0, min(s.ctx, s.vis) / BN - s.t0));
        int j = 0;
        for (; j < inside; ++j, ++t) tile(std::false_type{}, j);
        for (; j < s.tiles; ++j, ++t) tile(std::true_type{}, j);
        wait(&bar_o[(t - 1) % C::NPB], (uint32_t)(((t - 1) / C::NPB) & 1));
        tc_fence_after();
        if (tail_seen) named_bar(1 + w, 128);  // every thread's look at V
        const bool fix = tail_seen && *odd == piece && present;
        if (!present) {
          m = -INFINITY;
          l = 0.f;
        }
        const bool whole = !cut0 && !cut1;
        const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
        const int part = 2 * slot + (piece > 1);  // the run's first piece, or its last
        // O in 32 columns at a time (few registers: the loop above keeps the rest)
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          if (!wlive) break;
          uint32_t o[32];
          tmem_ld32_nowait(tO + 32 * c, o);
          tmem_ld_done(o);
          if (l == 0.f) {  // (nothing seen: the accumulator holds nothing of this row's)
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
          if (__builtin_expect(fix, 0)) {
            // Adds the non-finite values of V that this row sees (rare: rolled loops over
            // a copy in this warp's rows of the Q tile, which no product reads any more and
            // no other warp writes; a function of its own made the whole kernel 5 % slower,
            // calls being costly to allocate around)
            float* f = reinterpret_cast<float*>(sq + (warp & 3) * 32 * 128) + lane;
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i * 32] = __uint_as_float(o[i]);
            const int hi = min((s.t0 + s.tiles) * BN, s.vis);
#pragma unroll 1
            for (int pos = max(s.ctx, s.t0 * BN); pos < hi; ++pos) {
              const int j = pos - s.ctx;
              if (p.parents != nullptr ? !((mask[j >> 5] >> (j & 31)) & 1) : j > node) continue;
              const int page = __ldg(p.table + (int64_t)s.b * p.width + tree_page(p, g, pos));
              if (page < 0 || page >= p.pages) continue;
              const int64_t at =
                  ((int64_t)page * p.page + tree_page_row(p, g, pos)) * p.kv_heads + h;
              const char* v = p.v + (at * D + 32 * c) * 2;
#pragma unroll 1
              for (int i = 0; i < 32; ++i) {
                const float x = ld_elem_cached<kBF16>(v + 2 * i);
                if (!(fabsf(x) < INFINITY)) f[i * 32] += x;
              }
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(f[i * 32]);
          }
          __syncwarp();  // (the next piece's Q goes over f)
          if (live && whole) {
            uint4* dst = reinterpret_cast<uint4*>(p.o + (out * D + 32 * c) * 2);
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              dst[i >> 3] = make_uint4(
                  pack_bf16(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv),
                  pack_bf16(__uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv),
                  pack_bf16(__uint_as_float(o[i + 4]) * inv, __uint_as_float(o[i + 5]) * inv),
                  pack_bf16(__uint_as_float(o[i + 6]) * inv, __uint_as_float(o[i + 7]) * inv));
          } else if (live) {
            uint4* dst = ws_o + ((int64_t)part * (D / 4) + 8 * c) * ws_rows + row;
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              dst[(i >> 2) * ws_rows] = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        tc_fence_before();
        mbar_arrive(bar_ofree);
        if (live && whole && p.lse != nullptr)
          p.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        if (live && !whole) ws_ml[(int64_t)part * ws_rows + row] = make_float2(m, l);
      } else if (live) {
        // nothing of these tiles is visible to the row tile
        if (cut0 || cut1)
          ws_ml[(int64_t)(2 * slot + (piece > 1)) * ws_rows + row] = make_float2(-INFINITY, 0.f);
      }
    }
  }

  // The plan, for the join (whose blocks each made it again: large trees 240 -> 229 us),
  // by a warp that has loaded all its keys.
  if (p.batch <= kTreeWarpSeqs && blockIdx.x == 0 && warp == 12) {
    int32_t* out = tree_ws_plan<D>(p, g);
    const TreePlan plan = tree_plan<BN>(p, g);
    if (lane == 0) out[0] = plan.share, out[1] = plan.own;
    int base = 0;
#pragma unroll 1
    for (int b = lane; b - lane < (int)p.batch; b += 32) {
      const int v = tree_units<BN>(p, g, plan, b);
      int x = v;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      if (b < (int)p.batch) out[2 + b] = base + x - v;
      base += __shfl_sync(0xffffffffu, x, 31);
    }
  }

  // Copies end before the block does (they have, but where a wait gave up).
  for (int n = max(copies - 2, 0); n < copies; ++n)
    mbar_wait_bounded(&(warp >= 14 ? bar_vfull : bar_kfull)[n & 1], (uint32_t)((n >> 1) & 1), p.err);
  tc_fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(*tslot), "r"(512u)
                 : "memory");
}

// Joins the pieces of items cut by runs (the plan says which), and writes the rows
// of sequences that have no tile at all.  A thread takes one 16-byte chunk of one
// row, over all pieces (eight threads, each some of the pieces: one token 14.4 -> 14.0
// us, but 16 trees of 30 nodes 24.3 -> 24.8).
constexpr int kJoinT = 256;
template <int D>
__global__ void __launch_bounds__(kJoinT) tree_join_kernel(const TreeParams p, const TreeGeo g) {
  constexpr int BN = TreePL<D>::BN;
  const int tid = threadIdx.x;
  // block (x, z): item x of all, pipeline z of its group
  const int b = (int)blockIdx.x / g.KM, hm = (int)blockIdx.x - b * g.KM;
  const int tiles = tree_tiles<BN>(p, g, tree_context(p, g, b));
  const int all_rows = p.nodes * g.G, ws_rows = min(all_rows, kTM);
  const int flat = (int)blockIdx.y * kJoinT + tid;  // of the piece's chunks
  const int chunk = flat / ws_rows, row = flat - chunk * ws_rows;
  const int sub = (int)blockIdx.z, mb = g.MT / g.RB, hb = hm / mb;
  const int h = hb * g.HB + sub / g.RB, mt = (hm - hb * mb) * g.RB + sub % g.RB;
  const int R = mt * kTM + row, node = R / g.G;
  const int64_t out = ((int64_t)b * p.nodes + node) * p.heads + h * g.G + R - node * g.G;
  // Launched while the pieces are still being computed: every block waits for
  // them here, also one without work, so that this grid ends after that one.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the item's first run, the runs that hold a piece of it, the first one's piece
  int run0 = 0, n = 0, skip = 0;
  if (tiles > 0) {
    const int32_t* plan = tree_ws_plan<D>(p, g);
    const int share = plan[0], before = plan[2 + b];
    if (plan[1]) {
      n = tree_cdiv(tiles, share);
      run0 = before + hm * n;
    } else {
      const int start = before + hm * tiles;
      run0 = start / share;
      n = (start + tiles - 1) / share - run0 + 1;
      skip = run0 * share < start;
    }
  }
  if (n == 1) return;  // finished by its run
  if (chunk >= D / 4 || R >= all_rows) return;
  const float4* ws_o = reinterpret_cast<const float4*>(p.ws);
  const float2* ws_ml =
      reinterpret_cast<const float2*>(p.ws + (int64_t)g.max_slots * 2 * ws_rows * D);
  // an item's piece in a run is the run's last if it begins inside the run: its first
  auto part = [&](int i) { return 2 * ((run0 + i) * g.side + sub) + (i == 0 ? skip : 0); };
  float M = -INFINITY, L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  // pieces loaded at once: 8, or 2 where there are no more (an unused place costs as
  // much as a used one: large trees 232 -> 229 us)
  auto add = [&](auto at_once, int i0) {
    constexpr int U = decltype(at_once)::value;
    float2 ml[U];
    float4 x[U];
    float mx = M;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + i < n) {
        const int64_t pt = part(i0 + i);
        ml[i] = ws_ml[pt * ws_rows + row];
        x[i] = ws_o[(pt * (D / 4) + chunk) * ws_rows + row];
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) mx = fmaxf(mx, ml[i].x);
    const float keep = M == mx ? 1.f : ex2(M - mx);
    M = mx;
    L *= keep;
    o = make_float4(o.x * keep, o.y * keep, o.z * keep, o.w * keep);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (ml[i].y == 0.f) continue;  // a piece in which the row sees nothing: no output there
      const float a = ml[i].x == M ? 1.f : ex2(ml[i].x - M);
      L = fmaf(ml[i].y, a, L);
      o = make_float4(fmaf(x[i].x, a, o.x), fmaf(x[i].y, a, o.y), fmaf(x[i].z, a, o.z),
                      fmaf(x[i].w, a, o.w));
    }
  };
  if (n == 2) add(std::integral_constant<int, 2>{}, 0);
  else
    for (int i0 = 0; i0 < n; i0 += 8) add(std::integral_constant<int, 8>{}, i0);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  *reinterpret_cast<uint2*>(p.o + (out * D + 4 * chunk) * 2) =
      make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (chunk == 0 && p.lse != nullptr) p.lse[out] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

}  // namespace

const void* tree_rows_kernel(int d) {
  return d == 64    ? (const void*)tree_rows_kernel_t<64>
         : d == 128 ? (const void*)tree_rows_kernel_t<128>
                    : nullptr;
}

TreeKernels tree_kernels(int d) {
  if (d == 64)
    return {(const void*)tree_tc_kernel<64>, (const void*)tree_join_kernel<64>, kTreeThreads,
            TreePL<64>::kSmem, TreePL<64>::BN};
  return {(const void*)tree_tc_kernel<128>, (const void*)tree_join_kernel<128>, kTreeThreads,
          TreePL<128>::kSmem, TreePL<128>::BN};
}

const char* tree_tc_launch(const TreeParams& p, int d, int sms, cudaStream_t stream) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  if (encode == nullptr) return "cuTensorMapEncodeTiled is not available from the driver";
  const TreeKernels tk = tree_kernels(d);
  TreeGeo g{};
  g.box = 16;
  while (g.box < tk.bn && p.page % (2 * g.box) == 0) g.box *= 2;
  g.box_shift = 4;
  while ((1 << g.box_shift) < g.box) ++g.box_shift;
  g.page_shift = -1;
  for (int i = 4; i < 31; ++i)
    if (p.page == (1 << i)) g.page_shift = i;
  g.min_tiles = kTreeMinTiles;
  g.G = p.heads / p.kv_heads;
  const int64_t rows = (int64_t)p.nodes * g.G, mt = (rows + kTM - 1) / kTM;
  g.MT = (int)mt;
  // side by side: the most row tiles, then the most key heads, up to 16 in all
  g.RB = g.HB = 1;
  for (int i = 2; i <= 16; ++i)
    if (g.MT % i == 0) g.RB = i;
  for (int i = 2; i * g.RB <= 16; ++i)
    if (p.kv_heads % i == 0) g.HB = i;
  g.side = g.HB * g.RB;
  g.KM = p.kv_heads / g.HB * (g.MT / g.RB);
  g.cap = (int)(p.width * p.page);
  CUtensorMap maps[2];
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)p.kv_heads, (cuuint64_t)p.page,
                              (cuuint64_t)p.pages};
  const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)p.kv_heads * d * 2,
                                 (cuuint64_t)p.page * p.kv_heads * d * 2};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)g.box, 1}, es[4] = {1, 1, 1, 1};
  for (int i = 0; i < 2; ++i)
    if (encode(&maps[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<char*>(i ? p.v : p.k),
               dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return "tensor map encoding failed";
  g.max_slots = 2 * sms;
  g.groups = g.max_slots / g.side;
  TreeParams pc = p;
  void* args[] = {&maps[0], &maps[1], &pc, &g};
  if (cudaLaunchKernel(tk.main, dim3((unsigned)sms), dim3((unsigned)tk.threads), args,
                       (size_t)tk.smem, stream) != cudaSuccess)
    return "launch failed";
  void* jargs[] = {&pc, &g};
  const int64_t items = p.batch * g.KM;
  const unsigned groups =
      (unsigned)((std::min<int64_t>(rows, kTM) * (d / 4) + kJoinT - 1) / kJoinT);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)items, groups, (unsigned)g.side);
  cfg.blockDim = dim3(kJoinT);
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelExC(&cfg, tk.join, jargs) != cudaSuccess) return "join launch failed";
  return nullptr;
}

size_t tree_ws_bytes(int64_t batch, int64_t nodes, int heads, int kv_heads, int d, int sms) {
  const int64_t rows = std::min<int64_t>(nodes * (heads / kv_heads), kTM);
  return ((size_t)(2 * sms) * 2 * rows * (d + 2) + 2 + batch) * sizeof(float);
}

}  // namespace rr
