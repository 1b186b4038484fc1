// Attention over the bf16 paged cache for ragged chunks of new tokens, and for
// trees of windowed layers, on the 5th-generation tensor cores.
//
// What it computes.  A row (token i of sequence b, query head h) at position p
// sees the cached keys t with  t < limit  and, with a window,  t > p - window or
// t < sinks;  its output is softmax(scale q.k) v over them.
//   chunk: the rows are the last tokens of the cache itself, p = kv - len + i and
//          limit = p + 1 (causal);
//   tree:  the rows are tree nodes past a verified prefix, p = P + depth and
//          limit = P; the tree's own keys follow, gated by the ancestry mask (and
//          by the window, counted in depths).
//
// How.  The G query heads of a KV head share every key, so ROW_TILE / G tokens
// of G heads are the 128 rows of one MMA tile.  A work item is such a tile of one
// KV head and a split of its chain of 128-key tiles; only tiles that some row
// sees are in the chain: the sinks' tiles, then the window's.  One online softmax
// runs over the chain, and k_join_paged joins the splits of a cut chain.
//
// The kernel is persistent, one CTA an SM taking items from a counter, the
// longest first, with one role a warp, as tree attention's:
//   warp 0      takes the items (and hands them to the others through a queue in
//               shared memory); TMA loads of the K tiles
//   warp 3      TMA loads of the V tiles
//   warp 1      S(j) = Q K(j)^T, once PV has freed the S buffer
//   warp 2      O += P(j) V(j), P from TMEM
//   warps 4-11  softmax, two groups of 128 threads, each with an accumulator O, a
//               reference and a sum of its own, so that neither waits for the other.
// What a group takes:
//   heads of 128   half the keys of every tile: two O leave room for two S buffers only,
//                  and a tile's way through softmax, PV and the next QK has to be short.
//   heads of 64    every other tile; or, of a PAIR of row tiles that share each key
//                  tile, its own row tile, where the plan expects pairs to end sooner (it
//                  has a second row tile, and enough items).
// But for pairs, the groups are joined at an item's end, and each stores half of the channels.
//
// What bounds it.  Long chains of heads of 128: the tensor cores under the power cap
// (4096 tokens over 16K, 32 heads: 613-625 us in bursts, 1.55 PFLOP/s, 0.83 of the
// measured GEMM rate; 652-677 us back to back).  Heads of 64 have half the products for the
// same softmax, which then sets the pace (64 heads, 4 x 1024 tokens over 8K: 475-510 us, by
// the chip's heat, 1.0-1.08 PFLOP/s).  What it was before a tile's largest weight was looked for
// (at SUM_LIMIT): 449, without pairs 472 with blocks of 64, and 559 with blocks of 16, where
// it is the issue of 16 TMA boxes a tile.  The kernels of heads of 64 spill 28 to 88 bytes a
// thread at their cap of 168 registers, the trees' of 128 twelve, the chunks' none.  Single
// tokens: memory (32 sequences of 0-8K: 81 us, 6.2 TB/s, 0.91 of the measured copy).  An
// item costs 2 to 3 us beyond its tiles: the start of its pipeline, the last PV, the
// stores.  What carried it (64 heads of
// 128 and of 64 on 64 trees of 64 nodes over 8K, us):
//   one softmax group, 128 columns a thread                       848  823
//   two groups                                                    958  700
//   the issuers' loops run by whole warps on uniform values,
//     descriptors by offset, one elected lane issuing             778  684
//   each box issued by the lane that holds its place              788  620
//   heads of 64: tiles in turn, no look at a tile's maximum                592
// Tried and not kept: a barrier asked for a tile ahead (a poll that is not needed
// delays the warp: 671 -> 698); one lane issuing all boxes (656 -> 724); the groups held
// apart by half a period (580 -> 602); one P arrival a warp (no change); three-input
// maxima (no change: the compiler's own).  Pairs of heads of 128: 675 -> 825.  On pairs of
// heads of 64 (455): loads of 32 columns a step ahead 520, of 128 at once 564 (spills).
// Heads of 128 with one accumulator, shared references and three S buffers: 4K of 16K 611
// -> 597, 8 prompts of 512 35 -> 50.
//
// Masks cost nothing where a tile is wholly visible; elsewhere each row makes
// a word of its visible keys.  Keys that no row of the item sees may be
// anything, so their V rows are zeroed in shared memory before PV reads them
// (0 * NaN), and blocks that hold only such keys are not read at all: a
// windowed layer may have given them away.
//
// Every wait is bounded; a wait that runs out sets a flag, all roles wind down,
// let their loads and MMAs in flight finish, free the tensor memory and report
// TS_ERR_TIMEOUT for the sequences of the items they had not finished.
#include <algorithm>
#include <climits>
#include <cmath>

#include "attn_paged.cuh"
#include "fastexp.cuh"
#include "tensor_map.cuh"
#include "waits.cuh"

namespace ts {
namespace {

constexpr int NUM_THREADS = 384;
constexpr int GROUP_THREADS = 128;  // a softmax group: a row a thread
constexpr int K_WARP = 0, QK_WARP = 1, PV_WARP = 2, V_WARP = 3, SOFTMAX_WARP0 = 4, SOFTMAX_WARPS = 8;
constexpr int HALF = KV_TILE / 2;  // keys of a tile that one softmax group takes
constexpr uint32_t TMEM_COLS = 512;
// A row's weights are taken against a reference, the maximum of the first keys it
// sees, and may reach 2^40 of it (their precision does not depend on that).  Then the
// reference is raised and the sums are scaled down.
constexpr float RESCALE_THRESHOLD = 40.0f;
constexpr float SUM_LIMIT = 1099511627776.f;  // 2^40
// The weights are rounded to bf16 for the product with the values (half a step, 2^-8 of
// each at most) and summed before that, in fp32, for the log-sum-exp.  A weight that
// outweighs the others is seldom 1, so its rounding would be the output's; outputs are
// divided by a sum that takes the largest weight of each tile (of its half of one, where the
// groups share it) as rounded, and that error cancels.  With a hundredth of the keys eight
// times the others, outputs are off by 1.6e-3 to 1.7e-3 of themselves, 1.5e-3 to 1.6e-3 being
// their own rounding; 2.1e-3 to 2.3e-3 with the plain sum.  Summing all the rounded weights
// gives no less.  Heads of 128 know the largest score already; heads of 64 look for it, one
// instruction in six of the softmax: 2K prompts with a window 294 -> 311 us (361 with the sum
// of all, which takes heads of 128 from 614 to 648 on 4K of 16K).
constexpr float NEG_INF = -INFINITY;

template <int D, bool PAIR>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int TILE_BYTES = KV_TILE * D * 2;
  static constexpr int HALF_BYTES = KV_TILE * 128;
  static constexpr int Q_BYTES = ROW_TILE * D * 2;  // of a row tile
  static constexpr int SETS = PAIR ? 2 : 1;         // row tiles an item
  static constexpr int NST = D == 128 ? 3 : PAIR ? 5 : 6;  // tiles in each ring, K and V
  static constexpr int ITEM_Q = D == 128 ? 4 : 8;          // entries of the item queue: what shared memory leaves
  static_assert(D == 64 || !PAIR, "");
  // The two softmax groups: a row tile each of a pair; else on heads of 64 the key
  // tiles in turn, on heads of 128 half the keys of every tile each.
  static constexpr bool TURNS = PAIR || D == 64;
  // TMEM: the groups' accumulators at 0 and D, then the S buffers
  static constexpr uint32_t TMEM_S0 = 2 * D;
  static constexpr int NSB = (TMEM_COLS - TMEM_S0) / KV_TILE;  // 2 for heads of 128, 3 for 64
};

template <int D, bool PAIR>
struct __align__(1024) Smem {
  using C = Cfg<D, PAIR>;
  uint8_t q[C::SETS * C::Q_BYTES];
  uint8_t k[C::NST][C::TILE_BYTES];
  uint8_t v[C::NST][C::TILE_BYTES];
  uint64_t q_full, q_empty;
  uint64_t k_full[C::NST], v_full[C::NST];
  uint64_t k_empty[C::NST], v_empty[C::NST];
  uint64_t s_full[C::NSB], p_full[C::NSB][2], s_free[C::NSB];
  uint64_t o_last;  // an item's last PV has completed
  uint64_t ml_full, f_full, o_free;  // an item's end: see ml; both groups have read the accumulators
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort_flag;
  // the CTA's items in the order taken; pub published, done by how many softmax warps
  // they were stored (no warp is more than one item ahead of another)
  int4 item_q[C::ITEM_Q][4];
  int items_pub, items_done;
  // an item's end: group 1's (m, l) of each row, then from group 0 the factors of
  // both accumulators (1 KB each way would not fit beside heads of 128); and what group
  // 1's accumulator is to be divided by
  float2 ml[ROW_TILE];
  float norm[ROW_TILE];
};

struct KArgs {
  PagedArgs a;
  int box_rows, n_items, n_seqs, out32;
  FastDiv fd_hkv, fd_bs, fd_g;
  PagedSeq seq[PAGED_MAX_SEQS];
  PagedGaps gaps;
};

// Entry of an item: the last with item0 <= it.
__device__ __forceinline__ int entry_of(int it, const KArgs& t) {
  int lo = 0, hi = t.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.seq[mid].item0 <= it) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

struct Place {
  int e, rt, split, g;
};
__device__ __forceinline__ Place place_of(int it, const KArgs& t) {
  Place p;
  p.e = entry_of(it, t);
  const int k = it - t.seq[p.e].item0;
  const int u = t.fd_hkv.div(k);
  p.g = k - u * t.a.Hkv;
  const int back = u / t.seq[p.e].splits;
  p.split = u - back * t.seq[p.e].splits;
  p.rt = t.seq[p.e].row_tiles - 1 - back;
  return p;
}

// An item as the roles take it; four int4 of the queue.
struct Item {
  int b, g, split, e;
  int q0, i0, len, pos0;  // the tile's first row is token q0 + i0, the i0-th of len, at position pos0 (tree: the root's)
  int lo, hi, n_sink, win0;  // PagedSpan
  int t_begin, n_prefix, n_tiles, ps;  // n_tiles 0: nothing to do, or no more items
};
template <bool TREE>
__device__ __forceinline__ Item make_item(const Place& p, int b, int q0, int len, int kv, const KArgs& t) {
  const PagedArgs& a = t.a;
  Item I;
  I.b = b;
  I.g = p.g;
  I.split = p.split;
  I.e = p.e;
  I.q0 = q0;
  I.len = len;
  I.i0 = p.rt * a.tok;
  I.pos0 = TREE ? kv : kv - len + I.i0;
  const PagedSpan sp = TREE ? paged_span(kv, kv, a.window, a.sinks) : chunk_span(kv, len, I.i0, a.tok, a.window, a.sinks);
  I.lo = sp.lo;
  I.hi = sp.hi;
  I.n_sink = sp.n_sink;
  I.win0 = sp.win0;
  I.ps = paged_splits(sp.n, a.chunk_tiles, t.seq[p.e].splits);
  I.t_begin = paged_split_start(sp.n, I.ps, p.split);
  I.n_prefix = paged_split_start(sp.n, I.ps, p.split + 1) - I.t_begin;
  I.n_tiles = I.n_prefix + (TREE && p.split == I.ps - 1 ? ceil_div(a.N, KV_TILE) : 0);
  if (I.i0 >= len || p.split >= I.ps) I.n_tiles = 0;
  return I;
}
// First key of the item's prefix tile j.
__device__ __forceinline__ int tile_key(const Item& I, int j) {
  const int jj = I.t_begin + j;
  return (jj < I.n_sink ? jj : jj - I.n_sink + I.win0) * KV_TILE;
}

// The lengths of sequence b as the device has them.
struct Lens {
  int q0, len, kv;
  bool ok;  // they are what the launch was planned for, and the rows are in the cache
};
__device__ __forceinline__ int ld_early(const int* p) {  // issued where it is written
  int v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(reinterpret_cast<uint64_t>(p)) : "memory");
  return v;
}
template <bool TREE>
__device__ __forceinline__ Lens load_lens(int b, int planned, const PagedArgs& a) {
  Lens l;
  l.kv = ld_early(a.kv_len + b);
  const long long cap = min((long long)a.max_blocks * a.bs, 1ll << 30);
  if (TREE) {
    l.q0 = b * a.N;
    l.len = a.N;
    l.ok = l.kv >= 0 && l.kv <= cap;
  } else {
    l.q0 = ld_early(a.cu_len + b);
    const int q1 = ld_early(a.cu_len + b + 1), in_cache = a.appended ? ld_early(a.appended + b) : INT_MAX;
    l.ok = l.q0 >= 0 && q1 >= l.q0 && q1 <= a.T && q1 - l.q0 <= planned;
    l.len = l.ok ? q1 - l.q0 : 0;
    l.ok = l.ok && l.kv >= l.len && l.kv <= cap && in_cache >= l.len;
  }
  if (!l.ok) l.len = 0;  // nothing of it is read or written
  return l;
}

// One thread: sequence b is refused, unless it has an error already.
__device__ __forceinline__ void refuse(int32_t* status, int b) {
  if (status && status[b] == TS_OK) status[b] = TS_ERR_SHAPE;
}

// One thread: those of [c0, c1), planned without rows, that have some by now.
__device__ __forceinline__ void refuse_gap(const PagedArgs& a, int c0, int c1) {
  if (c0 >= c1 || a.cu_len[c0] == a.cu_len[c1]) return;
  for (int c = c0; c < c1; ++c)
    if (a.cu_len[c] != a.cu_len[c + 1]) refuse(a.status, c);
}
// At the first item of entry e: its neighbours.
template <bool TREE>
__device__ __forceinline__ void refuse_gaps(int e, const KArgs& t) {
  if (TREE || !t.a.status) return;
  const int b = t.seq[e].b;
  refuse_gap(t.a, t.gaps.before[e], b);
  if (b == t.gaps.last) refuse_gap(t.a, b + 1, t.gaps.end);
}

// The first n bits of a 64-bit word.
__device__ __forceinline__ uint64_t first_bits(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// One 32-byte store (a whole DRAM sector), to a 32-byte aligned address.
__device__ __forceinline__ void st_v8(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(reinterpret_cast<uint64_t>(p)),
               "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

template <int D, bool TREE, bool PAIR>
__global__ void __launch_bounds__(NUM_THREADS, 1)
k_attn_paged(const __grid_constant__ KArgs args, const __grid_constant__ CUtensorMap tm_q,
             const __grid_constant__ CUtensorMap tm_kc, const __grid_constant__ CUtensorMap tm_vc,
             const __grid_constant__ CUtensorMap tm_kt, const __grid_constant__ CUtensorMap tm_vt) {
  using C = Cfg<D, PAIR>;
  constexpr int NSB = C::NSB;
  constexpr uint32_t TMEM_S0 = C::TMEM_S0;
  extern __shared__ uint8_t smem_raw[];
  Smem<D, PAIR>& sm = *reinterpret_cast<Smem<D, PAIR>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const PagedArgs& a = args.a;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const bool leader = elect_one();  // one lane of the warp
  const Ctl ctl{&sm.abort_flag, a.wait_limit_ns};
  const int n_items = args.n_items;

  const Place pl0 = place_of(blockIdx.x, args);
  const int b0 = args.seq[pl0.e].b;
  if (warp == V_WARP && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_kc);
    tma_prefetch_desc(&tm_vc);
    if (TREE) {
      tma_prefetch_desc(&tm_kt);
      tma_prefetch_desc(&tm_vt);
    }
  }
  if (threadIdx.x == 0) {
    sm.abort_flag = 0;
    sm.items_pub = 0;
    sm.items_done = 0;
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_empty[i], 1);
    }
    for (int i = 0; i < NSB; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i][0], GROUP_THREADS);
      mbar_init(&sm.p_full[i][1], GROUP_THREADS);
      mbar_init(&sm.s_free[i], 1);
    }
    mbar_init(&sm.o_last, 1);
    mbar_init(&sm.ml_full, GROUP_THREADS);
    mbar_init(&sm.f_full, GROUP_THREADS);
    mbar_init(&sm.o_free, 2 * GROUP_THREADS);
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    fence_barrier_init();
  }
  if (warp == K_WARP) tmem_alloc(&sm.tmem_base, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  // nothing above read an input
  pdl_wait();
  // With a CTA an item nothing is taken from the counter and nothing goes through
  // the queue: every role reads the lengths itself.
  const bool single = (int)gridDim.x == n_items;
  const bool grabber = warp == K_WARP && !single;
  Lens l0{0, 0, 0, false};
  if (single || grabber) l0 = load_lens<TREE>(b0, args.seq[pl0.e].rows, a);
  if (single && threadIdx.x == 0) {
    if (!l0.ok) refuse(a.status, b0);
    if ((int)blockIdx.x == args.seq[pl0.e].item0) refuse_gaps<TREE>(pl0.e, args);
  }
  const Item item0 = make_item<TREE>(pl0, b0, l0.q0, l0.len, l0.kv, args);

  // Entry k of the queue (every role but the K producer; with a CTA an item every
  // role).  false: the wait gave up.
  auto queue_item = [&](int k, Item& I) -> bool {
    if (single) {
      I = item0;
      if (k > 0) I.n_tiles = 0;
      return true;
    }
    if (!wait_count(&sm.items_pub, k + 1, ctl)) return false;
    const int4* q = sm.item_q[k % C::ITEM_Q];
    const int4 x = q[0], y = q[1], z = q[2], w = q[3];
    I = Item{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w, w.x, w.y, w.z, w.w};
    return true;
  };
  // The K producer's lane 0: the next item, or -1.  The last of all requests puts
  // the counter back to zero.
  auto take_item = [&]() -> int {
    const unsigned v = atomicAdd(a.sched, 1u);
    if (v == (unsigned)(n_items - 1)) atomicExch(a.sched, 0u);
    const int it = (int)gridDim.x + (int)v;
    return it < n_items ? it : -1;
  };
  int held = -1;             // an item taken and not published yet
  bool exhausted = single;   // the counter said that none is left

  auto kv_producer = [&](bool is_v) -> int {
    const CUtensorMap* tm_pool = is_v ? &tm_vc : &tm_kc;
    const CUtensorMap* tm_node = is_v ? &tm_vt : &tm_kt;
    uint64_t* full = is_v ? sm.v_full : sm.k_full;
    uint64_t* empty = is_v ? sm.v_empty : sm.k_empty;
    const int g_box = args.box_rows;
    const int lg_boxes = __ffs(KV_TILE / g_box) - 1;  // 1 .. 8 boxes a tile
    const int n_boxes = 1 << lg_boxes, tpg = 32 >> lg_boxes;
    const uint32_t box_bytes = g_box * D * 2;
    const int koff = (lane & (n_boxes - 1)) * g_box;  // this lane's box of a tile
    int slot = 0, phase = 0;
    int jg = 0;  // tiles issued, over every item
    int cand = blockIdx.x;
    Place cpl = pl0;
    Lens cl = l0;
    if (grabber) held = cand;
    for (int k = 0;; ++k) {
      Item I;
      if (grabber) {
        I.n_tiles = 0;
        for (;;) {
          if (cand < 0) break;
          if (lane == 0) {
            if (!cl.ok) refuse(a.status, args.seq[cpl.e].b);
            if (cand == args.seq[cpl.e].item0) refuse_gaps<TREE>(cpl.e, args);
          }
          I = make_item<TREE>(cpl, args.seq[cpl.e].b, cl.q0, cl.len, cl.kv, args);
          if (I.n_tiles) break;
          int nx = -1;
          if (lane == 0) nx = take_item();
          cand = __shfl_sync(0xffffffffu, nx, 0);
          held = cand;
          exhausted = cand < 0;
          if (cand >= 0) {
            cpl = place_of(cand, args);
            cl = load_lens<TREE>(args.seq[cpl.e].b, args.seq[cpl.e].rows, a);
          }
        }
        bool ok = k < C::ITEM_Q;  // the entry's last user must be done
        if (!ok && lane == 0) ok = wait_count(&sm.items_done, SOFTMAX_WARPS * (k - C::ITEM_Q + 1), ctl);
        if (!__shfl_sync(0xffffffffu, ok, 0)) return jg;
        if (lane == 0) {
          int4* q = sm.item_q[k % C::ITEM_Q];
          q[0] = make_int4(I.b, I.g, I.split, I.e);
          q[1] = make_int4(I.q0, I.i0, I.len, I.pos0);
          q[2] = make_int4(I.lo, I.hi, I.n_sink, I.win0);
          q[3] = make_int4(I.t_begin, I.n_prefix, I.n_tiles, I.ps);
          publish(&sm.items_pub, k + 1);
          if (I.n_tiles)  // its queries, into L2, while the last item's keys are still at work
            for (int x = 0; x < C::SETS && I.i0 + x * a.tok_tile < I.len; ++x)
              for (int h = 0; h < C::HALVES; ++h)
                tma_prefetch_3d(&tm_q, 64 * h, I.g * a.G, I.q0 + I.i0 + x * a.tok_tile);
        }
        __syncwarp();
        held = -1;
        if (cand < 0) return jg;
        // take the next one now: its lengths load while this one streams
        int nx = -1;
        if (lane == 0) nx = take_item();
        cand = __shfl_sync(0xffffffffu, nx, 0);
        held = cand;
        exhausted = cand < 0;
        if (cand >= 0) {
          cpl = place_of(cand, args);
          cl = load_lens<TREE>(args.seq[cpl.e].b, args.seq[cpl.e].rows, a);
        }
      } else {
        const bool ok = queue_item(k, I);
        if (!__all_sync(0xffffffffu, ok)) return jg;
        if (I.n_tiles == 0) return jg;
      }
      const int b = I.b, n_prefix = I.n_prefix;
      const int* table_row = a.block_table + (size_t)b * a.max_blocks;
      // Block-table entries, a group of tiles ahead: lane L holds that of box
      // L % boxes of tile L / boxes of a group of 32 / boxes tiles, and makes the
      // box's place in the pool of it when the group's turn comes.  A box that no row
      // of the item sees into is not read.
      auto load_group = [&](int grp) -> int {
        const int j = grp * tpg + (lane >> lg_boxes);
        if (j >= n_prefix) return INT_MIN;
        const int t0 = tile_key(I, j) + koff;
        if (t0 >= I.hi || (t0 + g_box <= I.lo && t0 >= a.sinks)) return INT_MIN;
        const int blk = table_row[args.fd_bs.div(t0)];
        return blk == INT_MIN ? -1 : blk;
      };
      int raw = load_group(0);
      int at8 = -1;  // its rows in the pool, in groups of 8
      unsigned boxes = 0;  // which lanes' are read
      const int stop = !is_v && b == a.stall_seq ? a.stall_tile : I.n_tiles;
      for (int j = 0; j < I.n_tiles; ++j, ++jg) {
        uint8_t* dst = is_v ? sm.v[slot] : sm.k[slot];
        const int jt = j & (tpg - 1);
        if (jt == 0 && j < n_prefix) {
          const int grp = j >> (5 - lg_boxes);
          at8 = -1;
          if (raw != INT_MIN) {
            if (raw < 0 || raw >= a.num_blocks) {
              if (a.status) a.status[b] = TS_ERR_BAD_BLOCK;
              raw = 0;  // a valid block is read in its place
            }
            const int row = args.fd_bs.mod(tile_key(I, grp * tpg + (lane >> lg_boxes)) + koff);
            at8 = (raw * a.Hkv + I.g) * (a.bs >> 3) + (row >> 3);
          }
          boxes = __ballot_sync(0xffffffffu, at8 >= 0);
          raw = (grp + 1) * tpg < n_prefix ? load_group(grp + 1) : INT_MIN;
        }
        if (jg >= C::NST && !__all_sync(0xffffffffu, wait_bar(&empty[slot], phase ^ 1, ctl))) return jg;
        if (j == stop) return jg;
        if (j < n_prefix) {
          // the lanes that hold this tile's boxes issue them (bytes that land before
          // they are announced count all the same)
          if (leader) mbar_arrive_expect_tx(&full[slot], __popc((boxes >> (jt << lg_boxes)) & ((1u << n_boxes) - 1)) * box_bytes);
          if ((lane >> lg_boxes) == jt && at8 >= 0)
            tma_load_4d(dst + (lane & (n_boxes - 1)) * box_bytes, tm_pool, &full[slot], 0, 0, 0, at8);
        } else if (leader) {
          const int n0 = (j - n_prefix) * KV_TILE;  // nodes >= N read as zeros
          mbar_arrive_expect_tx(&full[slot], C::TILE_BYTES);
          for (int h = 0; h < C::HALVES; ++h) tma_load_4d(dst + h * C::HALF_BYTES, tm_node, &full[slot], 64 * h, I.g, n0, b);
        }
        __syncwarp();
        if (++slot == C::NST) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
  };
  int issued = 0;
  int q_issued = 0, q_landed = 0;

  if (warp == K_WARP || warp == V_WARP) {
    issued = kv_producer(warp == V_WARP);
  } else if (warp == QK_WARP) {
    // The whole warp runs the issuers' loops, on values that are the same on every
    // lane, and one lane issues: descriptors then stay in uniform registers.
    constexpr uint32_t ID_QK = idesc_bf16_f32(ROW_TILE, KV_TILE, 0, 0);
    const uint64_t q_desc = smem_desc_sw128(smem_u32(sm.q), 16, 1024);
    // cached tiles: [8-row group][64-column half]; tree tiles: [half][rows]
    const uint64_t k_desc = smem_desc_sw128(smem_u32(sm.k[0]), 16, C::HALVES * 1024);
    const uint64_t kt_desc = smem_desc_sw128(smem_u32(sm.k[0]), 16, 1024);
    int slot = 0, k_phase = 0, buf = 0, s_phase = 1;  // (the first NSB waits for s_free pass)
    bool ok = true;
    for (int k = 0; ok; ++k) {
      Item I;
      if (!__all_sync(0xffffffffu, queue_item(k, I))) break;
      const int n_tiles = __shfl_sync(0xffffffffu, I.n_tiles, 0), n_prefix = __shfl_sync(0xffffffffu, I.n_prefix, 0);
      if (n_tiles == 0) break;
      // this item's Q tile, once every QK of the last one has completed
      if (k > 0 && !__all_sync(0xffffffffu, wait_bar(&sm.q_empty, (k - 1) & 1, ctl))) break;
      if (leader) {
        mbar_arrive_expect_tx(&sm.q_full, C::SETS * C::Q_BYTES);
        for (int x = 0; x < C::SETS; ++x)
          for (int h = 0; h < C::HALVES; ++h)
            tma_load_3d(sm.q + x * C::Q_BYTES + h * (ROW_TILE * 128), &tm_q, &sm.q_full, 64 * h, I.g * a.G,
                        I.q0 + I.i0 + x * a.tok_tile);
      }
      __syncwarp();
      ++q_issued;
      if (!__all_sync(0xffffffffu, wait_bar(&sm.q_full, k & 1, ctl))) break;
      ++q_landed;
      for (int v = 0; v < C::SETS * n_tiles; ++v) {
        const int j = v / C::SETS, x = v % C::SETS;
        ok = __all_sync(0xffffffffu, (x > 0 || wait_bar(&sm.k_full[slot], k_phase, ctl)) &&
                                         wait_bar(&sm.s_free[buf], s_phase, ctl));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem + TMEM_S0 + buf * KV_TILE;
        const uint64_t qd = q_desc + x * (C::Q_BYTES >> 4);
        if (leader) {
          if (!TREE || j < n_prefix) {
            const uint64_t kd = k_desc + slot * (C::TILE_BYTES >> 4);
#pragma unroll
            for (int k2 = 0; k2 < D / 16; ++k2)
              mma_ss(d_tmem, qd + (((k2 >> 2) * (ROW_TILE * 128) + (k2 & 3) * 32) >> 4),
                     kd + (((k2 >> 2) * 1024 + (k2 & 3) * 32) >> 4), ID_QK, k2 > 0);
          } else {
            const uint64_t kd = kt_desc + slot * (C::TILE_BYTES >> 4);
#pragma unroll
            for (int k2 = 0; k2 < D / 16; ++k2)
              mma_ss(d_tmem, qd + (((k2 >> 2) * (ROW_TILE * 128) + (k2 & 3) * 32) >> 4),
                     kd + (((k2 >> 2) * C::HALF_BYTES + (k2 & 3) * 32) >> 4), ID_QK, k2 > 0);
          }
          mma_commit(&sm.s_full[buf]);
          if (x == C::SETS - 1) mma_commit(&sm.k_empty[slot]);
        }
        __syncwarp();
        if (x == C::SETS - 1 && ++slot == C::NST) {
          slot = 0;
          k_phase ^= 1;
        }
        if (++buf == NSB) {
          buf = 0;
          s_phase ^= 1;
        }
      }
      if (ok && leader) mma_commit(&sm.q_empty);
      __syncwarp();
    }
  } else if (warp == PV_WARP) {
    constexpr uint32_t ID_PV = idesc_bf16_f32(ROW_TILE, D, 0, 1);
    const uint64_t v_desc = smem_desc_sw128(smem_u32(sm.v[0]), 1024, C::HALVES * 1024);
    const uint64_t vt_desc = smem_desc_sw128(smem_u32(sm.v[0]), C::HALF_BYTES, 1024);
    int slot = 0, v_phase = 0, buf = 0, p_phase = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      Item I;
      if (!__all_sync(0xffffffffu, queue_item(k, I))) break;
      const int n_tiles = __shfl_sync(0xffffffffu, I.n_tiles, 0), n_prefix = __shfl_sync(0xffffffffu, I.n_prefix, 0);
      if (n_tiles == 0) break;
      if (k > 0 && !__all_sync(0xffffffffu, wait_bar(&sm.o_free, (k - 1) & 1, ctl))) break;
      for (int v = 0; v < C::SETS * n_tiles; ++v) {
        const int j = v / C::SETS;
        const bool last = v % C::SETS == C::SETS - 1;  // of the tile's uses
        const uint32_t p_tmem = tmem + TMEM_S0 + buf * KV_TILE;
        const bool tree = TREE && j >= n_prefix;
        const uint64_t vd = (tree ? vt_desc : v_desc) + slot * (C::TILE_BYTES >> 4);
        const int acc = C::TURNS ? (v & 1) * D : 0;  // (halves: the second half's is D)
        const bool fresh = v < (C::TURNS ? 2 : 1);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!C::TURNS || half == 0) {
            ok = __all_sync(0xffffffffu, wait_bar(&sm.p_full[buf][half], p_phase, ctl) &&
                                             (half || wait_bar(&sm.v_full[slot], v_phase, ctl)));
            if (!ok) break;
            tc_fence_after();
          }
          if (leader) {
            const uint32_t o = tmem + (C::TURNS ? acc : half * D);
            if (!tree) {
#pragma unroll
              for (int k2 = 0; k2 < HALF / 16; ++k2)
                mma_ts(o, p_tmem + half * HALF + k2 * 8,
                       vd + (((half * (HALF / 16) + k2) * 2 * C::HALVES * 1024) >> 4), ID_PV,
                       !fresh || k2 > 0 || (C::TURNS && half));
            } else {
#pragma unroll
              for (int k2 = 0; k2 < HALF / 16; ++k2)
                mma_ts(o, p_tmem + half * HALF + k2 * 8,
                       vd + (((half * (HALF / 16) + k2) * 2 * 1024) >> 4), ID_PV,
                       !fresh || k2 > 0 || (C::TURNS && half));
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        if (leader) {
          mma_commit(&sm.s_free[buf]);
          if (v == C::SETS * n_tiles - 1) mma_commit(&sm.o_last);
          if (last) mma_commit(&sm.v_empty[slot]);
        }
        __syncwarp();
        if (last && ++slot == C::NST) {
          slot = 0;
          v_phase ^= 1;
        }
        if (++buf == NSB) {
          buf = 0;
          p_phase ^= 1;
        }
      }
    }
  } else {
    // Keys of a tile that a group takes, in parts of 64: that many scores fit the
    // registers (and are read from TMEM again, 35 cycles, where they are wanted twice).
    constexpr int KEYS = C::TURNS ? KV_TILE : HALF, PARTS = KEYS / HALF, STEP = C::TURNS ? 2 : 1;
    const int half = (warp - SOFTMAX_WARP0) >> 2;  // the group, and its accumulator
    const int key_in = C::TURNS ? 0 : half * HALF;  // its first key of a tile
    const int r = (threadIdx.x - SOFTMAX_WARP0 * 32) & (GROUP_THREADS - 1);  // TMEM lane, and row of the tile
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_tmem = tmem + lane_base + half * D;
    const int i_in = args.fd_g.div(r);  // token of the tile, and head of the group
    const int h_in = r - i_in * a.G;
    const int set_in = PAIR ? half * a.tok_tile : 0;  // its first token of the item
    int jg = 0;  // S buffers filled, over every item
    Item I;
    bool ok = __all_sync(0xffffffffu, queue_item(0, I));
    for (int k = 0; ok && I.n_tiles; ++k) {
      const bool active = I.i0 + set_in + i_in < I.len;
      const int i = active ? I.i0 + set_in + i_in : I.len - 1;
      // the cached keys the row sees: t < hi, and t >= lo or t < sinks
      int lo, hi, hi_least, lo_most;
      uint64_t anc[2][PARTS] = {};  // the group's keys of the two tree tiles
      if (TREE) {
        const int P = I.pos0;
        uint64_t w4[4] = {0ull, 0ull, 0ull, 0ull};
        int depth = 0;
        if (active) {
          const uint64_t* arow = a.anc_mask + ((size_t)I.b * a.N + i) * a.W;
#pragma unroll
          for (int w = 0; w < 4; ++w)
            if (w < a.W) w4[w] = arow[w];
          depth = max(__popcll(w4[0]) + __popcll(w4[1]) + __popcll(w4[2]) + __popcll(w4[3]) - 1, 0);  // (an empty mask: 0)
        }
        lo = P + depth - a.window + 1;
        hi = hi_least = P;
        lo_most = P + a.N - a.window;
        // Ancestors out of the window.  Node indices rise along a chain, so the
        // k-th set bit is the ancestor at depth k: hidden if depth - k >= window
        // and P + k >= sinks.
        const int hide_end = depth + 1 - a.window, hide0 = max(a.sinks - P, 0);
        if (hide_end > hide0) {
          int at = 0;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint64_t left = w4[w];
            while (left && at < hide_end) {
              const uint64_t bit = left & (0ull - left);
              left ^= bit;
              if (at >= hide0) w4[w] ^= bit;
              ++at;
            }
          }
        }
#pragma unroll
        for (int h = 0; h < PARTS; ++h) {
          anc[0][h] = (C::TURNS ? h : half) ? w4[1] : w4[0];
          anc[1][h] = (C::TURNS ? h : half) ? w4[3] : w4[2];
        }
      } else {
        const int pos = I.pos0 + (i - I.i0);
        lo = pos - a.window + 1;
        hi = pos + 1;
        hi_least = I.pos0 + set_in + 1;
        lo_most = min(I.pos0 + set_in + a.tok_tile, I.hi) - a.window;
      }
      if (a.window == 0) lo = lo_most = 0;
      // Tiles j in [clear0, clear1) are wholly visible to the group's rows: those before
      // hold sinks, or keys that a later row's window is past; those after, keys
      // past an earlier row.
      int clear0 = 0;
      if (lo_most > 0) clear0 = I.n_sink + max(ceil_div(lo_most, KV_TILE) - I.win0, 0) - I.t_begin;
      const int clear1 = I.n_sink + hi_least / KV_TILE - I.win0 - I.t_begin;
      float m_run = NEG_INF, l_run = 0.f, norm_run = 0.f;  // norm: what the output is divided by
      const int first = C::TURNS ? half : 0;
      bool fresh = true;
      const int n_uses = C::SETS * I.n_tiles;
      for (int use = first; use < n_uses; use += STEP) {
        const int j = use / C::SETS, jt = jg + use, buf = jt % NSB;
        if (!__all_sync(0xffffffffu, wait_bar(&sm.s_full[buf], (jt / NSB) & 1, ctl))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t s_tmem = tmem + lane_base + TMEM_S0 + buf * KV_TILE + key_in;
        uint64_t see[PARTS];  // the keys this row sees, where it may not see all
        bool dead = false;
        int key0 = 0;
        const bool masked = j < clear0 || j >= clear1;
        if (masked) {
          const bool tree = TREE && j >= I.n_prefix;
          if (!tree) {
            key0 = tile_key(I, j) + key_in;
            dead = key0 + KEYS > I.hi || (key0 < I.lo && key0 + KEYS > a.sinks);
          }
#pragma unroll
          for (int h = 0; h < PARTS; ++h) {
            const int at = key0 + h * HALF;
            see[h] = tree ? anc[j > I.n_prefix][h]
                          : first_bits(hi - at) & (~first_bits(lo - at) | first_bits(a.sinks - at));
          }
        }
        float s[HALF];
        const auto load = [&](int h) {
          uint32_t u[2][32];
          tmem_ld32(s_tmem + h * HALF, u[0]);
          tmem_ld32(s_tmem + h * HALF + 32, u[1]);
          tmem_ld_wait();
          reg_fence32(u[0]);
          reg_fence32(u[1]);
#pragma unroll
          for (int e = 0; e < HALF; ++e) s[e] = __uint_as_float(u[e / 32][e % 32]);
          if (masked) {
            const uint64_t w = PARTS > 1 && h ? see[PARTS - 1] : see[0];
#pragma unroll
            for (int e = 0; e < HALF; ++e)
              if (!((w >> e) & 1ull)) s[e] = NEG_INF;
          }
        };
        const auto largest = [&]() {  // of s
          float mk[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) mk[e] = s[e];
#pragma unroll
          for (int c = 4; c < HALF; c += 4)
#pragma unroll
            for (int e = 0; e < 4; ++e) mk[e] = fmaxf(mk[e], s[c + e]);
          return fmaxf(fmaxf(mk[0], mk[1]), fmaxf(mk[2], mk[3]));
        };
        const uint64_t scale2 = fx::pack2(a.scale_log2, a.scale_log2);
        uint64_t negm2, sum2[2];
        float neg_m, top;  // top: the largest weight
        const auto against = [&](float m) {  // (-inf: nothing visible so far, every weight is 0)
          neg_m = m == NEG_INF ? 0.f : -m;
          negm2 = fx::pack2(neg_m, neg_m);
          sum2[0] = sum2[1] = 0ull;
          top = 0.f;
        };
        const auto weigh = [&](uint32_t (&pk)[HALF / 2]) {  // s to bf16 weights, and their sums
#pragma unroll
          for (int e = 0; e < HALF / 2; ++e) {
            float x0, x1;
            fx::unpack2(fx::fma2(fx::pack2(s[2 * e], s[2 * e + 1]), scale2, negm2), x0, x1);
            const float p0 = ex2(x0), p1 = ex2(x1);
            sum2[e & 1] = fx::add2(sum2[e & 1], fx::pack2(p0, p1));
            pk[e] = pack_bf16x2(p0, p1);
            if (C::TURNS) top = fx::max3(top, p0, p1);
          }
        };
        const auto total = [&]() {
          float r0, r1;
          fx::unpack2(fx::add2(sum2[0], sum2[1]), r0, r1);
          return r0 + r1;
        };
        float m_use = m_run, rowsum;
        if constexpr (C::TURNS) {
          // A row takes a new reference only by its own weights: where it has none
          // yet, or its sum has passed the limit.  The warp then looks for maxima and
          // takes the tile's weights once more.
          uint32_t pk[PARTS][HALF / 2];
          bool need = m_run == NEG_INF;
          bool look = fresh;  // (some row of the warp may have none)
          for (;;) {
            if (look) {
              float m_tile = NEG_INF;
#pragma unroll 1
              for (int h = 0; h < PARTS; ++h) {
                load(h);
                m_tile = fmaxf(m_tile, largest() * a.scale_log2);
              }
              if (need) m_use = fmaxf(m_run, m_tile);
            }
            against(m_use);
#pragma unroll
            for (int h = 0; h < PARTS; ++h) {
              load(h);
              weigh(pk[h]);
            }
            rowsum = total();
            const bool over = active && !need && !(rowsum <= SUM_LIMIT);
            if (!__any_sync(0xffffffffu, over)) break;
            need = need || over;
            look = true;
          }
          if (fresh) fresh = __any_sync(0xffffffffu, m_use == NEG_INF);
#pragma unroll
          for (int h = 0; h < PARTS; ++h) tmem_st32(s_tmem + h * HALF, pk[h]);
        } else {
          load(0);
          const float s_top = largest(), m_new = fmaxf(m_run, s_top * a.scale_log2);
          if (use == first || (active && m_new > m_run + RESCALE_THRESHOLD)) m_use = m_new;
          against(m_use);
          uint32_t pk[HALF / 2];
          weigh(pk);
          tmem_st32(s_tmem, pk);
          rowsum = total();
          top = ex2(fmaf(s_top, a.scale_log2, neg_m));  // as weigh made it
        }
        const bool rescale = use > first && active && m_use != m_run;
        if (dead && !(PAIR && half)) {
          // V rows that no row of the item sees hold whatever the pool, or the ring, had
          // there: zeroed, so that 0 * V is 0 (of a pair by the first group, whose PV is
          // the first to read the tile)
          const int vt = jt / C::SETS, slot = vt % C::NST;
          if (!__all_sync(0xffffffffu, wait_bar(&sm.v_full[slot], (vt / C::NST) & 1, ctl))) {
            ok = false;
            break;
          }
          // (16 bytes a store, a row's by adjacent threads: a row a thread would take its
          // stores through the same banks, 32 passes each)
#pragma unroll
          for (int n = 0; n < KEYS * C::HALVES * 8 / GROUP_THREADS; ++n) {
            const int c = n * GROUP_THREADS + r, piece = c >> 3, hh = piece / KEYS, vr = key_in + piece % KEYS;
            const int t = key0 + piece % KEYS;
            if (t >= I.hi || (t < I.lo && t >= a.sinks))
              *reinterpret_cast<uint4*>(sm.v[slot] + ((vr >> 3) * C::HALVES + hh) * 1024 + (vr & 7) * 128 + (c & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
        }
        if (use > first && __any_sync(0xffffffffu, rescale)) {
          // The accumulator's last PV complete (its S buffer is free again; the one
          // before that was when the buffer was filled, and the one after waits for
          // these weights, so the phase is no other's).  The whole warp takes part, by
          // 1 where a row's maximum did not move enough.
          const int last = jt - STEP;
          if (!__all_sync(0xffffffffu, wait_bar(&sm.s_free[last % NSB], (last / NSB) & 1, ctl))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float f = !rescale ? 1.f : m_run == NEG_INF ? 0.f : ex2(m_run - m_use);
          l_run *= f;
          norm_run *= f;
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t u0[32];
            tmem_ld32(o_tmem + c, u0);
            tmem_ld_wait();
            reg_fence32(u0);
#pragma unroll
            for (int e = 0; e < 32; ++e) u0[e] = __float_as_uint(__uint_as_float(u0[e]) * f);
            tmem_st32(o_tmem + c, u0);
          }
        }
        m_run = m_use;
        l_run += rowsum;
        norm_run += rowsum + (__bfloat162float(__float2bfloat16_rn(top)) - top);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sm.p_full[buf][C::TURNS ? 0 : half]);
      }
      jg += n_uses;
      if (!ok) break;
      // the item's end: its last PV, then the groups' halves joined, and each stores half
      // of the channels, of both accumulators; of a pair each stores its own row tile.
      if (!PAIR && half == 1) {
        sm.ml[r] = make_float2(m_run, l_run);
        sm.norm[r] = norm_run;
        mbar_arrive(&sm.ml_full);
      }
      Item next;  // asked for while the last PV runs
      ok = __all_sync(0xffffffffu, queue_item(k + 1, next));
      if (!ok) break;
      float f0 = 0.f, f1 = 0.f, lse2 = NEG_INF;
      if (PAIR) {
        if (l_run > 0.f) lse2 = m_run + __log2f(l_run);
        f0 = norm_run > 0.f ? 1.f / norm_run : 0.f;  // a row that sees no key: zeros
      } else if (half == 0) {
        ok = __all_sync(0xffffffffu, wait_bar(&sm.ml_full, k & 1, ctl));
        if (!ok) break;
        const float2 other = sm.ml[r];
        const float m_all = fmaxf(m_run, other.x);
        f0 = m_run == NEG_INF ? 0.f : ex2(m_run - m_all);
        f1 = other.x == NEG_INF ? 0.f : ex2(other.x - m_all);
        const float l_all = l_run * f0 + other.y * f1;
        const float norm = norm_run * f0 + sm.norm[r] * f1;
        const float inv = norm > 0.f ? 1.f / norm : 0.f;  // a row that sees no key: zeros
        if (l_all > 0.f) lse2 = m_all + __log2f(l_all);
        f0 *= inv;
        f1 *= inv;
        sm.ml[r] = make_float2(f0, f1);
        mbar_arrive(&sm.f_full);
      } else {
        ok = __all_sync(0xffffffffu, wait_bar(&sm.f_full, k & 1, ctl));
        if (!ok) break;
        f0 = sm.ml[r].x;
        f1 = sm.ml[r].y;
      }
      const bool direct = I.ps == 1;
      const PagedSeq& sq = args.seq[I.e];
      const size_t orow = direct ? (size_t)(I.q0 + i) * a.Hq + I.g * a.G + h_in
                                 : ((size_t)sq.part_row + (size_t)I.split * sq.rows + i) * a.Hq + I.g * a.G + h_in;
      ok = __all_sync(0xffffffffu, wait_bar(&sm.o_last, k & 1, ctl));
      if (!ok) break;
      tc_fence_after();
      const uint64_t f02 = fx::pack2(f0, f0), f12 = fx::pack2(f1, f1);
      constexpr int MINE = PAIR ? D : D / 2, PIECES = MINE / 16;  // channels a group stores; in 16s
      const int c0 = PAIR ? 0 : half * MINE;
      float x[16];
      const auto piece = [&](int c) {  // 16 channels of the row
        uint32_t u[16];
        if constexpr (PAIR) {
          tmem_ld16(o_tmem + c, u);
          tmem_ld_wait();
          reg_fence16(u);
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = __uint_as_float(u[e]) * f0;
        } else {
          uint32_t v[16];
          tmem_ld16(tmem + lane_base + c, u);
          // (the second group may have had no tile: its accumulator then holds anything)
          tmem_ld16(tmem + lane_base + (C::TURNS && I.n_tiles == 1 ? 0 : D) + c, v);
          tmem_ld_wait();
          reg_fence16(u);
          reg_fence16(v);
#pragma unroll
          for (int e = 0; e < 16; e += 2)
            fx::unpack2(fx::fma2(fx::pack2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), f12,
                                 fx::mul2(fx::pack2(__uint_as_float(u[e]), __uint_as_float(u[e + 1])), f02)),
                        x[e], x[e + 1]);
        }
      };
      if (direct) {
        // PIECES lanes exchange theirs, so that each store of the warp has whole lines:
        // a lane then has one piece of PIECES rows.
        uint32_t w[PIECES][8];
#pragma unroll
        for (int n = 0; n < PIECES; ++n) {
          piece(c0 + 16 * n);
#pragma unroll
          for (int e = 0; e < 8; ++e) w[n][e] = pack_bf16x2(x[2 * e], x[2 * e + 1]);
        }
#pragma unroll
        for (int bit = 1; bit < PIECES; bit <<= 1) {
          const bool upper = lane & bit;
#pragma unroll
          for (int n = 0; n < PIECES; ++n) {
            if (n & bit) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t got = __shfl_xor_sync(0xffffffffu, upper ? w[n][e] : w[n | bit][e], bit);
              if (upper) w[n][e] = got;
              else w[n | bit][e] = got;
            }
          }
        }
        const long long own = active ? (long long)orow : -1;
#pragma unroll
        for (int n = 0; n < PIECES; ++n) {
          const long long row = __shfl_sync(0xffffffffu, own, (lane & ~(PIECES - 1)) | n);
          if (row < 0) continue;
          __nv_bfloat16* dst = a.out + row * D + c0 + 16 * (lane & (PIECES - 1));
          if (args.out32) {
            st_v8(dst, w[n]);
          } else {
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[n][0], w[n][1], w[n][2], w[n][3]);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[n][4], w[n][5], w[n][6], w[n][7]);
          }
        }
        __syncwarp();
      } else {
#pragma unroll 1
        for (int c = c0; c < c0 + MINE; c += 16) {
          piece(c);
          if (!active) continue;
          float* dst = a.part_o + orow * D + c;
          st_v8(dst, reinterpret_cast<const uint32_t*>(x));
          st_v8(dst + 8, reinterpret_cast<const uint32_t*>(x) + 8);
        }
      }
      if (active && (PAIR || half == 0)) {
        if (!direct) a.part_lse[orow] = lse2;
        else if (a.lse) a.lse[orow] = lse2 * 0.69314718055994531f;
      }
      // the accumulators and statistics have been read: the next item may have them
      tc_fence_before();
      mbar_arrive(&sm.o_free);
      __syncwarp();
      if (lane == 0) {
        __threadfence_block();
        atomicAdd(&sm.items_done, 1);
      }
      I = next;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*ctl.flag) {
    // A wait gave up: nothing may still write this CTA's shared memory or TMEM
    // once it exits.
    if ((warp == K_WARP || warp == V_WARP) && lane == 0) {
      uint64_t* full = warp == K_WARP ? sm.k_full : sm.v_full;
      for (int j = max(0, issued - C::NST); j < issued; ++j) mbar_wait(&full[j % C::NST], (j / C::NST) & 1, a.wait_limit_ns);
    } else if ((warp == QK_WARP || warp == PV_WARP) && leader) {
      if (q_issued > q_landed) mbar_wait(&sm.q_full, (q_issued - 1) & 1, a.wait_limit_ns);
      uint64_t* d = &sm.drain[warp - QK_WARP];
      mma_commit(d);
      mbar_wait(d, 0, a.wait_limit_ns);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
      auto report = [&](int it) {
        if (it < 0 || !a.status) return;
        const Place p = place_of(it, args);
        const int b = args.seq[p.e].b;
        const Lens l = load_lens<TREE>(b, args.seq[p.e].rows, a);
        if (make_item<TREE>(p, b, l.q0, l.len, l.kv, args).n_tiles) a.status[b] = TS_ERR_TIMEOUT;
      };
      const int done = sm.items_done / SOFTMAX_WARPS;  // wholly
      if (single) {
        if (done == 0) report(blockIdx.x);
      } else {
        for (int k = done; k < sm.items_pub && k < done + C::ITEM_Q; ++k) {
          const int4* q = sm.item_q[k % C::ITEM_Q];
          if (q[3].z && a.status) a.status[q[0].x] = TS_ERR_TIMEOUT;
        }
      }
      report(held);
      while (!exhausted) {
        const int it = take_item();
        exhausted = it < 0;
        report(it);
      }
    }
  }
  pdl_trigger();
  if (warp == K_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Joins the splits of cut chains: out = sum_s 2^(L_s - M) O_s / sum_s 2^(L_s - M),
// M = max L_s.  D/8 lanes a row (token, head), 8 channels each; a group of GRP
// splits' loads is in flight at once.  Latency-bound: a few MB behind the attention (the
// plans count 3 us and its bytes).
constexpr int JOIN_THREADS = 128;
constexpr int JOIN_GRP = 8;

struct JoinArgs {
  PagedArgs a;
  int n_seqs;
  FastDiv fd_hq;
  PagedSeq seq[PAGED_MAX_SEQS];  // cut ones only; item0: first (token, head) row of the grid
};

template <int D, bool TREE>
__global__ void __launch_bounds__(JOIN_THREADS)
k_join_paged(const __grid_constant__ JoinArgs t) {
  constexpr int LPR = D / 8, ROWS = JOIN_THREADS / LPR;
  const PagedArgs& a = t.a;
  const int row = blockIdx.x * ROWS + (int)threadIdx.x / LPR;
  const int sub = (int)threadIdx.x % LPR;
  int e = 0, hi = t.n_seqs - 1;
  while (e < hi) {
    const int mid = (e + hi + 1) >> 1;
    if (t.seq[mid].item0 <= row) e = mid;
    else hi = mid - 1;
  }
  const PagedSeq& sq = t.seq[e];
  const int x = row - sq.item0;
  const int i = t.fd_hq.div(x), h = x - i * a.Hq;
  pdl_wait();
  pdl_trigger();
  if (i >= sq.rows) return;
  const Lens l = load_lens<TREE>(sq.b, sq.rows, a);
  if (i >= l.len) return;
  const PagedSpan sp = TREE ? paged_span(l.kv, l.kv, a.window, a.sinks)
                            : chunk_span(l.kv, l.len, i / a.tok * a.tok, a.tok, a.window, a.sinks);
  const int ps = paged_splits(sp.n, a.chunk_tiles, sq.splits);
  if (ps == 1) return;  // written by the attention kernel
  const size_t stride = (size_t)sq.rows * a.Hq;  // (token, head) rows of a split
  const size_t at = ((size_t)sq.part_row + i) * a.Hq + h;
  float m = NEG_INF, den = 0.f, acc[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) acc[c] = 0.f;
  for (int s0 = 0; s0 < ps; s0 += JOIN_GRP) {
    float w[JOIN_GRP];
    float4 x0[JOIN_GRP], x1[JOIN_GRP];
    float gm = NEG_INF;
#pragma unroll
    for (int s = 0; s < JOIN_GRP; ++s) {
      w[s] = NEG_INF;
      x0[s] = x1[s] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s0 + s < ps) {
        const size_t k = at + (s0 + s) * stride;
        w[s] = a.part_lse[k];
        const float4* p = reinterpret_cast<const float4*>(a.part_o + k * D + sub * 8);
        x0[s] = p[0];
        x1[s] = p[1];
      }
    }
#pragma unroll
    for (int s = 0; s < JOIN_GRP; ++s) gm = fmaxf(gm, w[s]);
    const float m_new = fmaxf(m, gm);
    if (m_new == NEG_INF) continue;  // nothing visible in these splits
    const float f = m == NEG_INF ? 0.f : exp2f(m - m_new);
    den *= f;
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c] *= f;
    m = m_new;
#pragma unroll
    for (int s = 0; s < JOIN_GRP; ++s) {
      const float p = exp2f(w[s] - m);
      den += p;
      acc[0] = fmaf(p, x0[s].x, acc[0]);
      acc[1] = fmaf(p, x0[s].y, acc[1]);
      acc[2] = fmaf(p, x0[s].z, acc[2]);
      acc[3] = fmaf(p, x0[s].w, acc[3]);
      acc[4] = fmaf(p, x1[s].x, acc[4]);
      acc[5] = fmaf(p, x1[s].y, acc[5]);
      acc[6] = fmaf(p, x1[s].z, acc[6]);
      acc[7] = fmaf(p, x1[s].w, acc[7]);
    }
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  const size_t orow = (size_t)(l.q0 + i) * a.Hq + h;
  uint32_t o[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) o[c] = pack_bf16x2(acc[2 * c] * inv, acc[2 * c + 1] * inv);
  reinterpret_cast<uint4*>(a.out + orow * D)[sub] = make_uint4(o[0], o[1], o[2], o[3]);
  if (a.lse && sub == 0) a.lse[orow] = den > 0.f ? (m + log2f(den)) * 0.69314718055994531f : NEG_INF;
}

template <int D, bool PAIR>
constexpr size_t smem_bytes() {
  return sizeof(Smem<D, PAIR>) + 1024;  // for the 1024-byte alignment of the swizzle atoms
}
static_assert(smem_bytes<128, false>() <= 227 * 1024 && smem_bytes<64, false>() <= 227 * 1024 &&
                  smem_bytes<64, true>() <= 227 * 1024,
              "");

template <int D, bool TREE, bool PAIR>
cudaError_t launch(const PagedArgs& a, const PagedPlan& pl, cudaStream_t s) {
  const PagedSeq* seq = pl.seq;
  const int n_seqs = pl.n_seqs, n_items = pl.n_items;
  KArgs t{};
  t.a = a;
  t.box_rows = KV_TILE;
  while (a.bs % t.box_rows != 0) t.box_rows >>= 1;
  t.n_items = n_items;
  t.n_seqs = n_seqs;
  t.out32 = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
  t.fd_hkv = FastDiv::make(a.Hkv);
  t.fd_bs = FastDiv::make(a.bs);
  t.fd_g = FastDiv::make(a.G);
  std::copy(seq, seq + n_seqs, t.seq);
  std::copy(pl.gaps.before, pl.gaps.before + n_seqs, t.gaps.before);
  t.gaps.last = pl.gaps.last;
  t.gaps.end = pl.gaps.end;
  CUtensorMap m_q, m_kc, m_vc, m_kt, m_vt;
  {  // q [T, Hq, D]: a box of 64 channels, G heads, ROW_TILE / G tokens is 64 channels of 128 rows
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.Hq, (uint64_t)a.T};
    const uint64_t str[2] = {(uint64_t)D * 2, (uint64_t)a.Hq * D * 2};
    const uint32_t box[3] = {64, (uint32_t)a.G, (uint32_t)a.tok_tile};
    if (!encode_bf16_sw128(&m_q, a.q, 3, dims, str, box)) return cudaErrorInvalidValue;
  }
  {  // pool [num_blocks, Hkv, bs, D] as 64 channels, 8 rows, halves, groups of 8 rows
    const uint64_t dims[4] = {64, 8, (uint64_t)(D / 64), (uint64_t)a.num_blocks * a.Hkv * (a.bs / 8)};
    const uint64_t str[3] = {(uint64_t)D * 2, 128, (uint64_t)8 * D * 2};
    const uint32_t box[4] = {64, 8, (uint32_t)(D / 64), (uint32_t)(t.box_rows / 8)};
    if (!encode_bf16_sw128(&m_kc, a.k_cache, 4, dims, str, box)) return cudaErrorInvalidValue;
    if (!encode_bf16_sw128(&m_vc, a.v_cache, 4, dims, str, box)) return cudaErrorInvalidValue;
  }
  m_kt = m_kc;
  m_vt = m_vc;
  if (TREE) {  // tree K/V [B, N, Hkv, D]: 128 nodes of one head; nodes >= N read as zeros
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)a.Hkv, (uint64_t)a.N, (uint64_t)a.B};
    const uint64_t str[3] = {(uint64_t)D * 2, (uint64_t)a.Hkv * D * 2, (uint64_t)a.N * a.Hkv * D * 2};
    const uint32_t box[4] = {64, 1, (uint32_t)KV_TILE, 1};
    if (!encode_bf16_sw128(&m_kt, a.k_tree, 4, dims, str, box)) return cudaErrorInvalidValue;
    if (!encode_bf16_sw128(&m_vt, a.v_tree, 4, dims, str, box)) return cudaErrorInvalidValue;
  }
  int ctas = sm_count();
  if (ctas <= 0) return cudaErrorInvalidDevice;
  if (a.max_ctas > 0 && a.max_ctas < ctas) ctas = a.max_ctas;
  const dim3 grid(n_items < ctas ? n_items : ctas);
  cudaError_t e = launch_pdl(k_attn_paged<D, TREE, PAIR>, grid, dim3(NUM_THREADS), smem_bytes<D, PAIR>(), s, t, m_q, m_kc, m_vc,
                             m_kt, m_vt);
  if (e != cudaSuccess || pl.part_rows == 0) return e;
  JoinArgs j{};
  j.a = a;
  j.fd_hq = FastDiv::make(a.Hq);
  int rows = 0;
  for (int k = 0; k < n_seqs; ++k) {
    if (seq[k].splits == 1) continue;
    j.seq[j.n_seqs] = seq[k];
    j.seq[j.n_seqs++].item0 = rows;
    rows += seq[k].rows * a.Hq;
  }
  const int per = JOIN_THREADS / (D / 8);
  return launch_pdl(k_join_paged<D, TREE>, dim3(ceil_div(rows, per)), dim3(JOIN_THREADS), 0, s, j);
}

// The plan of a launch's sequences: how long a split may be, and whether an item
// takes a pair of row tiles.  Every chain of key tiles (an item's rows of a KV head) is
// an item or, cut, several; a CTA an SM takes them longest first.  In units of 0.8 us,
// a tile costs tile_time on an SM (STREAMED times as much where no other row tile brings
// its keys to L2), an item its tiles and 3 more (its start and its end).  The launch ends
// when the SMs have shared all of that out: a batch of few sequences, whose items may
// differ much, is dealt out as the kernel will; of many, the average item says it.  And it
// does not end before the keys and values have come from memory (which the last items, and
// the items' starts, do not keep busy).  Cut chains cost a second kernel and their partial
// results' round trip.  On fourteen ragged batches the plans were within 0 to 12 % of the
// best of a sweep (by averages alone, a prompt's 1024 tokens beside 64-tile chains of
// single tokens were left uncut: 73 us, now 65).  More than FEW_SEQS sequences are judged by
// the average all the same, since dealing out takes time with the square of their number: nine more
// sequences with a token of 5 keys make that batch 73 us again.
struct Chains {
  int count;     // items' rows
  int most;      // tiles of the longest chain
  double total;  // tiles of all
};
struct Cut {
  int chunk_tiles;
  double cost;
};
// A tile's time.  Heads of 64 with blocks of 16 wait for the boxes' issue, which a pair
// shares between two row tiles.
double tile_time(int D, int bs, bool pair) { return D == 128 ? 1.0 : pair ? 1.4 : bs % 32 ? 0.86 : 0.74; }

constexpr double STREAMED = 1.2;
constexpr int FEW_SEQS = 16;

// When the last of n groups of items is done, on PLAN_SMS SMs that take them longest first:
// at[] and sms[], ascending, so many SMs are free at that time.
double dealt_out(double* time, double* count, int n) {
  double at[2 * FEW_SEQS + 2], sms[2 * FEW_SEQS + 2];
  int m = 1;
  at[0] = 0;
  sms[0] = PLAN_SMS;
  for (int k = 1; k < n; ++k)  // longest first
    for (int j = k; j > 0 && time[j] > time[j - 1]; --j) {
      std::swap(time[j], time[j - 1]);
      std::swap(count[j], count[j - 1]);
    }
  for (int k = 0; k < n; ++k) {
    for (double left = count[k]; left > 0;) {
      const double take = std::min(left, sms[0]), end = at[0] + time[k];
      left -= take;
      sms[0] -= take;
      int to = sms[0] > 0 ? m : m - 1;  // entries once the first, used up, is gone
      if (sms[0] <= 0) {
        std::copy(at + 1, at + m, at);
        std::copy(sms + 1, sms + m, sms);
      }
      m = to;
      while (to > 0 && at[to - 1] > end) {
        at[to] = at[to - 1];
        sms[to] = sms[to - 1];
        --to;
      }
      if (to > 0 && at[to - 1] == end) {
        sms[to - 1] += take;
        for (; to < m; ++to) at[to] = at[to + 1], sms[to] = sms[to + 1];
      } else {
        at[to] = end;
        sms[to] = take;
        ++m;
      }
    }
  }
  return at[m - 1];
}

Cut plan_cut(const Chains* c, const int* rows, int n, int Hkv, int Hq, int D, int tree_tiles, double tile) {
  constexpr double item_cost = 3.0, join_launch = 4.0, unit_bytes = 5.4e6;  // traffic in a unit
  int longest = 1;
  double streamed = 0;
  for (int k = 0; k < n; ++k) {
    longest = std::max(longest, c[k].most);
    streamed += c[k].most + tree_tiles;  // a sequence's row tiles read the same keys
  }
  const double memory = streamed * Hkv * (double)(4 * KV_TILE * D) / unit_bytes;
  Cut best{longest, 1e300};
  const auto look = [&](int chunk) {  // what cutting to so many tiles costs
    double items = 0, part_rows = 0, longest_item = 0, work = 0, time[FEW_SEQS], count[FEW_SEQS];
    int worst = 0;
    for (int k = 0; k < n; ++k) {
      const int ps = paged_splits(c[k].most, chunk, INT_MAX);
      const double own = tile * (c[k].count == 1 ? STREAMED : 1.0), group = (double)c[k].count * ps * Hkv;
      const double mean = own * (c[k].total / c[k].count + tree_tiles) / ps + item_cost;
      items += group;
      work += group * mean;
      worst = std::max(worst, ceil_div(c[k].most, ps));
      longest_item = std::max(longest_item, own * (ceil_div(c[k].most, ps) + tree_tiles) + item_cost);
      if (ps > 1) part_rows += (double)ps * rows[k];
      if (n <= FEW_SEQS) {
        time[k] = mean;
        count[k] = group;
      }
    }
    const double waves = items / PLAN_SMS;
    double cost = std::max(std::max(longest_item, work / PLAN_SMS), memory + 0.25 * tile * worst + 2.0 * std::ceil(waves));
    const double join = part_rows > 0 ? join_launch + 2.0 * part_rows * Hq * (4.0 * D + 4.0) / unit_bytes : 0.0;
    if (n > FEW_SEQS || waves > 4) cost = std::max(cost, work / items * (waves > 1 ? waves + 0.5 : 1.0));
    else if (waves > 1 && cost + join < best.cost) cost = std::max(cost, dealt_out(time, count, n));
    cost += join;
    if (cost < best.cost) best = Cut{chunk, cost};
    return cost;
  };
  for (int s = 1, last = 0; s <= 256; s += 1 + s / 8) {
    const int chunk = ceil_div(longest, s);
    if (chunk == last) continue;
    last = chunk;
    if (look(chunk) > 1.5 * best.cost || chunk == 1) break;
  }
  if (n <= FEW_SEQS)  // or those cut that are longer than one of them
    for (int k = 0; k < n; ++k)
      if (c[k].most < longest && 2 * c[k].most > longest) look(c[k].most);
  return best;
}

// The chains of sequence b's items of `tok` tokens.
template <bool TREE>
Chains chains_of(const PagedArgs& a, int tok, int len, int kv) {
  Chains c;
  c.count = ceil_div(len, tok);
  if (TREE) {
    c.most = paged_span(kv, kv, a.window, a.sinks).n;
    c.total = (double)c.most * c.count;
    return c;
  }
  const int first = chunk_span(kv, len, 0, tok, a.window, a.sinks).n;
  const int last = chunk_span(kv, len, (c.count - 1) * tok, tok, a.window, a.sinks).n;
  c.most = std::max(std::max(first, last), 1);
  // a window's chains may be a tile longer or shorter in between
  if (a.window > 0 && c.count > 2)
    c.most = std::max(c.most, std::min(ceil_div(kv, KV_TILE),
                                       ceil_div(a.window + tok, KV_TILE) + 1 + ceil_div(a.sinks, KV_TILE)));
  c.total = 0.5 * (first + last) * c.count;
  return c;
}

// Sequences [b0, pl->b_end) of a call: their entries, in the order the items are taken.
template <bool TREE>
void plan_launch(const PagedArgs& a, const int32_t* cu_len_host, const int32_t* kv_host, int b0, PagedPlan* pl) {
  Chains both[2][PAGED_MAX_SEQS];
  int rows[PAGED_MAX_SEQS], bs[PAGED_MAX_SEQS], order[PAGED_MAX_SEQS], before[PAGED_MAX_SEQS];
  int n = 0, b = b0, gap = b0;
  bool pairs = false;  // some sequence has a second row tile
  for (; b < a.B; ++b) {
    const int len = TREE ? a.N : cu_len_host[b + 1] - cu_len_host[b];
    if (len == 0) continue;
    if (n == PAGED_MAX_SEQS) break;
    before[n] = gap;
    gap = b + 1;
    rows[n] = len;
    bs[n] = b;
    both[0][n] = chains_of<TREE>(a, a.tok_tile, len, kv_host[b]);
    pairs = pairs || len > a.tok_tile;
    order[n] = n;
    ++n;
  }
  pl->b_end = b;
  pl->n_seqs = n;
  pl->n_items = 0;
  pl->part_rows = 0;
  pl->chunk_tiles = 1;
  pl->pair = false;
  pl->ok = true;
  if (n == 0) return;
  pl->gaps.last = bs[n - 1];
  pl->gaps.end = b;
  const int tree_tiles = TREE ? ceil_div(a.N, KV_TILE) : 0;
  Cut cut = plan_cut(both[0], rows, n, a.Hkv, a.Hq, a.D, tree_tiles, tile_time(a.D, a.bs, false));
  if (a.D == 64 && pairs) {
    for (int k = 0; k < n; ++k) both[1][k] = chains_of<TREE>(a, 2 * a.tok_tile, rows[k], kv_host[bs[k]]);
    const Cut p = plan_cut(both[1], rows, n, a.Hkv, a.Hq, a.D, tree_tiles, tile_time(a.D, a.bs, true));
    pl->pair = p.cost < cut.cost;
    if (pl->pair) cut = p;
  }
  const Chains* c = both[pl->pair];
  pl->chunk_tiles = cut.chunk_tiles;
  int each[PAGED_MAX_SEQS];
  for (int k = 0; k < n; ++k) {
    const int ps = paged_splits(c[k].most, pl->chunk_tiles, INT_MAX);
    each[k] = ceil_div(c[k].most, ps);
  }
  std::stable_sort(order, order + n, [&](int x, int y) { return each[x] > each[y]; });
  long long items = 0, part = 0;
  for (int k = 0; k < n; ++k) {
    const int x = order[k];
    PagedSeq& q = pl->seq[k];
    q.item0 = (int)items;
    q.b = bs[x];
    q.row_tiles = c[x].count;
    q.splits = paged_splits(c[x].most, pl->chunk_tiles, INT_MAX);
    q.rows = rows[x];
    q.part_row = (int)part;
    pl->gaps.before[k] = before[x];
    items += (long long)q.row_tiles * q.splits * a.Hkv;
    if (q.splits > 1) part += (long long)q.splits * q.rows;
    if (items > (1ll << 30) || part * a.Hq >= (1ll << 31)) pl->ok = false;
  }
  pl->n_items = (int)items;
  pl->part_rows = part;
}

size_t plan_bytes(const PagedArgs& a, long long part_rows) {
  return ATTN_SCHED_BYTES + (size_t)part_rows * a.Hq * (4 * a.D + 4);
}

template <bool TREE>
size_t workspace_of(const PagedArgs& a, const int32_t* cu_len_host, const int32_t* kv_host, PagedPlan* first) {
  plan_launch<TREE>(a, cu_len_host, kv_host, 0, first);
  if (!first->ok) return 0;
  long long most = first->part_rows;
  for (int b = first->b_end; b < a.B;) {
    PagedPlan pl;
    plan_launch<TREE>(a, cu_len_host, kv_host, b, &pl);
    if (!pl.ok) return 0;
    most = std::max(most, pl.part_rows);
    b = pl.b_end;
  }
  return plan_bytes(a, most);
}

template <bool TREE>
cudaError_t run(PagedArgs a, const int32_t* cu_len_host, const int32_t* kv_host, const PagedPlan& first, void* workspace,
                cudaStream_t s) {
  a.sched = static_cast<unsigned*>(workspace);
  PagedPlan later;
  for (int b = 0; b < a.B;) {
    if (b > 0) plan_launch<TREE>(a, cu_len_host, kv_host, b, &later);
    const PagedPlan& pl = b > 0 ? later : first;
    b = pl.b_end;
    if (pl.n_items == 0) continue;
    a.chunk_tiles = pl.chunk_tiles;
    a.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + ATTN_SCHED_BYTES);
    a.part_lse = a.part_o + (size_t)pl.part_rows * a.Hq * a.D;
    a.tok = pl.pair ? 2 * a.tok_tile : a.tok_tile;
    const auto f = a.D == 128 ? launch<128, TREE, false> : pl.pair ? launch<64, TREE, true> : launch<64, TREE, false>;
    const cudaError_t e = f(a, pl, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int D, bool TREE, bool PAIR>
cudaError_t opt_in() {
  return cudaFuncSetAttribute(k_attn_paged<D, TREE, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)smem_bytes<D, PAIR>());
}

}  // namespace

cudaError_t attn_paged_prepare() {
  cudaError_t e = opt_in<128, false, false>();
  if (e == cudaSuccess) e = opt_in<128, true, false>();
  if (e == cudaSuccess) e = opt_in<64, false, false>();
  if (e == cudaSuccess) e = opt_in<64, true, false>();
  if (e == cudaSuccess) e = opt_in<64, false, true>();
  if (e == cudaSuccess) e = opt_in<64, true, true>();
  return e;
}

size_t attn_paged_workspace(const PagedArgs& a, const int32_t* cu_len_host, const int32_t* kv_host, PagedPlan* first) {
  return cu_len_host ? workspace_of<false>(a, cu_len_host, kv_host, first) : workspace_of<true>(a, cu_len_host, kv_host, first);
}

cudaError_t launch_attn_paged(const PagedArgs& a, const int32_t* cu_len_host, const int32_t* kv_host,
                              const PagedPlan& first, void* workspace, cudaStream_t s) {
  return cu_len_host ? run<false>(a, cu_len_host, kv_host, first, workspace, s)
                     : run<true>(a, cu_len_host, kv_host, first, workspace, s);
}

}  // namespace ts
