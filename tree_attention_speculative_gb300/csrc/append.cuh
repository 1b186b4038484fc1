// What the calls that append a ragged batch of new tokens to a paged cache share:
// the check of a sequence and its new length, and where a token goes.  A is an
// argument block with cu_len, prefix_len, block_table, new_prefix_len, status, B,
// T, Hkv, bs, num_blocks and max_blocks (treespec.h: tree_cache_append_q8).
#pragma once

#include "internal.cuh"

namespace ts {

constexpr int APPEND_MAX_LEN = 1 << 30;  // positions stay far inside 32 bits

// A warp checks sequence b, all of it, and writes its new length: one with a bad
// block keeps its old one, so what was written past it never counts.  Returns how
// many tokens it has become longer.
template <class A>
__device__ __forceinline__ int append_sequence(const A& a, int b, int lane) {
  const int P = a.prefix_len[b], c0 = a.cu_len[b], c1 = a.cu_len[b + 1];
  const int st = a.status ? a.status[b] : TS_OK;
  // its rows are its own: no sequence before it ends, and none after it begins, among them
  bool own = true;
#pragma unroll 4
  for (int i = lane; i <= a.B; i += 32) {
    const int c = a.cu_len[i];
    own = own && (i <= b ? c <= c0 : c >= c1);
  }
  own = __all_sync(0xffffffffu, own);
  const bool sized = own && P >= 0 && P <= APPEND_MAX_LEN && c0 >= 0 && c1 >= c0 && c1 <= a.T &&
                     c1 - c0 <= APPEND_MAX_LEN - P;
  bool ok = sized;
  if (sized && c1 > c0) {
    const int last = (P + (c1 - c0) - 1) / a.bs;
    for (int i = P / a.bs + lane; i <= last; i += 32) {
      const int blk = i < a.max_blocks ? a.block_table[(size_t)b * a.max_blocks + i] : -1;
      if (blk < 0 || blk >= a.num_blocks) {
        ok = false;
        break;
      }
    }
  }
  ok = __all_sync(0xffffffffu, ok);
  const int longer = ok && st == TS_OK ? c1 - c0 : 0;
  if (lane == 0) {
    a.new_prefix_len[b] = P + longer;
    if (!ok && st == TS_OK && a.status) a.status[b] = sized ? TS_ERR_BAD_BLOCK : TS_ERR_SHAPE;
  }
  return longer;
}

// Whether cu_len rises throughout, which makes every sequence's rows its own: this
// thread's part of the answer (all `threads` of them are to hold).
template <class A>
__device__ __forceinline__ bool append_ordered(const A& a, int thread, int threads) {
  bool ok = true;
  for (int i = thread; i < a.B; i += threads) ok = ok && a.cu_len[i] <= a.cu_len[i + 1];
  return ok;
}

// Where it does not: whether the rows of the sequence that append_place found for
// token t are its own (append_sequence's test).
template <class A>
__device__ __forceinline__ bool append_owns(const A& a, int t) {
  int lo = 0, hi = a.B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_len[mid + 1] <= t) lo = mid + 1;
    else hi = mid;
  }
  if (lo == a.B) return false;
  const int c0 = a.cu_len[lo], c1 = a.cu_len[lo + 1];
  bool own = true;
  for (int i = 0; i <= a.B; ++i) own = own && (i <= lo ? a.cu_len[i] <= c0 : a.cu_len[i] >= c1);
  return own;
}

// Token t's position (-1: it is no sequence's, or its sequence gets nothing) and
// the pool row of its KV head 0 (-1: no valid block).
struct AppendPlace {
  int pos;
  long long row;
};
template <class A>
__device__ __forceinline__ AppendPlace append_place(const A& a, int t) {
  // the sequence b with cu_len[b] <= t < cu_len[b + 1]
  int lo = 0, hi = a.B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_len[mid + 1] <= t) lo = mid + 1;
    else hi = mid;
  }
  AppendPlace p{-1, -1};
  if (lo < a.B) {
    const int c0 = a.cu_len[lo], c1 = a.cu_len[lo + 1], P = a.prefix_len[lo];
    const int st = a.status ? a.status[lo] : TS_OK;
    if (st == TS_OK && c0 >= 0 && t >= c0 && t < c1 && c1 <= a.T && P >= 0 && P <= APPEND_MAX_LEN &&
        c1 - c0 <= APPEND_MAX_LEN - P) {
      p.pos = P + (t - c0);
      const int i = p.pos / a.bs;
      const int blk = i < a.max_blocks ? a.block_table[(size_t)lo * a.max_blocks + i] : -1;
      if (blk >= 0 && blk < a.num_blocks) p.row = (long long)blk * a.Hkv * a.bs + (p.pos - i * a.bs);
    }
  }
  return p;
}

}  // namespace ts
