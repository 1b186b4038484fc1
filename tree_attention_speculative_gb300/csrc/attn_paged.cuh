// What the kernels of attn_paged.cu share: a call's sequences as they are
// planned, and which tiles of the cache a tile of rows has to see.
#pragma once

#include "internal.cuh"

namespace ts {

constexpr int PAGED_MAX_SEQS = 256;  // sequences a launch; more go in several

// One sequence of a launch.  Its items are numbered item0 .. : row tiles or pairs of
// them (the last, which see the most keys, first), splits, KV heads.
struct PagedSeq {
  int item0;
  int b;
  int row_tiles; // or pairs
  int splits;    // its chains of key tiles are cut in so many at most
  int rows;      // tokens it was planned for
  int part_row;  // splits > 1: its first row (a token's) among the partial results
};

// The sequences of a launch that had no rows when it was planned: [before[e], b) are those
// ahead of entry e's sequence b, [last + 1, end) those behind the last.
struct PagedGaps {
  int before[PAGED_MAX_SEQS];
  int last, end;
};

struct PagedArgs {
  const __nv_bfloat16* q;  // [T, Hq, D]
  const __nv_bfloat16* k_cache;
  const __nv_bfloat16* v_cache;
  const int32_t* block_table;
  const int32_t* cu_len;  // chunk: rows cu_len[b] .. cu_len[b+1]-1 are sequence b's
  const int32_t* kv_len;  // chunk: tokens in the cache, the rows' own last; tree: the verified prefix
  const int32_t* appended;  // chunk: how many rows are in the cache; null: all
  const __nv_bfloat16* k_tree;
  const __nv_bfloat16* v_tree;
  const uint64_t* anc_mask;
  __nv_bfloat16* out;
  float* lse;
  int32_t* status;
  unsigned* sched;  // item counter: zero before and after a launch
  float* part_o;    // [rows of cut chains, Hq, D] normalised, and
  float* part_lse;  // [.., Hq] their base-2 log-sum-exp
  int B, T, N, Hq, Hkv, G, D, W;  // N, W: tree
  int bs, num_blocks, max_blocks;
  float scale_log2;
  int window, sinks;  // window 0: every earlier key
  int chunk_tiles;    // key tiles a split at most, by the host's lengths
  int tok_tile;       // tokens a row tile: ROW_TILE / G
  int tok;            // tokens an item: of a row tile, or of a pair
  unsigned long long wait_limit_ns;
  int stall_seq, stall_tile, max_ctas;  // testing (internal.cuh: AttnArgs)
};

// The tiles of cached keys that rows from position `first` on, with keys below
// `hi` to see, have to read: n_sink tiles from 0 on, then those from win0 on.
// lo: the first key, past the sinks, that any of them sees.
struct PagedSpan {
  int lo, hi, n_sink, win0, n;
};
__host__ __device__ inline PagedSpan paged_span(int first, int hi, int window, int sinks) {
  PagedSpan s;
  s.hi = hi;
  s.lo = window > 0 && first - window + 1 > 0 ? first - window + 1 : 0;
  const int tiles = ceil_div(hi, KV_TILE);
  s.win0 = s.lo >= hi ? tiles : s.lo / KV_TILE;
  int sk = s.lo < hi ? s.lo : hi;
  if (sinks < sk) sk = sinks;
  s.n_sink = ceil_div(sk, KV_TILE);
  if (s.n_sink > s.win0) s.n_sink = s.win0;
  s.n = s.n_sink + tiles - s.win0;
  return s;
}
// The span of a row tile whose first token is the i0-th of `len`.
__host__ __device__ inline PagedSpan chunk_span(int kv, int len, int i0, int tok, int window, int sinks) {
  const int last = (i0 + tok < len ? i0 + tok : len) - 1;
  return paged_span(kv - len + i0, kv - len + last + 1, window, sinks);
}
// Splits of a chain of n tiles.  A chain that has outgrown its plan (a captured
// call, with longer sequences) keeps the planned number, of longer splits.
__host__ __device__ inline int paged_splits(int n, int chunk_tiles, int most) {
  const int s = ceil_div(n, chunk_tiles);
  return s < 1 ? 1 : s > most ? most : s;
}
// Tiles [n s / ps, n (s + 1) / ps) are split s of ps (n <= 2^23 + 2^23, s <= ps <= 256).
__host__ __device__ inline int paged_split_start(int n, int ps, int s) {
  return ps == 1 ? (s ? n : 0) : (int)((unsigned)n * (unsigned)s / (unsigned)ps);
}

// A launch: sequences [.., b_end) of the call, at most PAGED_MAX_SEQS with rows.
struct PagedPlan {
  PagedSeq seq[PAGED_MAX_SEQS];
  PagedGaps gaps;
  int n_seqs, n_items, chunk_tiles, b_end;
  long long part_rows;  // tokens' rows of partial results
  bool pair;            // an item takes two row tiles
  bool ok;              // its items and rows can be numbered
};

cudaError_t attn_paged_prepare();
// Bytes a call needs (0: more than a launch can number), and its first launch's plan.
// cu_len_host NULL: a tree.
size_t attn_paged_workspace(const PagedArgs& a, const int32_t* cu_len_host, const int32_t* kv_host, PagedPlan* first);
cudaError_t launch_attn_paged(const PagedArgs& a, const int32_t* cu_len_host, const int32_t* kv_host,
                              const PagedPlan& first, void* workspace, cudaStream_t s);

}  // namespace ts
