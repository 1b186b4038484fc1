// Writing the 8-bit paged KV cache: prompt tokens (k_append_q8) and accepted
// paths (k_commit_q8), quantised row by row as they are stored (quant_row.cuh).
//
// Both are memory-bound: 2D bytes of bf16 read and D + 1 written a row.  D/8
// lanes take a row, 16 bytes each, so a warp reads whole 512-byte runs, and
// the row's maximum is a few shuffles.
//
// k_append_q8: a CTA takes a run of (token, head) rows, whatever sequences
// they belong to.  One thread a token first finds the token's sequence (a
// binary search of cu_len) and its destination row, while the CTA's first rows
// are already on their way; rows with no valid destination are not stored.
// Warps of the first CTAs check a whole sequence each and write its new
// length: a sequence with a bad block keeps its old one, so what was written
// past it never counts.
//
// k_commit_q8: one CTA a sequence, which checks every destination before it
// writes any, so a sequence is never left half-committed; the new length is
// written after a barrier, so it may alias the old one.
#include "append.cuh"
#include "quant_row.cuh"

namespace ts {
namespace {

constexpr int APPEND_THREADS = 256;
constexpr int APPEND_MAX_ROWS = 64;  // (token, head) rows a CTA at most, K and V each
constexpr int COMMIT_Q8_THREADS = 512;

// Eight CTAs an SM (32 registers): 149K tokens of 8 heads of 128 in 127 us, 6.7
// TB/s, against 134 us with five (45 registers; 16 tokens then take 3.1 us, not 3.4).
template <int D>
__global__ void __launch_bounds__(APPEND_THREADS, 8)
k_append_q8(const __grid_constant__ AppendArgs a, FastDiv heads) {
  constexpr int LANES = D / 8;
  constexpr int GROUPS = APPEND_THREADS / LANES;
  constexpr int UN = 2;  // rows in flight a thread, K and V each
  __shared__ long long dest[APPEND_MAX_ROWS + 1];  // pool row of head 0 of each token of the CTA, or -1
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();

  if ((int)blockIdx.x < a.len_ctas) {  // a warp a sequence: its blocks and its new length
    const int b = blockIdx.x * (APPEND_THREADS / 32) + warp;
    if (b >= a.B) return;
    append_sequence(a, b, lane);
    return;
  }

  const long long total = (long long)a.T * a.Hkv;
  const long long u0 = (long long)(blockIdx.x - a.len_ctas) * a.rows;
  const int n = (int)min((long long)a.rows, total - u0);
  const int t0 = (int)(u0 / a.Hkv), g0 = (int)(u0 - (long long)t0 * a.Hkv);
  const int ntok = heads.div(g0 + n - 1) + 1;
  const int grp = threadIdx.x / LANES, sub = threadIdx.x % LANES;

  uint4 kx[UN], vx[UN];
  const auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int r = r0 + u * GROUPS;
      if (r < n) {
        const int k = heads.div(g0 + r);
        const size_t head = (size_t)(g0 + r - k * a.Hkv) * D + sub * 8;
        kx[u] = *reinterpret_cast<const uint4*>(a.k + (size_t)(t0 + k) * a.k_token + head);
        vx[u] = *reinterpret_cast<const uint4*>(a.v + (size_t)(t0 + k) * a.v_token + head);
      } else {
        kx[u] = vx[u] = make_uint4(0, 0, 0, 0);
      }
    }
  };
  load(grp);
  if ((int)threadIdx.x < ntok) dest[threadIdx.x] = append_place(a, t0 + threadIdx.x).row;
  __syncthreads();
  const int rounds = (n + GROUPS * UN - 1) / (GROUPS * UN);  // the same on every lane: the shuffles need them all
  for (int it = 0; it < rounds; ++it) {
    const int r0 = grp + it * GROUPS * UN;
    if (it > 0) load(r0);
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int r = r0 + u * GROUPS;
      int ks, vs;
      const uint2 kc = q8_row<LANES>(kx[u], &ks);
      const uint2 vc = q8_row<LANES>(vx[u], &vs);
      if (r < n) {
        const int k = heads.div(g0 + r);
        const long long base = dest[k];
        if (base >= 0) {
          const size_t row = (size_t)base + (size_t)(g0 + r - k * a.Hkv) * a.bs;
          *reinterpret_cast<uint2*>(a.k_cache + row * D + sub * 8) = kc;
          *reinterpret_cast<uint2*>(a.v_cache + row * D + sub * 8) = vc;
          if (sub == 0) reinterpret_cast<uint16_t*>(a.kv_scale)[row] = (uint16_t)(ks | (vs << 8));
        }
      }
    }
  }
}

template <int D>
__global__ void __launch_bounds__(COMMIT_Q8_THREADS)
k_commit_q8(const __grid_constant__ CommitQ8Args a, FastDiv heads) {
  constexpr int LANES = D / 8;
  constexpr int GROUPS = COMMIT_Q8_THREADS / LANES;
  __shared__ long long dest[MAX_NODES];  // pool row of head 0 of each path step
  __shared__ int node[MAX_NODES];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x;
  const int P = a.prefix_len[b];
  const int L = a.accept_len[b];
  const int st = a.status ? a.status[b] : TS_OK;
  // a path has at most N steps
  const bool commit = st == TS_OK && L >= 0 && L <= a.max_depth && L < a.N && P >= 0 && P <= APPEND_MAX_LEN;
  const int steps = commit ? L + 1 : 0;
  bool ok = true;
  if ((int)threadIdx.x < steps) {
    const int d = threadIdx.x;
    const int x = a.accepted[(size_t)b * (a.max_depth + 1) + d];
    const int i = (P + d) / a.bs;
    const int blk = i < a.max_blocks ? a.block_table[(size_t)b * a.max_blocks + i] : -1;
    ok = x >= 0 && x < a.N && blk >= 0 && blk < a.num_blocks;
    node[d] = x;
    dest[d] = (long long)blk * a.Hkv * a.bs + (P + d - i * a.bs);
  }
  const bool write = __syncthreads_and(ok) && commit;
  if (write) {
    const int n = steps * a.Hkv;
    const int grp = threadIdx.x / LANES, sub = threadIdx.x % LANES;
    const int rounds = (n + GROUPS - 1) / GROUPS;
    for (int it = 0; it < rounds; ++it) {
      const int r = grp + it * GROUPS;
      uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
      size_t row = 0;
      if (r < n) {
        const int d = heads.div(r), g = r - d * a.Hkv;
        const size_t src = (((size_t)b * a.N + node[d]) * a.Hkv + g) * D + sub * 8;
        kx = *reinterpret_cast<const uint4*>(a.k_tree + src);
        vx = *reinterpret_cast<const uint4*>(a.v_tree + src);
        row = (size_t)dest[d] + (size_t)g * a.bs;
      }
      int ks, vs;
      const uint2 kc = q8_row<LANES>(kx, &ks);
      const uint2 vc = q8_row<LANES>(vx, &vs);
      if (r < n) {
        *reinterpret_cast<uint2*>(a.k_cache + row * D + sub * 8) = kc;
        *reinterpret_cast<uint2*>(a.v_cache + row * D + sub * 8) = vc;
        if (sub == 0) reinterpret_cast<uint16_t*>(a.kv_scale)[row] = (uint16_t)(ks | (vs << 8));
      }
    }
  }
  if (threadIdx.x == 0) {
    a.new_prefix_len[b] = write ? P + L + 1 : P;  // every thread read prefix_len before the barrier
    if (st == TS_OK && !write && a.status) {
      if (commit) a.status[b] = TS_ERR_BAD_BLOCK;
    }
  }
}

}  // namespace

cudaError_t launch_append_q8(AppendArgs a, cudaStream_t s) {
  // Rows a CTA: one round of its row groups (32 rows of 128, 64 of 64), so that
  // few rows spread over the SMs; past four waves of CTAs 64 rows, which halves
  // the searches.  8 heads of 128: 149K tokens 127 us (32 rows 135 us), 4K tokens
  // 6.4 us (64 rows 6.8 us), 16 tokens 3.4 us (4.5 us).  Heads of 64 on 32 rows,
  // half a round: 15.2 against 10.8 us for 16K tokens.
  const long long total = (long long)a.T * a.Hkv;
  a.rows = a.D == 64 || total > (long long)APPEND_MAX_ROWS * 4 * PLAN_SMS ? APPEND_MAX_ROWS : APPEND_MAX_ROWS / 2;
  a.len_ctas = ceil_div(a.B, APPEND_THREADS / 32);
  const long long ctas = (total + a.rows - 1) / a.rows + a.len_ctas;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  const FastDiv fd = FastDiv::make(a.Hkv);
  return a.D == 128 ? launch_pdl(k_append_q8<128>, dim3((unsigned)ctas), dim3(APPEND_THREADS), 0, s, a, fd)
                    : launch_pdl(k_append_q8<64>, dim3((unsigned)ctas), dim3(APPEND_THREADS), 0, s, a, fd);
}

cudaError_t launch_commit_q8(const CommitQ8Args& a, cudaStream_t s) {
  const FastDiv fd = FastDiv::make(a.Hkv);
  return a.D == 128 ? launch_pdl(k_commit_q8<128>, dim3(a.B), dim3(COMMIT_Q8_THREADS), 0, s, a, fd)
                    : launch_pdl(k_commit_q8<64>, dim3(a.B), dim3(COMMIT_Q8_THREADS), 0, s, a, fd);
}

}  // namespace ts
