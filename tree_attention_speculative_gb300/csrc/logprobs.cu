// Log probabilities of given tokens, entropies and the most likely alternatives of
// rows of logits, in one pass over the rows.
//
// With y = (x - m) log2(e) / temperature over a row, m its maximum,
//   S = sum 2^y,  U = sum 2^y y:   log p(x) = (x - m) / temperature - ln 2 log2 S,
//                                  entropy  = ln 2 (log2 S - U / S).
// Each thread keeps m, S and U of its values (rescaled when its m grows), which are
// joined over the CTA and over the row's cluster.  All terms of U have one sign.
// A value of -inf, or so low that 2^y is 0 in fp32, adds nothing to either.
//
// The alternatives.  A thread also remembers the largest of its values, which
// 16-byte vector holds it, and the largest of its other vectors.  At the row's end the
// CTA finds the `top` threads whose largest are best (by value, then by the lower
// index): the row's best `top` values are all in those threads' columns, since every
// value elsewhere is behind `top` better ones.  Such a thread reads its vector again;
// where another of its vectors reaches the last of those largest too, which is rare,
// a warp reads its whole column.  What reaches it is ranked.  So the pass over the row
// has no exchange between threads and no list to keep.
//
// Memory-bound: a row is read once.  A cluster of 1 to 8 CTAs takes a row, more
// where there are few; CTA 0 joins the CTAs' results over distributed shared
// memory, so there is no workspace.  2048 fp32 rows of 128256, 20 alternatives: 181 us,
// 5.8 TB/s, 0.85 of the copy rate; without alternatives 164, reading the columns of the
// k threads whole 194.  The same in bf16 125 (half the bytes, the same conversions and
// exponentials); 96 rows (49 MB, part of them in L2 from the call before) 16 us, one row
// 8.7: latency.
#include <cooperative_groups.h>

#include <algorithm>

#include "fastexp.cuh"
#include "internal.cuh"

namespace ts {
namespace {

namespace cg = cooperative_groups;

// Threads a CTA: 256, four CTAs an SM (a row's end is shorter, and more of the others
// run beside it), where a CTA then still holds a whole row; else 512.  4096 rows of
// 32000 100 us (122 with 512), 500 of 1000 7.1 (11.4), 2048 bf16 rows of 128256 124
// (138); 2048 fp32 rows of 128256, two CTAs of 256 a row, 194 (179).
constexpr int LP_FEW = 256, LP_MANY = 512;
constexpr int LP_COLUMN = 64;     // vectors a thread at most: two a lane when a warp reads a column again
constexpr int LP_SM_THREADS = 1024;  // threads that run on an SM at once
constexpr float LP_LOW = -200.f;  // 2^LOW is 0 in fp32

// Larger float, larger unsigned; -0 as +0.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
constexpr uint32_t ORDERED_NEG_INF = 0x007fffffu;  // ordered(-inf): not above it, no alternative

__device__ __forceinline__ float lp_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4, UN = 4;  // values a vector; vectors in flight a thread
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[4]) {
    v[0] = __uint_as_float(r.x);
    v[1] = __uint_as_float(r.y);
    v[2] = __uint_as_float(r.z);
    v[3] = __uint_as_float(r.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8, UN = 2;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&v)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
};
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }

// A row cut into 16-byte vectors at 16-byte boundaries: vector j holds elements
// j * N - lead .. of it; the first and the last may stick out of the row.
template <typename T>
struct Row {
  const T* x;
  int V, lead, vecs;
  __device__ __forceinline__ Row(const T* p, int v) : x(p), V(v) {
    lead = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    vecs = (lead + v + Vec<T>::N - 1) / Vec<T>::N;
  }
  __device__ __forceinline__ bool whole(int j) const { return j * Vec<T>::N >= lead && (j + 1) * Vec<T>::N - lead <= V; }
  __device__ __forceinline__ uint4 raw(int j) const {
    uint4 r;
    const T* p = x + (j * Vec<T>::N - lead);
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(reinterpret_cast<uint64_t>(p)));
    return r;
  }
  __device__ __forceinline__ void part(int j, float (&v)[Vec<T>::N]) const {
#pragma unroll
    for (int e = 0; e < Vec<T>::N; ++e) {
      const int i = j * Vec<T>::N - lead + e;
      v[e] = i >= 0 && i < V ? widen(x[i]) : -INFINITY;
    }
  }
  __device__ __forceinline__ void get(int j, float (&v)[Vec<T>::N]) const {
    if (whole(j)) Vec<T>::unpack(raw(j), v);
    else part(j, v);
  }
};

struct Stats {
  float m, s, u;
};
// b joined to a, both over the same scale k.
__device__ __forceinline__ Stats join(const Stats& a, const Stats& b, float k) {
  const float m = fmaxf(a.m, b.m);
  const float base = m == -INFINITY ? 0.f : m;
  const float da = fmaxf((a.m - base) * k, LP_LOW), db = fmaxf((b.m - base) * k, LP_LOW);
  const float fa = lp_ex2(da), fb = lp_ex2(db);
  Stats r;
  r.m = m;
  r.s = fa * a.s + fb * b.s;
  r.u = fa * (a.u + da * a.s) + fb * (b.u + db * b.s);
  return r;
}

template <int LP_THREADS>
struct Shared {
  static constexpr int LP_WARPS = LP_THREADS / 32;
  Stats warp[LP_WARPS];
  Stats all;                                   // the CTA's
  unsigned long long best[LOGPROB_MAX_TOP];    // its alternatives, best first; 0: none
  int column[LOGPROB_MAX_TOP];                 // the columns read again
  int n_columns, n_found;
  uint32_t low[LP_WARPS], high[LP_WARPS];      // of the threads' largest
  float token;                                 // the given token's logit
  unsigned long long found[LP_COLUMN / 32 * LOGPROB_MAX_TOP * LOGPROB_MAX_TOP];
};

// Every thread of the CTA: how many have pred set.
__device__ __forceinline__ int count(bool pred) { return __syncthreads_count(pred); }

// found[0 .. n) ranked: the best `top` to best[], in order.  Keys are distinct.
template <int LP_THREADS>
__device__ __forceinline__ void rank_found(Shared<LP_THREADS>& sh, int n, int top) {
  for (int c = threadIdx.x; c < n; c += LP_THREADS) {
    const unsigned long long key = sh.found[c];
    int rank = 0;
    for (int o = 0; o < n; ++o) rank += sh.found[o] > key;
    if (rank < top) sh.best[rank] = key;
  }
}

template <typename T, int LP_THREADS>
__global__ void __launch_bounds__(LP_THREADS, LP_SM_THREADS / LP_THREADS)
k_logprobs(const __grid_constant__ LogprobArgs a) {
  constexpr int LP_WARPS = LP_THREADS / 32;
  constexpr int N = Vec<T>::N, LP_UN = Vec<T>::UN;
  __shared__ Shared<LP_THREADS> sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), ranks = cluster.num_blocks();
  const int r = blockIdx.x / ranks;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  const long long src = a.rows ? a.rows[r] : r;
  if (src < 0 || src >= a.M) return;  // the same on every CTA of the cluster
  const Row<T> row(static_cast<const T*>(a.logits) + src * a.row_stride, a.V);
  const int j0 = rank * a.slice, j1 = min(j0 + a.slice, row.vecs);  // this CTA's vectors
  const float k = a.inv_temp_log2e;

  // One pass: batches of LP_UN vectors.
  Stats st{-INFINITY, 0.f, 0.f};
  float best_v = -INFINITY, next_v = -INFINITY;  // the largest, and that of the other vectors
  int best_j = -1;
  // the next batch's loads are in flight while one is at work
  const auto whole = [&](int j) {
    const int last = j + (LP_UN - 1) * LP_THREADS;
    return last < j1 && row.whole(j) && row.whole(last);
  };
  uint4 next[LP_UN];
  bool loaded = whole(j0 + tid);
  if (loaded) {
#pragma unroll
    for (int u = 0; u < LP_UN; ++u) next[u] = row.raw(j0 + tid + u * LP_THREADS);
  }
  if (rank == 0 && tid == LP_THREADS - 1 && a.tokens) {
    const int t = a.tokens[r];
    sh.token = t >= 0 && t < a.V ? widen(row.x[t]) : 0.f;
  }
  for (int j = j0 + tid; j < j1; j += LP_UN * LP_THREADS) {
    float v[LP_UN][N];
    if (loaded) {
#pragma unroll
      for (int u = 0; u < LP_UN; ++u) Vec<T>::unpack(next[u], v[u]);
    } else {
#pragma unroll
      for (int u = 0; u < LP_UN; ++u) {
        if (j + u * LP_THREADS < j1) {
          row.get(j + u * LP_THREADS, v[u]);
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e) v[u][e] = -INFINITY;
        }
      }
    }
    const int jn = j + LP_UN * LP_THREADS;
    loaded = whole(jn);
    if (loaded) {
#pragma unroll
      for (int u = 0; u < LP_UN; ++u) next[u] = row.raw(jn + u * LP_THREADS);
    }
    float top = st.m;
#pragma unroll
    for (int u = 0; u < LP_UN; ++u) {
      float vm = v[u][0];
#pragma unroll
      for (int e = 1; e < N; ++e) vm = fmaxf(vm, v[u][e]);
      if (vm > best_v) {
        next_v = best_v;
        best_v = vm;
        best_j = j + u * LP_THREADS;
      } else {
        next_v = fmaxf(next_v, vm);
      }
      top = fmaxf(top, vm);
    }
    if (top > st.m) {
      const float d = fmaxf((st.m - top) * k, LP_LOW);
      const float f = lp_ex2(d);
      st.u = f * (st.u + d * st.s);
      st.s *= f;
      st.m = top;
    }
    const float base = st.m == -INFINITY ? 0.f : st.m;
    uint64_t s2 = 0ull, u2 = 0ull;
    const uint64_t nb2 = fx::pack2(-base, -base), k2 = fx::pack2(k, k);
#pragma unroll
    for (int u = 0; u < LP_UN; ++u) {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        float y0, y1;
        fx::unpack2(fx::mul2(fx::add2(fx::pack2(v[u][e], v[u][e + 1]), nb2), k2), y0, y1);
        y0 = fmaxf(y0, LP_LOW);
        y1 = fmaxf(y1, LP_LOW);
        const uint64_t p2 = fx::pack2(lp_ex2(y0), lp_ex2(y1));
        s2 = fx::add2(s2, p2);
        u2 = fx::fma2(p2, fx::pack2(y0, y1), u2);
      }
    }
    float x0, x1;
    fx::unpack2(s2, x0, x1);
    st.s += x0 + x1;
    fx::unpack2(u2, x0, x1);
    st.u += x0 + x1;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stats b;
    b.m = __shfl_xor_sync(0xffffffffu, st.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, st.s, o);
    b.u = __shfl_xor_sync(0xffffffffu, st.u, o);
    st = join(st, b, k);
  }
  if (lane == 0) sh.warp[warp] = st;
  if (tid == 0) sh.n_columns = sh.n_found = 0;
  if (tid < LOGPROB_MAX_TOP) sh.best[tid] = 0ull;
  __syncthreads();
  if (warp == 0) {
    Stats b = lane < LP_WARPS ? sh.warp[lane] : Stats{-INFINITY, 0.f, 0.f};
#pragma unroll
    for (int o = LP_WARPS / 2; o > 0; o >>= 1) {
      Stats c;
      c.m = __shfl_xor_sync(0xffffffffu, b.m, o);
      c.s = __shfl_xor_sync(0xffffffffu, b.s, o);
      c.u = __shfl_xor_sync(0xffffffffu, b.u, o);
      b = join(b, c, k);
    }
    if (lane == 0) sh.all = b;
  }

  const int top = a.top;
  if (top > 0) {
    // The value that the top-th best of the threads' largest reaches, bit by bit
    // from above, until as many threads reach it as are wanted.
    const bool any = best_v > -INFINITY;
    const uint32_t mine = any ? ordered(best_v) : 0u;
    uint32_t least = ORDERED_NEG_INF + 1;
    int reach = count(any);
    if (reach > top) {
      // (the bits that all of them share need no search)
      const uint32_t wl = __reduce_min_sync(0xffffffffu, any ? mine : 0xffffffffu), wh = __reduce_max_sync(0xffffffffu, mine);
      if (lane == 0) {
        sh.low[warp] = wl;
        sh.high[warp] = wh;
      }
      __syncthreads();
      const uint32_t lo = __reduce_min_sync(0xffffffffu, sh.low[lane % LP_WARPS]);
      const uint32_t hi = __reduce_max_sync(0xffffffffu, sh.high[lane % LP_WARPS]);
      const int first = 31 - __clz(lo ^ hi);  // -1: all alike
      uint32_t bits = first < 0 ? lo : first == 31 ? 0u : lo >> (first + 1) << (first + 1);
      for (int bit = first; bit >= 0 && reach != top; --bit) {
        const uint32_t trial = bits | (1u << bit);
        const int n = count(any && mine >= trial);
        if (n >= top) {
          bits = trial;
          reach = n;
        }
      }
      least = max(bits, least);
    }
    bool in = any && mine >= least;
    if (reach > top) {
      // more threads share that very value: of those the lowest indices
      const int above = count(mine > least);
      uint32_t limit = 0;  // the largest vector number with fewer than enough below it
      for (int bit = 30; bit >= 0; --bit) {
        const uint32_t trial = limit | (1u << bit);
        if (count(in && mine == least && (uint32_t)best_j < trial) < top - above) limit = trial;
      }
      in = in && (mine > least || (uint32_t)best_j <= limit);
    }
    const auto key_of = [&](float v, int i) {  // i: its index in the row
      const uint32_t o = ordered(v);
      return o >= least ? ((unsigned long long)o << 32) | (0xffffffffu - (uint32_t)i) : 0ull;
    };
    if (in && ordered(next_v) < least) {
      float v[N];
      row.get(best_j, v);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const unsigned long long key = key_of(v[e], best_j * N - row.lead + e);
        if (key) sh.found[atomicAdd(&sh.n_found, 1)] = key;
      }
    } else if (in) {
      sh.column[atomicAdd(&sh.n_columns, 1)] = tid;
    }
    __syncthreads();
    const int columns = min(sh.n_columns, top);
    for (int ch = warp; ch < columns * (LP_COLUMN / 32); ch += LP_WARPS) {
      const int j = j0 + sh.column[ch / (LP_COLUMN / 32)] + (lane + ch % (LP_COLUMN / 32) * 32) * LP_THREADS;
      float v[N];
      if (j < j1) {
        row.get(j, v);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = -INFINITY;
      }
      unsigned long long key[N];
      int n = 0;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        key[e] = key_of(v[e], j * N - row.lead + e);
        n += key[e] != 0ull;
      }
      const int all = __reduce_add_sync(0xffffffffu, n);
      if (all <= top) {
        int at = 0;
        if (n) at = atomicAdd(&sh.n_found, n);
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (key[e]) sh.found[at++] = key[e];
      } else {  // the best `top` of these, one after the other
        int at = 0;
        if (lane == 0) at = atomicAdd(&sh.n_found, top);
        at = __shfl_sync(0xffffffffu, at, 0);
        for (int t = 0; t < top; ++t) {
          unsigned long long b = 0;
#pragma unroll
          for (int e = 0; e < N; ++e) b = key[e] > b ? key[e] : b;
          const unsigned long long mine_b = b;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long c2 = __shfl_xor_sync(0xffffffffu, b, o);
            b = c2 > b ? c2 : b;
          }
          if (mine_b == b) {
#pragma unroll
            for (int e = 0; e < N; ++e)
              if (key[e] == b) key[e] = 0ull;
          }
          if (lane == 0) sh.found[at + t] = b;
        }
      }
    }
    __syncthreads();
    rank_found(sh, sh.n_found, top);
  }
  cluster.sync();
  if (rank == 0) {
    if (ranks > 1) {
      // the other CTAs' lists beside this one's, ranked again
      if (top > 0) {
        for (int e = tid; e < ranks * top; e += LP_THREADS) {
          const int c = e / top;
          sh.found[e] = cluster.map_shared_rank(&sh, c)->best[e - c * top];
        }
        __syncthreads();
        if (tid < LOGPROB_MAX_TOP) sh.best[tid] = 0ull;
        __syncthreads();
        const int n = ranks * top;
        for (int c = tid; c < n; c += LP_THREADS) {
          const unsigned long long key = sh.found[c];
          if (key == 0ull) continue;
          int place = 0;
          for (int o = 0; o < n; ++o) place += sh.found[o] > key;
          if (place < top) sh.best[place] = key;
        }
      }
      if (tid == 0) {
        Stats b = sh.all;
        for (int c = 1; c < ranks; ++c) b = join(b, cluster.map_shared_rank(&sh, c)->all, k);
        sh.all = b;
      }
    }
    __syncthreads();
    const Stats b = sh.all;
    const bool empty = b.m == -INFINITY;  // nothing in the row has any probability
    const float ls = log2f(b.s);
    constexpr float LN2 = 0.69314718055994531f;
    if (tid == 0) {
      if (a.logprob) {
        const int t = a.tokens[r];
        float lp = t == -1 ? 0.f : NAN;
        if (t >= 0 && t < a.V) lp = empty ? -INFINITY : (sh.token - b.m) * a.inv_temp - ls * LN2;
        a.logprob[r] = lp;
      }
      if (a.entropy) a.entropy[r] = empty ? 0.f : (ls - b.u / b.s) * LN2;
    }
    if (tid < top) {
      const unsigned long long key = sh.best[tid];
      const size_t at = (size_t)r * top + tid;
      if (a.top_ids) a.top_ids[at] = key ? (int)(0xffffffffu - (uint32_t)key) : -1;
      if (a.top_logprobs) a.top_logprobs[at] = key ? (unordered((uint32_t)(key >> 32)) - b.m) * a.inv_temp - ls * LN2 : -INFINITY;
    }
  }
  if (ranks > 1) cluster.sync();  // the CTAs' shared memory stays until it has been read
}

template <typename T, int LP_THREADS>
cudaError_t launch(LogprobArgs a, int vecs, cudaStream_t s) {
  // CTAs a row: one, or as many as the SMs hold at once where there are few rows
  // (and a CTA keeps a vector for each thread), or a thread's column allows.  96 rows of
  // 128256: 3 a row 16.3 us, 1 20.4, 6 29; 8 rows, 8 a row 9.1, 4 8.9, 2 10.4.
  int c = PLAN_SMS * (LP_SM_THREADS / LP_THREADS) / a.R;
  c = std::min(std::min(c, 8), vecs / LP_THREADS);
  c = std::max(c, ceil_div(vecs, LP_COLUMN * LP_THREADS));
  if (c < 1) c = 1;
  a.slice = ceil_div(vecs, c);
  cudaLaunchConfig_t cfg{};
  if ((long long)a.R * c > 0x7fffffffll) return cudaErrorInvalidValue;
  cfg.gridDim = dim3((unsigned)(a.R * c));
  cfg.blockDim = dim3(LP_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = c;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_logprobs<T, LP_THREADS>, a);
}

template <typename T>
cudaError_t launch(const LogprobArgs& a, cudaStream_t s) {
  const int vecs = a.V / Vec<T>::N + 2;
  return vecs <= LP_COLUMN * LP_FEW ? launch<T, LP_FEW>(a, vecs, s) : launch<T, LP_MANY>(a, vecs, s);
}

}  // namespace

cudaError_t launch_logprobs(LogprobArgs a, cudaStream_t s) {
  return a.half ? launch<__nv_bfloat16>(a, s) : launch<float>(a, s);
}

}  // namespace ts
