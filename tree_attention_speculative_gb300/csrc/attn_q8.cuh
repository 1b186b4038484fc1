// What the kernels of tree attention over the 8-bit paged cache share: the plan
// and its segments, bounded waits, the code loaders, and the conversions of
// values and queries.  attn_q8.cu says what they are for.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "quant_row.cuh"
#include "sm100.cuh"
#include "tensor_map.cuh"

namespace ts {

using namespace sm100;

constexpr int Q8_THREADS = 512;
constexpr int K_WARP = 0, QK_WARP = 1, PV_WARP = 2, V_WARP = 3, CONVERT_WARP0 = 4;
constexpr int NVB = 2;       // widened V tiles
constexpr int SLOT = 16384;  // a ring slot: 128 tokens of 128 codes, or a 64-column half of a bf16 tree tile
constexpr float NEG_INF = -INFINITY;
// fp32's least magnitude.  No row's factor is less, whatever its query and the scale:
// the logits of masked keys, -inf, times 0 would be NaN.
constexpr float LEAST = 1.401298464324817e-45f;
// Units of N * G up to FEW_ROWS rows with heads of 128 go to attn_q8_few.cu, which
// says how the two forms compare.  Its channels are the 128 MMA rows of O, so heads
// of 64 stay with attn_q8.cu.
constexpr int FEW_ROWS = 8;

// The CTAs' runs: CTA c starts at tile tile[c] of chain chain[c] and ends where
// c + 1 starts.  Chain (rt * B + b) * Hkv + g.
constexpr int MAX_CTAS = 256;
struct Runs {
  int n;
  int chain[MAX_CTAS + 1];
  int tile[MAX_CTAS + 1];
};

struct Q8Args {
  AttnArgs a;
  const uint8_t* kv_scale;
  // Parts of chains, rows being 128 here and FEW_ROWS in attn_q8_few.cu.
  float* part_o;     // [2 n, rows, D]: normalised
  float* part_lse;   // [2 n, rows]: base-2 log-sum-exp
  int box_rows, nodes_per_tile, units, n_tree;
  int out32;
  FastDiv fd_units, fd_hkv, fd_bs, fd_g;
  Runs runs;
};

// A segment: tiles [t_begin, t_begin + n_prefix) of a chain, and its tree tiles
// if it begins the chain.
struct Seg {
  int rt, b, g;
  int t_begin, n_prefix, n_tree, n_tiles;
  int P;
  bool p_ok;
  bool whole;  // all of the chain: its rows are the output
};
__host__ __device__ __forceinline__ Seg make_seg(int chain, int cta, int p_dev, const Q8Args& t) {
  Seg s;
  s.rt = t.fd_units.div(chain);
  const int u = chain - s.rt * t.units;
  s.b = t.fd_hkv.div(u);
  s.g = u - s.b * t.a.Hkv;
  const long long cap = min((long long)t.a.max_blocks * t.a.bs, 1ll << 30);
  s.P = (int)min((long long)max(p_dev, 0), cap);
  s.p_ok = s.P == p_dev;
  const int tiles = prefix_tiles(s.P);
  const bool from_start = chain != t.runs.chain[cta] || t.runs.tile[cta] == 0;
  const bool to_end = chain != t.runs.chain[cta + 1];
  s.t_begin = from_start ? 0 : min(t.runs.tile[cta], tiles);
  const int t_end = to_end ? tiles : min(t.runs.tile[cta + 1], tiles);
  s.n_prefix = max(t_end - s.t_begin, 0);
  s.n_tree = from_start ? t.n_tree : 0;
  s.n_tiles = s.n_prefix + s.n_tree;
  s.whole = from_start && to_end;
  return s;
}
__host__ __device__ __forceinline__ int seq_of(int chain, const Q8Args& t) {
  const int u = chain - t.fd_units.div(chain) * t.units;
  return t.fd_hkv.div(u);
}

struct Ctl {
  volatile int* flag;
  uint64_t limit;
};
// Bounded waits that also give up as soon as another role has aborted.  The
// polling is out of line: inlined at some twenty places, with the clock and the
// flag, it makes the kernel half as large again, and the warps at work wait for
// instructions (1.40 against 1.09 ms on 64 sequences of 8K tokens).
static __device__ __noinline__ bool wait_more(uint64_t* bar, uint32_t parity, volatile int* flag, uint64_t limit) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i) {
      if (mbar_try_wait(bar, parity)) return true;
    }
    if (*flag) return false;
    if (globaltimer_ns() - t0 > limit) {
      *flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, const Ctl& c) {
  return mbar_try_wait(bar, parity) || wait_more(bar, parity, c.flag, c.limit);
}
static __device__ __noinline__ bool wait_count(const int* counter, int target, volatile int* flag, uint64_t limit) {
  const uint32_t addr = smem_u32(counter);
  uint64_t t0 = 0;
#pragma unroll 1
  for (int i = 0;; ++i) {
    int v;
    asm volatile("ld.acquire.cta.shared::cta.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    if (v >= target) return true;
    if ((i & 15) == 15) {
      if (*flag) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > limit) {
        *flag = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait_count(const int* counter, int target, const Ctl& c) {
  return wait_count(counter, target, c.flag, c.limit);
}
__device__ __forceinline__ void publish(int* counter, int v) {
  asm volatile("st.release.cta.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(counter)), "r"(v) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float pow2_of(int biased) { return __uint_as_float((uint32_t)biased << 23); }

// A row's power of two as the multipliers of widen16: 2^(s - 127) * 2^120 in
// one bf16 pair, or where that is too large (s > 134), in two.
struct WideScale {
  uint32_t m1, m2;  // m1 is 0 for a row to be zeroed
  __device__ __forceinline__ WideScale(uint32_t s, bool keep) {
    const uint32_t b1 = min(s + 120u, 254u), b2 = s + 247u - b1;
    m1 = !keep ? 0u : s == 255u ? 0x7fff7fffu : (b1 << 7) | (b1 << 23);  // (255: a NaN row)
    m2 = (b2 << 7) | (b2 << 23);  // 1 for all but the largest rows
  }
};
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two bytes of w, each sign-extended to 16 bits (prmt's msb selector bit repeats a byte's sign).
template <uint32_t SEL>
__device__ __forceinline__ uint32_t two_bytes(uint32_t w) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(r) : "r"(w), "n"(SEL));
  return r;
}
// 16 codes times the row's power of two as bf16, two 16-byte chunks.  A code's
// sign, exponent and mantissa, put where bf16 has them, are its value times
// 2^-120 (subnormal codes too), so a bit shuffle and a product do: exact, and
// half the cost of going through fp16 and fp32.  (A NaN code would come out as a
// number, but rows that have any are marked by their scale byte.)
__device__ __forceinline__ void widen16(const uint4& c, uint32_t m1, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    // shifted so that a code's 4 + 3 bits end at bit 4
    o[2 * k] = mul_bf16x2((two_bytes<0x9180>(w[k]) << 4) & 0x87f087f0u, m1);
    o[2 * k + 1] = mul_bf16x2((two_bytes<0xb3a2>(w[k]) << 4) & 0x87f087f0u, m1);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// A node that no row sees may hold anything (the padding of a smaller tree),
// and 0 * inf is NaN: a row of tree values that are not all finite becomes
// zeros where no word of the mask column has its bit.
template <int D>
__device__ __noinline__ void clear_unseen(uint8_t* row, const uint64_t* word, int bit, int N, int W) {
  uint32_t top = 0;
#pragma unroll 1
  for (int c = 0; c < D / 8; ++c) {
    const uint4 y = *reinterpret_cast<const uint4*>(row + (c >> 3) * (KV_TILE * 128) + (((c ^ (threadIdx.x & 7)) & 7) << 4));
    top = q8_max2_nan(top, q8_max2_nan(q8_max2_nan(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu),
                                       q8_max2_nan(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu)));
  }
  if ((q8_max2_nan(top, top >> 16) & 0x7fffu) < 0x7f80u) return;
  uint64_t seen = 0;
#pragma unroll 1
  for (int n = 0; n < N; ++n) seen |= word[(size_t)n * W];
  if ((seen >> bit) & 1) return;
#pragma unroll 1
  for (int c = 0; c < D / 8; ++c)
    *reinterpret_cast<uint4*>(row + (c >> 3) * (KV_TILE * 128) + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
  fence_proxy_async();
}

// Four bf16 channels of a query times inv as e4m3: hi, and lo = what hi leaves.
__device__ __forceinline__ void split4(uint32_t w0, uint32_t w1, float inv, uint32_t& hi, uint32_t& lo) {
  uint32_t h[2], l[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t w = k ? w1 : w0;
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
    const float2 g = make_float2(f.x * inv, f.y * inv);
    h[k] = __nv_cvt_float2_to_fp8x2(g, __NV_SATFINITE, __NV_E4M3);
    const float2 u = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)h[k], __NV_E4M3)));
    l[k] = __nv_cvt_float2_to_fp8x2(make_float2(g.x - u.x, g.y - u.y), __NV_SATFINITE, __NV_E4M3);
  }
  hi = h[0] | (h[1] << 16);
  lo = l[0] | (l[1] << 16);
}

// 8 bytes from global to shared memory, asynchronously; cp_async_arrive arrives
// on the barrier once this thread's have landed.
__device__ __forceinline__ void cp_async8(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The K and V warps: a warp streams the run's codes of one pool into its ring
// (K: the tree's bf16 keys first, 64 channels a slot; V: with each tile its
// tokens' scale bytes).  `issued` counts the slots filled, for the teardown.
template <int D, class S>
__device__ __forceinline__ void load_codes(S& sm, const Q8Args& args, bool is_v, const CUtensorMap* tm_pool,
                                           const CUtensorMap* tm_kt, int cta, int chain0, int chain1, const Ctl& ctl,
                                           int& issued) {
  const AttnArgs& a = args.a;
  const int lane = threadIdx.x & 31;
  uint64_t* full = is_v ? sm.v_full : sm.k_full;
  uint64_t* empty = is_v ? sm.v_empty : sm.k_empty;
  const int nst = is_v ? S::NSV : S::NSK;
  const int g_box = args.box_rows, lg_boxes = __ffs(KV_TILE / g_box) - 1, g_boxes = 1 << lg_boxes;
  const int g_tpg = 32 >> lg_boxes;  // tiles a group of 32 table entries covers
  const uint32_t box_bytes = g_box * D;
  const int koff = (lane & (g_boxes - 1)) * g_box;
  const int row_step = args.fd_bs.mod(KV_TILE);
  int slot = 0, phase = 0;
  bool ok = true;
  // the next slot once it is free; false if the wait gave up
  auto take = [&]() -> bool {
    bool r = true;
    if (issued >= nst) {
      if (lane == 0) r = wait_bar(&empty[slot], phase ^ 1, ctl);
      r = __shfl_sync(0xffffffffu, r, 0);
    }
    return r;
  };
  auto next = [&]() {
    ++issued;
    if (++slot == nst) {
      slot = 0;
      phase ^= 1;
    }
  };
  int p_next = chain0 <= chain1 ? a.prefix_len[seq_of(chain0, args)] : 0;
  for (int chain = chain0; ok && chain <= chain1; ++chain) {
    const Seg I = make_seg(chain, cta, p_next, args);
    if (chain < chain1) p_next = a.prefix_len[seq_of(chain + 1, args)];  // on its way while this one runs
    const int stop = !is_v && I.b == a.stall_seq ? a.stall_tile : I.n_tiles;
    if (!is_v) {
      for (int tt = 0; ok && tt < I.n_tree; ++tt) {
        if (tt == stop) ok = false;
        for (int h = 0; ok && h < D / 64; ++h) {
          if (!(ok = take())) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&full[slot], KV_TILE * 128);
            tma_load_4d(sm.k[slot], tm_kt, &full[slot], 64 * h, I.g, tt * KV_TILE, I.b);
          }
          __syncwarp();
          next();
        }
      }
    }
    const int* table_row = a.block_table + (size_t)I.b * a.max_blocks;
    // lane L holds the table entry of box (L % boxes) of tile (L / boxes) of a
    // group of tiles; the next group loads while this one is issued
    auto load_group = [&](int grp) -> int {
      const int t = grp * g_tpg + (lane >> lg_boxes);
      const int t0 = (I.t_begin + t) * KV_TILE + koff;
      return t < I.n_prefix && t0 < I.P ? table_row[args.fd_bs.div(t0)] : 0;
    };
    int grp_cur = load_group(0);
    int grp_nxt = I.n_prefix > g_tpg ? load_group(1) : 0;
    int key = I.t_begin * KV_TILE + koff;
    int row = args.fd_bs.mod(key);
    int jt = 0;
    for (int j = 0; ok && j < I.n_prefix; ++j) {
      if (j + I.n_tree == stop || !take()) {
        ok = false;
        break;
      }
      if (jt == 0 && j > 0) {
        grp_cur = grp_nxt;
        const int g2 = (j >> (5 - lg_boxes)) + 1;
        grp_nxt = g2 * g_tpg < I.n_prefix ? load_group(g2) : 0;
      }
      int blk = __shfl_sync(0xffffffffu, grp_cur, (jt << lg_boxes) + lane);
      const bool issue = lane < g_boxes && key < I.P;
      if (issue && (blk < 0 || blk >= a.num_blocks)) {
        if (a.status) a.status[I.b] = TS_ERR_BAD_BLOCK;
        blk = 0;
      }
      const unsigned mask = __ballot_sync(0xffffffffu, issue);
      if (lane == 0) mbar_arrive_expect_tx(&full[slot], __popc(mask) * box_bytes);
      __syncwarp();
      if (issue) tma_load_3d((is_v ? sm.v[slot] : sm.k[slot]) + lane * box_bytes, tm_pool, &full[slot], 0, row, blk * a.Hkv + I.g);
      if (is_v) {
        // scale bytes of tokens 4 lane .. 4 lane + 3 (of one block: blocks are multiples of 16)
        const int box = 4 * lane / g_box;
        const int blk_s = __shfl_sync(0xffffffffu, blk, box), row_s = __shfl_sync(0xffffffffu, row, box) + 4 * lane - box * g_box;
        if (key - koff + 4 * lane < I.P)
          cp_async8(&sm.v_scale[slot][4 * lane], args.kv_scale + 2 * (((size_t)blk_s * a.Hkv + I.g) * a.bs + row_s));
        cp_async_arrive(&full[slot]);
      }
      __syncwarp();
      key += KV_TILE;
      row += row_step;
      if (row >= a.bs) row -= a.bs;
      jt = (jt + 1) & (g_tpg - 1);
      next();
    }
  }
}

cudaError_t attn_q8_few_prepare();
cudaError_t launch_attn_q8_few(const Q8Args& t, bool cut, const CUtensorMap& kc, const CUtensorMap& vc,
                               const CUtensorMap& kt, const CUtensorMap& vt, cudaStream_t s);

}  // namespace ts
