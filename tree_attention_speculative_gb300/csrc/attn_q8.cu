// Tree attention over the 8-bit paged cache, on tcgen05 with TMEM and TMA.
//
// The mathematics is that of attn_tc.cu: the G query heads of a sequence's N
// nodes are packed as the rows of one (sequence, KV head) unit, 128 rows a
// tile, and one online softmax runs over the tree's own keys (gated by the
// ancestry bits) and the prefix in 128-token tiles.  What differs is that a
// prefix row is D e4m3 codes and a power of two.
//
// Keys stay 8-bit.  q . k is taken on e4m3 tensor operands with q split in
// two: with the row of q scaled by a power of two to within 448, hi = e4m3(q)
// and lo = e4m3(q - hi) hold all 8 bits of a bf16 significand: exactly down to
// 2^-2, 2^-9.8 of the row's largest, which is past 224, and below that to half of
// lo's last step of 2^-9, 2^-17.8 of it.
// S = hi . k + lo . k then costs as many MMA cycles as bf16 (e4m3 runs at twice
// its rate) and the keys need no conversion; the key's power of two and the
// row's multiply the logits in fp32.
// Values are widened to bf16, which holds code * 2^e exactly (a 4-bit
// significand), so P V is the bf16 product of the bf16 kernel.  (e4m3 weights
// for an 8-bit P V would need two terms as well, and lose every weight below
// 2^-18 of the row's largest.)
//
// What bounds it.  Bytes: 2 D + 2 a token and KV head, half of bf16: a 128-token
// tile is 32.5 KB, 0.73 us of one SM's share of HBM.  Its products take 1024 MMA
// cycles (0.5 us).  It takes 1.25 us, and no unit is full: 59-64 % of the issue
// slots, the tensor pipe 37-43 %, shared memory 37-43 %, DRAM 42 % (15 % where the
// products are the most).  What a tile waits for is its chain of stages, S,
// softmax, widening, P V, each of one or two warps a partition that mostly wait
// for their own last instruction or load.  So the loops are kept short (a larger
// kernel fetches its instructions more slowly than it runs them), no maximum is
// taken in the common case, and the scale bytes arrive by asynchronous copies.
// 16 prefixes of 1-16K tokens, 26 nodes: 91 us (3.2 TB/s); 64 x 8K tokens with 512
// rows a unit: 1.09 ms (1.01 PFLOP/s); 4 x 128K with 768 rows: 1.58 ms; heads of
// 64: 81 us, 0.96 ms and (one node of 32 heads, 32 prefixes of 0-8K) 78 us.  Units
// of up to 8 rows of heads of 128 go to attn_q8_few.cu.
//
// Work split.  A chain is one row tile of one unit: its tree tiles, then its
// prefix tiles.  The host lays all chains end to end, row tile by row tile, and
// cuts them into one run of equal weight a CTA (one CTA an SM), so every SM
// finishes at the same time whatever the lengths.  CTAs of the same units and
// different row tiles run in step and share the K/V tiles in L2.  A CTA does
// whole chains and at most two parts of chains; a part leaves its normalised
// rows and their log-sum-exp in fp32, and k_merge_q8 joins the parts of each cut
// chain.  The lists are static: every role walks its CTA's run by itself.  A
// chain's lengths are the device's, so a captured launch stays right when
// prefixes have grown since the plan.  A segment (a chain, or a part of one)
// costs 6 us beyond its tiles: its tree tile, the splitting of its queries, the
// epilogue.
//
//   warp 0       TMEM allocation; TMA loads of the K codes (and bf16 tree keys)
//   warp 1       QK issuer: loads each segment's Q tile; S(j) = Q K(j)^T
//   warp 2       PV issuer: O += P(j) V(j)
//   warp 3       TMA loads of the V codes; asynchronous copies of the tokens'
//                scale bytes beside them
//   warps 4-7    conversion: thread t owns token t of a tile and row t of Q.
//                Splits the Q tile into hi and lo (in place), hands the keys'
//                powers of two to the softmax a tile ahead, widens V with the
//                values' (rows past the prefix become zeros).  The tree's V is
//                loaded straight into the widened buffer.
//   warps 8-15   softmax, two groups: thread r of a group owns row r (TMEM lane
//                r), the groups the lower and upper 64 keys of every tile, each
//                with its own O, reference and sum, joined at a segment's end.
//                Two warps a partition hide each other's latency, and need no
//                exchange within a tile.
//
// Every wait is bounded; one that runs out aborts the CTA, which lets what it
// has in flight land and reports TS_ERR_TIMEOUT for the sequences of the
// segments it did not finish.
#include "attn_q8.cuh"
#include "fastexp.cuh"

#include <algorithm>
#include <type_traits>

namespace ts {
namespace {

constexpr int THREADS = Q8_THREADS;
constexpr int CONVERT_THREADS = 128;
constexpr int SOFTMAX_THREADS = 256;
constexpr int SOFTMAX_WARP0 = 8;
// TMEM: an O for each half of a tile's keys, then the S buffers
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t TMEM_O = 0;
constexpr uint32_t O_STRIDE = 128;
constexpr uint32_t TMEM_S0 = 256;
constexpr int NSB = 2;        // S buffers
constexpr int HALF_KEYS = 64;  // keys of a tile a softmax group takes
constexpr int NT = 4;   // tiles' key scales in flight
// The weights are rounded to bf16 for the product (half a step, 2^-8 of each at
// most; as in attn_tc.cu) and summed before that, in fp32, for the log-sum-exp.
// Outputs are divided by the sum of the rounded ones, so that the error of a
// weight that outweighs the others cancels: with hot keys the outputs are then as
// exact as their own rounding lets them be.  What rounding adds to the sum is
// taken for the chunks of 32 keys that weigh more than all before them (64
// sequences of 8K tokens: 1086 us; for every chunk 1218).
// A row keeps the reference m it took from its first keys until the weights of
// 32 keys sum past RESCALE_SUM.  bf16 P, fp32 sums and O have the same precision
// at every magnitude, so weights up to 2^40 are as good as weights up to 1, and
// O is hardly ever rescaled, hot keys or not.  (Sums then stay finite for
// values up to 2^127 / (2^40 x keys), past 2^69.)
constexpr float RESCALE_SUM = 1099511627776.f;  // 2^40

template <int D>
struct Cfg {
  static constexpr int HALVES = D / 64;
  static constexpr int WIDE_BYTES = KV_TILE * D * 2;  // a bf16 tile, and the Q tile
  static constexpr int HALF_BYTES = KV_TILE * 128;
  // As many tiles in flight as shared memory holds; a V tile also has a widened buffer to wait in.
  static constexpr int NSK = D == 128 ? 3 : 5;
  static constexpr int NSV = D == 128 ? 4 : 5;
};

template <int D>
struct __align__(1024) Smem {
  using C = Cfg<D>;
  static constexpr int NSK = C::NSK, NSV = C::NSV;
  uint8_t q[C::WIDE_BYTES];  // bf16 [half][row][128 B]; then hi and lo of a piece's 64 channels, 64 bytes each, in its place
  uint8_t k[C::NSK][SLOT];
  uint8_t v[C::NSV][SLOT];
  uint16_t v_scale[C::NSV][KV_TILE];  // with each V tile its tokens' scale bytes: K row's, V row's
  uint8_t pad[1024 - (C::NSV * KV_TILE * 2) % 1024];
  uint8_t vb[NVB][C::WIDE_BYTES];  // bf16 [half][token][128 B]
  // Scales of tile j (entry j % NT): the token's power of two for its key, and
  // the row's factor (the query's power of two times scale * log2 e).
  float key_scale[NT][KV_TILE];
  float row_scale[NT][ROW_TILE];
  float half_norm[2][ROW_TILE];  // the sum of the rounded weights
  float2 half_ml[2][ROW_TILE];  // (maximum, sum) of each half, at the end of a segment
  // q_free: no product reads the bf16 Q any more, it may be split in place
  uint64_t q_full, q_free, q8_full, q_empty;
  uint64_t k_full[C::NSK], k_empty[C::NSK];
  uint64_t v_full[C::NSV], v_empty[C::NSV];
  uint64_t vb_full[NVB], vb_empty[NVB], vt_full[NVB];
  uint64_t t_full[NT], t_empty[NT];
  uint64_t s_full[NSB], p_full[NSB], s_free[NSB];
  uint64_t o_ready;
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort_flag;
  int pv_done;    // PVs completed, published by the PV issuer
  int segs_done;  // segments stored
};

__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(reinterpret_cast<uint64_t>(p)),
               "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Scales what a row has so far by f: `chunks` of P (16 columns each), and O,
// which must then hold every earlier PV.  Out of line: it is hardly ever run.
template <int D>
__device__ __noinline__ void rescale_tmem(uint32_t p_tmem, int chunks, uint32_t o_tmem, bool with_o, float f) {
  tmem_st_wait();
  tc_fence_after();
#pragma unroll 1
  for (int i = 0; i < chunks; ++i) {
    uint32_t w[16];
    tmem_ld16(p_tmem + i * 16, w);
    tmem_ld_wait();
    reg_fence16(w);
#pragma unroll
    for (int e = 0; e < 16; ++e)
      w[e] = pack_bf16x2(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xffff0000u) * f);
    tmem_st16(p_tmem + i * 16, w);
  }
#pragma unroll 1
  for (int d = 0; with_o && d < D; d += 32) {
    uint32_t w[32];
    tmem_ld32(o_tmem + d, w);
    tmem_ld_wait();
    reg_fence32(w);
#pragma unroll
    for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * f);
    tmem_st32(o_tmem + d, w);
  }
}

// The sum of 32 weights as rounded to bf16.  Out of line: seldom run.
__device__ __noinline__ float rounded_sum(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f, uint32_t g,
                                          uint32_t h, uint32_t i, uint32_t j, uint32_t k, uint32_t l, uint32_t m, uint32_t n,
                                          uint32_t o, uint32_t p) {
  const uint32_t w[16] = {a, b, c, d, e, f, g, h, i, j, k, l, m, n, o, p};
  float s0 = 0.f, s1 = 0.f;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    s0 += __uint_as_float(w[q] << 16);
    s1 += __uint_as_float(w[q] & 0xffff0000u);
  }
  return s0 + s1;
}

// Columns [c, c + 32) of a row, the two halves' O joined (zeros for a row that
// saw nothing, whatever its O holds).
__device__ __forceinline__ void join_o(uint32_t o_tmem, int c, float f0, float f1, uint32_t (&u)[32]) {
  uint32_t v[32];
  tmem_ld32(o_tmem + c, u);
  tmem_ld32(o_tmem + O_STRIDE + c, v);
  tmem_ld_wait();
  reg_fence32(u);
  reg_fence32(v);
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    const float p = f0 == 0.f ? 0.f : __uint_as_float(u[e]) * f0;
    u[e] = __float_as_uint(f1 == 0.f ? p : fmaf(__uint_as_float(v[e]), f1, p));
  }
}
// D/2 channels of a row, fp32 to a part or bf16 to the output.  A loop each: one
// for both made the loop over the tiles slower (heads of 64, 64 sequences of 8K
// tokens: 962 us, out of line 1173; 16 prefixes of 1-16K, heads of 128: 91, in
// line 100).
template <int D>
__device__ __forceinline__ void store_part(uint32_t o_tmem, float f0, float f1, float* part, bool active) {
#pragma unroll 1
  for (int c = 0; c < D / 2; c += 32) {
    uint32_t u[32];
    __syncwarp();  // (TMEM loads want the warp together)
    join_o(o_tmem, c, f0, f1, u);
    if (!active) continue;
#pragma unroll
    for (int q = 0; q < 4; ++q) st_global_v8(part + c + 8 * q, u + 8 * q);
  }
}
template <int D>
__device__ __forceinline__ void store_out(uint32_t o_tmem, float f0, float f1, __nv_bfloat16* out, int out32, bool active) {
#pragma unroll 1
  for (int c = 0; c < D / 2; c += 32) {
    uint32_t u[32], w[16];
    __syncwarp();  // (TMEM loads want the warp together)
    join_o(o_tmem, c, f0, f1, u);
    if (!active) continue;
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1]));
    if (out32) {
      st_global_v8(out + c, w);
      st_global_v8(out + c + 16, w + 8);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) reinterpret_cast<uint4*>(out + c)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
k_attn_q8(const __grid_constant__ Q8Args args, const __grid_constant__ CUtensorMap tm_q,
          const __grid_constant__ CUtensorMap tm_kc, const __grid_constant__ CUtensorMap tm_vc,
          const __grid_constant__ CUtensorMap tm_kt, const __grid_constant__ CUtensorMap tm_vt) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  // (an offset from the array, not a rounded address, so that accesses stay shared-memory ones)
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023));
  const AttnArgs& a = args.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Ctl ctl{&sm.abort_flag, a.wait_limit_ns};
  const int cta = blockIdx.x;
  const int chain0 = args.runs.chain[cta];
  // the run's last chain: where the next CTA starts, unless that is the chain's first tile
  const int chain1 = args.runs.chain[cta + 1] - (args.runs.tile[cta + 1] == 0 ? 1 : 0);

  if (threadIdx.x == 0) {
    sm.abort_flag = 0;
    sm.pv_done = 0;
    sm.segs_done = 0;
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_free, 1);
    mbar_init(&sm.q8_full, CONVERT_THREADS);
    mbar_init(&sm.q_empty, 1);
    for (int i = 0; i < C::NSK; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < C::NSV; ++i) {
      mbar_init(&sm.v_full[i], 1 + 32);  // the tile, and each lane's scale bytes
      mbar_init(&sm.v_empty[i], CONVERT_THREADS);
    }
    for (int i = 0; i < NVB; ++i) {
      mbar_init(&sm.vb_full[i], CONVERT_THREADS);
      mbar_init(&sm.vb_empty[i], 1);
      mbar_init(&sm.vt_full[i], 1);
    }
    for (int i = 0; i < NT; ++i) {
      mbar_init(&sm.t_full[i], CONVERT_THREADS);
      mbar_init(&sm.t_empty[i], SOFTMAX_THREADS / 32);
    }
    for (int i = 0; i < NSB; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], SOFTMAX_THREADS);
      mbar_init(&sm.s_free[i], 1);
    }
    mbar_init(&sm.o_ready, 1);
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    fence_barrier_init();
  }
  if (warp == V_WARP && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_kc);
    tma_prefetch_desc(&tm_vc);
    tma_prefetch_desc(&tm_kt);
    tma_prefetch_desc(&tm_vt);
    if (chain0 <= chain1) {
      // the first Q tile, prefix length and table entry, into L2 (prefetches read no data; see sm100.cuh)
      const Seg I = make_seg(chain0, cta, 0, args);
      for (int h = 0; h < C::HALVES; ++h) tma_prefetch_4d(&tm_q, 64 * h, I.g * a.G, I.rt * args.nodes_per_tile, I.b);
      prefetch_l2(a.prefix_len + I.b);
      const int i = args.fd_bs.div(args.runs.tile[cta] * KV_TILE);
      prefetch_l2(a.block_table + (size_t)I.b * a.max_blocks + (i < a.max_blocks ? i : a.max_blocks - 1));
    }
  }
  if (warp == K_WARP) tmem_alloc(&sm.tmem_base, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  pdl_wait();

  // what a role has started and not seen land, for the teardown of an aborted CTA
  int issued = 0;                  // K or V ring slots this warp filled
  int q_issued = 0, q_landed = 0;  // Q tiles
  int vt_issued[NVB] = {0, 0};     // tree V tiles, by buffer

  if (warp == K_WARP || warp == V_WARP) {
    load_codes<D>(sm, args, warp == V_WARP, warp == V_WARP ? &tm_vc : &tm_kc, &tm_kt, cta, chain0, chain1, ctl, issued);
  } else if (warp == QK_WARP) {
    if (lane == 0) {
      // ------------------------------------------------------------ QK issuer
      constexpr uint32_t ID_BF16 = idesc_bf16_f32(ROW_TILE, KV_TILE, 0, 0);
      constexpr uint32_t ID_E4M3 = idesc_e4m3_f32(ROW_TILE, KV_TILE);
      const uint32_t q_addr = smem_u32(sm.q);
      int jg = 0;         // tiles
      int kq = 0;         // K ring slots
      int q8 = 0;         // Q tiles split
      bool ok = true;
      int p_next = chain0 <= chain1 ? a.prefix_len[seq_of(chain0, args)] : 0;
      for (int chain = chain0; ok && chain <= chain1; ++chain) {
        const Seg I = make_seg(chain, cta, p_next, args);
        if (chain < chain1) p_next = a.prefix_len[seq_of(chain + 1, args)];
        if (I.n_tiles == 0) continue;
        if (q_issued > 0 && !(ok = wait_bar(&sm.q_empty, (q_issued - 1) & 1, ctl))) break;
        mbar_arrive_expect_tx(&sm.q_full, C::WIDE_BYTES);
        for (int h = 0; h < C::HALVES; ++h)
          tma_load_4d(sm.q + h * (ROW_TILE * 128), &tm_q, &sm.q_full, 64 * h, I.g * a.G, I.rt * args.nodes_per_tile, I.b);
        ++q_issued;
        if (chain < chain1) {  // the next segment's Q tile, into L2
          const Seg nx = make_seg(chain + 1, cta, 0, args);
          for (int h = 0; h < C::HALVES; ++h) tma_prefetch_4d(&tm_q, 64 * h, nx.g * a.G, nx.rt * args.nodes_per_tile, nx.b);
        }
        if (!(ok = wait_bar(&sm.q_full, (q_issued - 1) & 1, ctl))) break;
        ++q_landed;
        if (I.n_tree == 0) mbar_arrive(&sm.q_free);  // no tree: at once
        for (int j = 0; j < I.n_tiles; ++j, ++jg) {
          const bool tree = j < I.n_tree;
          if (j == I.n_tree) {
            if (!(ok = wait_bar(&sm.q8_full, q8 & 1, ctl))) break;
            ++q8;
          }
          const int s0 = kq % C::NSK, s1 = (kq + 1) % C::NSK;
          ok = wait_bar(&sm.k_full[s0], (kq / C::NSK) & 1, ctl);
          if (ok && tree && C::HALVES == 2) ok = wait_bar(&sm.k_full[s1], ((kq + 1) / C::NSK) & 1, ctl);
          if (ok && jg >= NSB) ok = wait_bar(&sm.s_free[jg % NSB], ((jg / NSB) - 1) & 1, ctl);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d_tmem = tmem + TMEM_S0 + (jg % NSB) * 128;
          const uint32_t k0 = smem_u32(sm.k[s0]);
          if (tree) {
            const uint32_t k1 = smem_u32(sm.k[s1]);
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
              mma_ss(d_tmem, smem_desc_sw128(q_addr + (i >> 2) * (ROW_TILE * 128) + (i & 3) * 32, 16, 1024),
                     smem_desc_sw128((i >> 2 ? k1 : k0) + (i & 3) * 32, 16, 1024), ID_BF16, i > 0);
            mma_commit(&sm.s_full[jg % NSB]);
            for (int h = 0; h < C::HALVES; ++h) mma_commit(&sm.k_empty[h ? s1 : s0]);
            kq += C::HALVES;
            if (j == I.n_tree - 1 && I.n_prefix > 0) mma_commit(&sm.q_free);
          } else {
            const uint64_t q_desc = smem_desc_sw128(q_addr, 16, 1024);
            const uint64_t k_desc = D == 128 ? smem_desc_sw128(k0, 16, 1024) : smem_desc_sw64(k0, 16, 512);
            // 32 channels a step: those of piece h, hi and then lo
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const int h = i >> 2, low = (i >> 1) & 1, step = i & 1;
              const uint64_t qd = q_desc + ((h * (ROW_TILE * 128) + low * 64 + step * 32) >> 4);
              const uint64_t kd = k_desc + (((D == 128 ? h * 64 : 0) + step * 32) >> 4);
              mma_ss_f8(d_tmem, qd, kd, ID_E4M3, i > 0);
            }
            mma_commit(&sm.s_full[jg % NSB]);
            mma_commit(&sm.k_empty[s0]);
            kq += 1;
          }
        }
        if (ok) mma_commit(&sm.q_empty);
      }
    }
  } else if (warp == PV_WARP) {
    if (lane == 0) {
      // ------------------------------------------------------------ PV issuer
      constexpr uint32_t ID_PV = idesc_bf16_f32(ROW_TILE, D, 0, 1);
      int jg = 0;
      bool ok = true;
      int p_next = chain0 <= chain1 ? a.prefix_len[seq_of(chain0, args)] : 0;
      for (int chain = chain0; ok && chain <= chain1; ++chain) {
        const Seg I = make_seg(chain, cta, p_next, args);
        if (chain < chain1) p_next = a.prefix_len[seq_of(chain + 1, args)];
        for (int j = 0; j < I.n_tiles; ++j, ++jg) {
          const int buf = jg % NVB;
          ok = wait_bar(&sm.p_full[jg % NSB], (jg / NSB) & 1, ctl) && wait_bar(&sm.vb_full[buf], (jg / NVB) & 1, ctl);
          if (!ok) break;
          tc_fence_after();
          const uint64_t v_desc = smem_desc_sw128(smem_u32(sm.vb[buf]), C::HALF_BYTES, 1024);
          const uint32_t p_tmem = tmem + TMEM_S0 + (jg % NSB) * 128;
#pragma unroll
          for (int i = 0; i < KV_TILE / 16; ++i)
            mma_ts(tmem + TMEM_O + (i >> 2) * O_STRIDE, p_tmem + (i >> 2) * HALF_KEYS + (i & 3) * 8,
                   v_desc + ((i * 2048) >> 4), ID_PV, j > 0 || (i & 3) > 0);
          mma_commit(&sm.o_ready);
          mma_commit(&sm.s_free[jg % NSB]);
          mma_commit(&sm.vb_empty[buf]);
          if (!(ok = wait_bar(&sm.o_ready, jg & 1, ctl))) break;
          tc_fence_after();
          publish(&sm.pv_done, jg + 1);
        }
      }
    }
  } else if (warp < SOFTMAX_WARP0) {
    // ------------------------------------------------------------ conversion
    const int ct = threadIdx.x - CONVERT_WARP0 * 32;  // token of a tile, row of Q
    const int swz = ct & 7;
    int jg = 0, vq = 0, qn = 0, q8 = 0;
    int vt_seen[NVB] = {0, 0};
    bool ok = true;
    int p_next = chain0 <= chain1 ? a.prefix_len[seq_of(chain0, args)] : 0;
    for (int chain = chain0; ok && chain <= chain1; ++chain) {
      const Seg I = make_seg(chain, cta, p_next, args);
      if (chain < chain1) p_next = a.prefix_len[seq_of(chain + 1, args)];  // on its way while this one runs
      if (I.n_tiles == 0) continue;
      float row_scale = 0.f;
      // The Q tile, row ct: scaled to within 448, hi and lo in place.  (q_free
      // comes once a segment with prefix tiles, in step with q8_full; q_full also
      // for the others, but none can follow before q8_full.)
      auto split_q = [&]() -> bool {
        if (!(wait_bar(&sm.q_free, q8 & 1, ctl) && wait_bar(&sm.q_full, qn & 1, ctl))) return false;
        uint32_t m = 0;
#pragma unroll 1
        for (int c = 0; c < D / 8; ++c) {
          const uint4 y = *reinterpret_cast<const uint4*>(sm.q + (c >> 3) * (ROW_TILE * 128) + ct * 128 + (((c & 7) ^ swz) << 4));
          m = q8_max2(m, q8_max2(q8_max2(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu), q8_max2(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu)));
        }
        m = q8_max2(m, m >> 16) & 0xffffu;
        const int s = q8_scale_byte(m);
        const float inv = pow2_of(254 - s);
        // an infinite query has no finite logits
        row_scale = m == 0x7f80u ? __uint_as_float(0x7fffffffu) : fmaxf(pow2_of(s) * a.scale_log2, LEAST);
#pragma unroll 1
        for (int h = 0; h < C::HALVES; ++h) {
          uint8_t* piece = sm.q + h * (ROW_TILE * 128) + ct * 128;
          uint4 x[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) x[c] = *reinterpret_cast<const uint4*>(piece + ((c ^ swz) << 4));
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 16 channels: a 16-byte chunk of hi and one of lo
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint4& y = x[2 * c + (e >> 1)];
              split4((e & 1) ? y.z : y.x, (e & 1) ? y.w : y.y, inv, hi[e], lo[e]);
            }
            *reinterpret_cast<uint4*>(piece + ((c ^ swz) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(piece + (((c + 4) ^ swz) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
        fence_proxy_async();
        mbar_arrive(&sm.q8_full);
        ++q8;
        return true;
      };
      for (int j = -1; j < I.n_tiles; ++j) {
        const bool tree = j >= 0 && j < I.n_tree;
        const int buf = jg % NVB;
        uint8_t* wide = sm.vb[buf];
        if (j >= 0 && jg >= NVB && !(ok = wait_bar(&sm.vb_empty[buf], ((jg / NVB) - 1) & 1, ctl))) break;
        if (tree) {
          if (ct == 0) {
            mbar_arrive_expect_tx(&sm.vt_full[buf], C::WIDE_BYTES);
            for (int h = 0; h < C::HALVES; ++h)
              tma_load_4d(wide + h * C::HALF_BYTES, &tm_vt, &sm.vt_full[buf], 64 * h, I.g, j * KV_TILE, I.b);
            if (buf) ++vt_issued[1];
            else ++vt_issued[0];
          }
        }
        // The scales of tile j + 1 (the tree's: 1) go to the softmax, ahead of the values of tile j.
        if (j + 1 < I.n_tiles) {
          const int jt = j < 0 ? jg : jg + 1, p = j + 1 - I.n_tree, vt = vq + (j >= I.n_tree ? 1 : 0);
          float key = 1.f, rs = a.scale_log2;
          if (p == 0 && !(ok = split_q())) break;
          if (p >= 0) {
            if (!(ok = wait_bar(&sm.v_full[vt % C::NSV], (vt / C::NSV) & 1, ctl))) break;
            key = (I.t_begin + p) * KV_TILE + ct < I.P ? pow2_of(sm.v_scale[vt % C::NSV][ct] & 0xff) : 0.f;
            rs = row_scale;
          }
          if (jt >= NT && !(ok = wait_bar(&sm.t_empty[jt % NT], ((jt / NT) - 1) & 1, ctl))) break;
          sm.key_scale[jt % NT][ct] = key;
          sm.row_scale[jt % NT][ct] = rs;
          mbar_arrive(&sm.t_full[jt % NT]);
        }
        if (j >= 0 && !tree) {
          const bool inside = (I.t_begin + j - I.n_tree) * KV_TILE + ct < I.P;
          const int slot = vq % C::NSV;
          const uint8_t* src = sm.v[slot] + ct * D;
          const uint32_t sc = sm.v_scale[slot][ct];
          // sc: the K row's byte, then the V row's; rows past the prefix become zeros.
          // One 16-code chunk an iteration, the next one on its way; rolled, so that
          // it stays in the instruction cache beside the softmax.
          const WideScale ws(inside ? sc >> 8 : 0u, inside);
          auto chunk = [&](int c) {  // chunk c of this row, where the 128-byte (D = 128) or 64-byte swizzle put it
            return *reinterpret_cast<const uint4*>(src + ((D == 128 ? c ^ swz : c ^ ((ct >> 1) & 3)) << 4));
          };
          uint8_t* row = wide + ct * 128;
          uint4 x = chunk(0);
#pragma unroll 2
          for (int c = 0; c < D / 16; ++c) {
            const uint4 x_next = chunk((c + 1) & (D / 16 - 1));
            uint4 lo, hi;
            widen16(x, ws.m1, lo, hi);
            uint8_t* to = row + (c >> 2) * C::HALF_BYTES;
            *reinterpret_cast<uint4*>(to + (((2 * (c & 3)) ^ swz) << 4)) = lo;
            *reinterpret_cast<uint4*>(to + (((2 * (c & 3) + 1) ^ swz) << 4)) = hi;
            x = x_next;
          }
          if (inside && ws.m2 != 0x3f803f80u) {  // (a row beyond 2^15: the rest of its power of two)
#pragma unroll 1
            for (int e = 0; e < D / 2; ++e) {
              uint32_t* w = reinterpret_cast<uint32_t*>(row + (e >> 5) * C::HALF_BYTES + (((e & 31) >> 2) << 4)) + (e & 3);
              *w = mul_bf16x2(*w, ws.m2);
            }
          }
          mbar_arrive(&sm.v_empty[slot]);
          ++vq;
          fence_proxy_async();
          mbar_arrive(&sm.vb_full[buf]);
        }
        if (tree) {
          if (!(ok = wait_bar(&sm.vt_full[buf], (buf ? vt_seen[1] : vt_seen[0]) & 1, ctl))) break;
          if (buf) ++vt_seen[1];
          else ++vt_seen[0];
          const int node = j * KV_TILE + ct;
          if (node < a.N) clear_unseen<D>(wide + ct * 128, a.anc_mask + (size_t)I.b * a.N * a.W + (node >> 6), node & 63, a.N, a.W);
          mbar_arrive(&sm.vb_full[buf]);
        }
        if (j >= 0) ++jg;
      }
      ++qn;
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int half = (warp - SOFTMAX_WARP0) >> 2;  // keys [64 half, 64 half + 64) of every tile
    const int r = (warp & 3) * 32 + lane;
    const int R = a.N * a.G;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_tmem = tmem + lane_base + TMEM_O + half * O_STRIDE;
    int jg = 0;
    bool ok = true;
    int p_next = chain0 <= chain1 ? a.prefix_len[seq_of(chain0, args)] : 0;
    for (int chain = chain0; ok && chain <= chain1; ++chain) {
      const Seg I = make_seg(chain, cta, p_next, args);
      if (chain < chain1) p_next = a.prefix_len[seq_of(chain + 1, args)];  // on its way while this one runs
      if (!I.p_ok && r == 0 && a.status) a.status[I.b] = TS_ERR_SHAPE;
      const int grow = I.rt * ROW_TILE + r;
      const bool active = grow < R;
      const int node = active ? args.fd_g.div(grow) : 0;
      const int h = I.g * a.G + (active ? grow - node * a.G : 0);
      // a warp none of whose rows exist only keeps the barriers going
      const bool busy = I.rt * ROW_TILE + (r & ~31) < R;
      const int slot = 2 * cta + (chain != chain0 ? 1 : 0);
      uint64_t anc[2] = {0ull, 0ull};  // this half's word of each tree tile
      if (active && I.n_tree > 0) {
        const uint64_t* arow = a.anc_mask + ((size_t)I.b * a.N + node) * a.W;
#pragma unroll
        for (int w = 0; w < 2; ++w)
          if (2 * w + half < a.W) anc[w] = arow[2 * w + half];
      }
      // reference, sum, and what rounding adds to the sum (rows of the padding,
      // which see nothing, need no reference)
      float m_run = active ? NEG_INF : 0.f, l_run = 0.f, excess = 0.f;
      for (int j = 0; j < I.n_tiles; ++j, ++jg) {
        const int tb = jg % NT;
        if (!__all_sync(0xffffffffu, wait_bar(&sm.t_full[tb], (jg / NT) & 1, ctl) &&
                                         wait_bar(&sm.s_full[jg % NSB], (jg / NSB) & 1, ctl))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t s_tmem = tmem + lane_base + TMEM_S0 + (jg % NSB) * 128 + half * HALF_KEYS;
        const bool tree = j < I.n_tree;
        // which of this half's keys the row sees; a whole prefix tile needs no mask
        const int valid = I.P - (I.t_begin + j - I.n_tree) * KV_TILE - half * HALF_KEYS;
        const uint64_t see = tree ? (j == 0 ? anc[0] : anc[1]) : valid <= 0 ? 0ull : (1ull << (valid & 63)) - 1ull;
        const float row_scale = sm.row_scale[tb][r];
        const uint64_t scale2 = fx::pack2(row_scale, row_scale);
        // 32 columns at a time, in a loop that stays rolled: unrolled over the
        // tile, softmax and conversion together overflowed the instruction
        // caches (3 of 8 stall cycles an issue, 2.5 us a tile).
        auto columns = [&](auto masked) -> bool {
#pragma unroll 1
          for (int c = 0; c < HALF_KEYS / 32; ++c) {
            uint32_t u[32];
            tmem_ld32(s_tmem + c * 32, u);
            float4 ks[8];  // on their way with S
#pragma unroll
            for (int e = 0; e < 8; ++e)
              ks[e] = reinterpret_cast<const float4*>(sm.key_scale[tb] + half * HALF_KEYS + c * 32)[e];
            tmem_ld_wait();
            reg_fence32(u);
            uint64_t y[16];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              y[2 * e] = fx::mul2(fx::pack2(__uint_as_float(u[4 * e]), __uint_as_float(u[4 * e + 1])), fx::pack2(ks[e].x, ks[e].y));
              y[2 * e + 1] = fx::mul2(fx::pack2(__uint_as_float(u[4 * e + 2]), __uint_as_float(u[4 * e + 3])), fx::pack2(ks[e].z, ks[e].w));
            }
            if constexpr (decltype(masked)::value) {
              const uint32_t bits = (uint32_t)(see >> (32 * c));
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float x0, x1;
                fx::unpack2(y[e], x0, x1);
                y[e] = fx::pack2((bits >> (2 * e)) & 1u ? x0 : NEG_INF, (bits >> (2 * e + 1)) & 1u ? x1 : NEG_INF);
              }
            }
            // p = 2^(y * row_scale - m) as bf16, and their sum.  No maximum is
            // taken: a sum past 2^RESCALE says that m is too low, and a row
            // without an m has no key yet; then m is set and the chunk repeated.
            uint32_t pk[16];
            float sum;
#pragma unroll 1
            while (true) {
              const float m_exp = m_run == NEG_INF ? 0.f : m_run;  // (no key so far: every p is 0)
              const uint64_t negm2 = fx::pack2(-m_exp, -m_exp);
              uint64_t sum2[2] = {0ull, 0ull};
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float x0, x1;
                fx::unpack2(fx::fma2(y[e], scale2, negm2), x0, x1);
                const float p0 = ex2(x0), p1 = ex2(x1);
                sum2[e & 1] = fx::add2(sum2[e & 1], fx::pack2(p0, p1));
                pk[e] = pack_bf16x2(p0, p1);
              }
              float r0, r1;
              fx::unpack2(fx::add2(sum2[0], sum2[1]), r0, r1);
              sum = r0 + r1;
              const bool high = sum > RESCALE_SUM || m_run == NEG_INF;
              if (!__any_sync(0xffffffffu, high)) break;
              float mx = NEG_INF;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float x0, x1;
                fx::unpack2(y[e], x0, x1);
                mx = fmaxf(mx, fmaxf(x0, x1));
              }
              mx *= row_scale;
              const bool move = high && mx > m_run;  // (the sum was high, or these are the row's first keys)
              if (!__any_sync(0xffffffffu, move)) break;
              // What the row has so far is scaled down (the warp together; the others by 1).
              const float f = !move ? 1.f : (m_run == NEG_INF ? 0.f : ex2(m_run - mx));
              if (move) m_run = mx;
              l_run *= f;
              excess *= f;
              if (j > 0 && !__all_sync(0xffffffffu, wait_count(&sm.pv_done, jg, ctl))) return false;
              rescale_tmem<D>(s_tmem, c, o_tmem, j > 0, f);
            }
            if (__any_sync(0xffffffffu, sum > l_run)) {  // (the warp goes together; a row adds its own chunks' only)
              const float more = rounded_sum(pk[0], pk[1], pk[2], pk[3], pk[4], pk[5], pk[6], pk[7], pk[8], pk[9], pk[10],
                                             pk[11], pk[12], pk[13], pk[14], pk[15]) - sum;
              excess += sum > l_run ? more : 0.f;
            }
            l_run += sum;
            tmem_st16(s_tmem + c * 16, pk);
          }
          return true;
        };
        if (busy) ok = tree || valid < HALF_KEYS ? columns(std::true_type{}) : columns(std::false_type{});
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.t_empty[tb]);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sm.p_full[jg % NSB]);
      }
      // End of the segment: the two halves' O, each with its maximum and sum,
      // are joined, normalised and stored, D/2 channels by each group.  (A warp
      // whose wait gave up comes here too: its partner may be waiting.)
      sm.half_ml[half][r] = make_float2(m_run, l_run);
      sm.half_norm[half][r] = l_run + excess;
      ok = ok && (I.n_tiles == 0 || wait_count(&sm.pv_done, jg, ctl));
      ok = named_barrier_and(1 + (warp & 3), 64, ok);
      if (!ok) break;
      tc_fence_after();
      const float2 other = sm.half_ml[half ^ 1][r];
      const float m = fmaxf(m_run, other.x);
      const float w_own = m_run == NEG_INF ? 0.f : ex2(m_run - m), w_other = other.x == NEG_INF ? 0.f : ex2(other.x - m);
      const float l = l_run * w_own + other.y * w_other;
      const bool none = l == 0.f;  // the row saw no key
      const float norm = (l_run + excess) * w_own + sm.half_norm[half ^ 1][r] * w_other;
      const float inv = none ? 0.f : 1.f / norm;
      const float lse2 = none ? NEG_INF : m + __log2f(l);
      const size_t orow = ((size_t)I.b * a.N + node) * a.Hq + h;
      const float f0 = half == 0 ? w_own * inv : w_other * inv, f1 = half == 0 ? w_other * inv : w_own * inv;
      if (I.n_tiles == 0) {
        if (active && half == 0) args.part_lse[(size_t)slot * ROW_TILE + r] = NEG_INF;
      } else if (busy) {
        const uint32_t o_row = tmem + lane_base + TMEM_O + half * (D / 2);
        if (I.whole) {
          if (active && half == 0 && a.lse) a.lse[orow] = lse2 * 0.69314718055994531f;
          store_out<D>(o_row, f0, f1, a.out + orow * D + half * (D / 2), args.out32, active);
        } else {
          if (active && half == 0) args.part_lse[(size_t)slot * ROW_TILE + r] = lse2;
          store_part<D>(o_row, f0, f1, args.part_o + ((size_t)slot * ROW_TILE + r) * D + half * (D / 2), active);
        }
      }
      // both halves have read O, and each other's sums, before the next segment's first P
      tc_fence_before();
      named_barrier_and(1 + (warp & 3), 64, true);
      if (half == 0 && r == 0) publish(&sm.segs_done, chain - chain0 + 1);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*ctl.flag) {
    // A wait gave up.  Nothing may still write this CTA's shared memory or TMEM
    // once it exits: wait (bounded) for the newest loads of each ring, for a Q
    // tile, for the tree's V tiles and for every MMA started.
    if (warp == V_WARP) asm volatile("cp.async.wait_all;" ::: "memory");
    if ((warp == K_WARP || warp == V_WARP) && lane == 0) {
      uint64_t* full = warp == V_WARP ? sm.v_full : sm.k_full;
      const int nst = warp == V_WARP ? C::NSV : C::NSK;
      for (int j = max(0, issued - nst); j < issued; ++j) mbar_wait(&full[j % nst], (j / nst) & 1, a.wait_limit_ns);
    } else if ((warp == QK_WARP || warp == PV_WARP) && lane == 0) {
      if (q_issued > q_landed) mbar_wait(&sm.q_full, (q_issued - 1) & 1, a.wait_limit_ns);
      uint64_t* d = &sm.drain[warp - QK_WARP];
      mma_commit(d);
      mbar_wait(d, 0, a.wait_limit_ns);
    } else if (threadIdx.x == CONVERT_WARP0 * 32) {  // (thread 0 of the conversion loads the tree's V)
      for (int i = 0; i < NVB; ++i)
        if (vt_issued[i] > 0) mbar_wait(&sm.vt_full[i], (vt_issued[i] - 1) & 1, a.wait_limit_ns);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && a.status) {
      for (int chain = chain0 + sm.segs_done; chain <= chain1; ++chain) a.status[seq_of(chain, args)] = TS_ERR_TIMEOUT;
    }
  }
  pdl_trigger();
  if (warp == K_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

// Joins the parts of each cut chain: block (c, i) the chain that begins in CTA
// c and ends in a later one, rows 128/gridDim.y of it from i on.  With parts
// O_s, L_s (base 2): out = sum 2^(L_s - M) O_s / sum 2^(L_s - M).
constexpr int MERGE_THREADS = 128;
template <int D>
__global__ void __launch_bounds__(MERGE_THREADS)
k_merge_q8(const __grid_constant__ Q8Args args) {
  constexpr int LANES = D / 8;
  constexpr int ROWS = MERGE_THREADS / LANES;
  const AttnArgs& a = args.a;
  const Runs& runs = args.runs;
  const int c = blockIdx.x;
  const int chain = runs.chain[c + 1];
  if (runs.tile[c + 1] == 0 || (runs.chain[c] == chain && runs.tile[c] > 0)) return;  // nothing cut, or not begun here
  const int rt = args.fd_units.div(chain), u = chain - rt * args.units;
  const int b = args.fd_hkv.div(u), g = u - b * a.Hkv;
  const int r = blockIdx.y * ROWS + (int)threadIdx.x / LANES, sub = (int)threadIdx.x % LANES;
  const int grow = rt * ROW_TILE + r;
  if (grow >= a.N * a.G) return;
  const int first = 2 * c + (runs.chain[c] != chain ? 1 : 0);
  int last = c + 1;
  while (last + 1 < runs.n && runs.chain[last + 1] == chain && runs.tile[last + 1] > 0) ++last;
  pdl_wait();
  pdl_trigger();
  float m = NEG_INF, den = 0.f, acc[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) acc[k] = 0.f;
  for (int p = c; p <= last; ++p) {
    const int slot = p == c ? first : 2 * p;
    const float lse = args.part_lse[(size_t)slot * ROW_TILE + r];
    if (lse == NEG_INF) continue;  // a part without keys: its values were not written
    const float4* o = reinterpret_cast<const float4*>(args.part_o + ((size_t)slot * ROW_TILE + r) * D + sub * 8);
    const float4 lo = o[0], hi = o[1];
    const float m_new = fmaxf(m, lse);
    const float f = m == NEG_INF ? 0.f : exp2f(m - m_new), w = exp2f(lse - m_new);
    den = den * f + w;
    const float x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = fmaf(w, x[k], acc[k] * f);
    m = m_new;
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  const int node = args.fd_g.div(grow);
  const size_t orow = ((size_t)b * a.N + node) * a.Hq + g * a.G + (grow - node * a.G);
  uint32_t o[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = pack_bf16x2(acc[2 * k] * inv, acc[2 * k + 1] * inv);
  reinterpret_cast<uint4*>(a.out + orow * D)[sub] = make_uint4(o[0], o[1], o[2], o[3]);
  if (a.lse && sub == 0) a.lse[orow] = den == 0.f ? NEG_INF : (m + log2f(den)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ plan

// The runs.  A chain weighs its prefix tiles and `head` more: its tree tiles,
// Q tile and epilogue.
// SEG_COST: a segment's start and end in tiles' worth of time (32 sequences of
// 0-8K tokens, one node each: 64 us; with 3, 70 us; 16 of 1-16K, 26 nodes: 91 us;
// with 3, 93 us).
constexpr int SEG_COST = 5;
// No CTA for less weight than this: more of them leave more parts to merge (one
// sequence of 1K tokens, 8 KV heads: 16.7 us; with 3 the same, with 6, 20.3, with
// 12, 23.9; of 4K tokens: 20.8 us; with 3, 22.3, with 6, 22.2, with 12, 27.3).
constexpr int MIN_RUN = 4;
// Where every chain weighs this at most and has an SM, none is cut: the merge
// costs more than it saves (16 sequences of 512 tokens: 15.1 us, cut 18.2).
constexpr int WHOLE = 12;
constexpr int SLIVER = 2;  // no part of fewer tiles: it would cost a segment's start and end

Runs plan_runs(const ts_attn_params* p) {
  Runs r{};
  const int G = p->Hq / p->Hkv;
  const int row_tiles = ceil_div(p->N * G, ROW_TILE);
  const int head = ceil_div(p->N, KV_TILE) + SEG_COST;
  long long per_rt = 0, longest = 0;
  for (int b = 0; b < p->B; ++b) {
    const long long w = prefix_tiles(p->prefix_len_host[b]) + head;
    per_rt += w * p->Hkv;
    longest = std::max(longest, w);
  }
  const long long total = per_rt * row_tiles;
  const long long chains = (long long)p->B * p->Hkv * row_tiles;
  const bool one_each = chains <= PLAN_SMS && longest <= WHOLE;
  const long long n = one_each ? chains : std::min<long long>(PLAN_SMS, std::max(chains, total / MIN_RUN));
  r.n = (int)n;
  int c = 0;
  long long acc = 0;  // weight before the sequence at hand
  for (int rt = 0; rt < row_tiles; ++rt) {
    for (int b = 0; b < p->B; ++b) {
      const long long tiles = prefix_tiles(p->prefix_len_host[b]), w = tiles + head;
      const int chain_b = (rt * p->B + b) * p->Hkv;
      // the runs that start within these Hkv chains
      while (c < r.n) {
        const long long at = one_each ? 0 : total * c / r.n - acc;
        if (!one_each && at >= w * p->Hkv) break;
        if (one_each && c >= chain_b + p->Hkv) break;
        int g = one_each ? c - chain_b : (int)(at / w);
        long long t = one_each ? 0 : at % w - head;
        if (t < SLIVER) t = 0;
        if (tiles - t < SLIVER && t > 0) {
          t = 0;
          ++g;
        }
        r.chain[c] = chain_b + g;
        r.tile[c] = (int)t;
        ++c;
      }
      acc += w * p->Hkv;
    }
  }
  r.chain[r.n] = (int)chains;
  r.tile[r.n] = 0;
  return r;
}

bool any_cut(const Runs& r) {
  for (int c = 1; c < r.n; ++c)
    if (r.tile[c] > 0) return true;
  return false;
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }
bool few_rows(int N, int G, int D) { return N * G <= FEW_ROWS && D == 128; }
// Two parts a CTA at most, of `rows` rows each.
size_t part_o_bytes(const Runs& r, int rows, int D) { return any_cut(r) ? round256((size_t)2 * r.n * rows * D * 4) : 0; }
size_t part_lse_bytes(const Runs& r, int rows) { return any_cut(r) ? round256((size_t)2 * r.n * rows * 4) : 0; }

bool encode_codes(CUtensorMap* m, const void* base, int D, const AttnArgs& a, int box_rows) {
  // codes [num_blocks * Hkv, bs, D]: a box is box_rows tokens, every channel,
  // swizzled over its 128-byte (D = 128) or 64-byte rows
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  std::memset(m, 0, sizeof(*m));
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)a.bs, (cuuint64_t)a.num_blocks * a.Hkv};
  const cuuint64_t str[2] = {(cuuint64_t)D, (cuuint64_t)a.bs * D};
  const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)box_rows, 1};
  const cuuint32_t one[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, str, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
constexpr size_t smem_bytes() {
  return sizeof(Smem<D>) + 1024;
}
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory of a CTA");

template <int D>
cudaError_t launch(Q8Args& t, const AttnQ8Args& q, cudaStream_t s) {
  const AttnArgs& a = q.a;
  CUtensorMap m_q, m_kc, m_vc, m_kt, m_vt;
  {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)a.Hq, (uint64_t)a.N, (uint64_t)a.B};
    const uint64_t str[3] = {(uint64_t)D * 2, (uint64_t)a.Hq * D * 2, (uint64_t)a.N * a.Hq * D * 2};
    const uint32_t box[4] = {64, (uint32_t)a.G, (uint32_t)(ROW_TILE / a.G), 1};
    if (!encode_bf16_sw128(&m_q, a.q, 4, dims, str, box)) return cudaErrorInvalidValue;
  }
  if (!encode_codes(&m_kc, q.k_codes, D, a, t.box_rows) || !encode_codes(&m_vc, q.v_codes, D, a, t.box_rows))
    return cudaErrorInvalidValue;
  {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)a.Hkv, (uint64_t)a.N, (uint64_t)a.B};
    const uint64_t str[3] = {(uint64_t)D * 2, (uint64_t)a.Hkv * D * 2, (uint64_t)a.N * a.Hkv * D * 2};
    const uint32_t box[4] = {64, 1, (uint32_t)KV_TILE, 1};
    if (!encode_bf16_sw128(&m_kt, a.k_tree, 4, dims, str, box) || !encode_bf16_sw128(&m_vt, a.v_tree, 4, dims, str, box))
      return cudaErrorInvalidValue;
  }
  if (few_rows(a.N, a.G, D)) return launch_attn_q8_few(t, any_cut(t.runs), m_kc, m_vc, m_kt, m_vt, s);
  cudaError_t e = launch_pdl(k_attn_q8<D>, dim3(t.runs.n), dim3(THREADS), smem_bytes<D>(), s, t, m_q, m_kc, m_vc, m_kt, m_vt);
  if (e != cudaSuccess || !any_cut(t.runs)) return e;
  const dim3 grid(t.runs.n, ROW_TILE / (MERGE_THREADS / (D / 8)));
  return launch_pdl(k_merge_q8<D>, grid, dim3(MERGE_THREADS), 0, s, t);
}

}  // namespace

cudaError_t attn_q8_prepare() {
  cudaError_t e = cudaFuncSetAttribute(k_attn_q8<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<128>());
  if (e != cudaSuccess) return e;
  e = attn_q8_few_prepare();
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(k_attn_q8<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<64>());
}

size_t attn_q8_workspace(const ts_attn_params* p) {
  const Runs r = plan_runs(p);
  const int rows = few_rows(p->N, p->Hq / p->Hkv, p->D) ? FEW_ROWS : ROW_TILE;
  return 256 + part_o_bytes(r, rows, p->D) + part_lse_bytes(r, rows);
}

cudaError_t launch_attn_q8(const AttnQ8Args& q, const ts_attn_params* p, void* workspace, cudaStream_t s) {
  const AttnArgs& a = q.a;
  Q8Args t{};
  t.a = a;
  t.kv_scale = q.kv_scale;
  t.runs = plan_runs(p);
  char* ws = static_cast<char*>(workspace) + 256;
  t.part_o = reinterpret_cast<float*>(ws);
  t.part_lse = reinterpret_cast<float*>(ws + part_o_bytes(t.runs, few_rows(a.N, a.G, a.D) ? FEW_ROWS : ROW_TILE, a.D));
  t.box_rows = KV_TILE;
  while (a.bs % t.box_rows != 0) t.box_rows >>= 1;
  t.nodes_per_tile = ROW_TILE / a.G;
  t.units = a.B * a.Hkv;
  t.n_tree = ceil_div(a.N, KV_TILE);
  t.out32 = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
  t.fd_units = FastDiv::make(t.units);
  t.fd_hkv = FastDiv::make(a.Hkv);
  t.fd_bs = FastDiv::make(a.bs);
  t.fd_g = FastDiv::make(a.G);
  return a.D == 128 ? launch<128>(t, q, s) : launch<64>(t, q, s);
}

}  // namespace ts
