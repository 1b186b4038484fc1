// Tree attention over the 8-bit paged cache for units of few rows: N * G up to
// 8 query rows of heads of 128 (single nodes and the smallest trees).
//
// attn_q8.cu gives a tile's 128 MMA rows to the queries, so with four of them
// nearly all of its products, and of the shared memory they read, are padding.
// Here the tokens are the rows: S^T = K [q_hi; q_lo]^T reads a tile of codes
// once for both terms of the split queries (columns 0-7 hi, 8-15 lo), and
// O^T = V^T P^T has the channels as rows, with the widened values of the other
// form as its transposed operand.  A softmax thread owns a token of the tile,
// with every row's logit of it, and a channel of the output.
//
// The reference of a row's weights is then one value for a whole group of
// threads.  It is set at the row's first tile, and again if one of its weights
// passes 2^40: the threads vote once a tile.  Sums stay with the threads until the
// segment's end.  Two groups take alternate tiles, each with a reference, sums
// and an O of its own, joined at the segment's end: with one group a tile took
// 1.1 us, the latency of its softmax; with two, 0.85.
//
// Weights are bf16 in the product.  They are summed twice: as they are, for the
// log-sum-exp, and as rounded, for the output, where the error of a weight that
// outweighs the others then cancels.  (With what bf16 leaves of them in the eight
// idle columns of P^T the outputs had their own rounding alone, but 32 single
// nodes took 74 us, against 61 without either.)
//
// What bounds it: bytes of codes, 32.5 KB a tile and SM (0.73 us of its share
// of HBM), and where sequences are short a segment's start and end (about 5 us:
// the split queries, the tree's tile, the join).  32 sequences of 0-8K tokens,
// one node of 32 heads on 8: 64 us (3.9 TB/s; the other form 88), in blocks of 16
// tokens 72 (88); of 64 heads on 8, 74 us (89); 256 of 4K: 439 us (4.9 TB/s; 582).
// Not beyond 8 rows: with 16 a thread's registers and instructions double, and 16
// prefixes of 1-16K took 105 us against the other form's 85 of that time.
//
// Warps: 0-3 as in attn_q8.cu; 4-11 widen values (half a token's channels a
// thread) and split the queries; 12-19 softmax.
#include "attn_q8.cuh"

namespace ts {
namespace {

constexpr int FEW_D = 128;
constexpr int CONVERT_THREADS = 256;
constexpr int SOFTMAX_WARP0 = 12;
constexpr int NSB = 4;                            // S buffers
constexpr int COLS = 2 * FEW_ROWS;                // of S: hi and lo of every row
constexpr int P_ROWS = 16;                        // the fewest an MMA takes; those past FEW_ROWS hold anything
constexpr uint32_t TMEM_COLS = 256;
constexpr uint32_t TMEM_O = 0;                    // each group's
constexpr uint32_t O_STRIDE = 32;
constexpr uint32_t TMEM_S0 = 128;
constexpr float HIGH_WEIGHT = 1099511627776.f;    // 2^40 (attn_q8.cu: RESCALE_SUM)
constexpr int THREADS = 640;
constexpr int GROUP = 128;                        // softmax threads of a group
constexpr int VOTE_BARRIER = 1, SEG_BARRIER = 3;  // named barriers: a group's (1, 2), and both groups'

struct __align__(1024) Smem {
  static constexpr int NSK = 4, NSV = 4;
  uint8_t k[NSK][SLOT];
  uint8_t v[NSV][SLOT];
  uint8_t vb[NVB][KV_TILE * FEW_D * 2];  // bf16 [half][token][128 B]
  uint8_t q[2][COLS * FEW_D * 2];        // bf16 [half][column][128 B] for the tree (its lo columns are 0)
  uint8_t q8[2][COLS * FEW_D];           // e4m3 [column][128 B]
  uint8_t p[NVB][P_ROWS * KV_TILE * 2];  // bf16 [64 tokens][row][128 B]
  uint16_t v_scale[NSV][KV_TILE];
  float row_scale[4][FEW_ROWS];  // of segment s in entry s % 4; so the rows' ancestry words
  uint64_t anc[4][FEW_ROWS];
  float tree_scale[FEW_ROWS];
  float warp_max[2][4][FEW_ROWS], ref[2][FEW_ROWS];  // by group
  float2 warp_sum[2][4][FEW_ROWS];                   // of the weights, and of the rounded ones
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[NSK], k_empty[NSK];
  uint64_t v_full[NSV], v_empty[NSV];
  uint64_t vb_full[NVB], vb_empty[NVB], vt_full[NVB];
  uint64_t s_full[NSB], s_free[NSB];
  uint64_t p_full[NVB];
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort_flag;
  int q_done;     // segments whose queries are split, published by the QK issuer
  int segs_done;  // segments stored
};
static_assert(sizeof(Smem) + 1024 <= 232448, "shared memory of a CTA");

__global__ void __launch_bounds__(THREADS, 1)
k_attn_q8_few(const __grid_constant__ Q8Args args, const __grid_constant__ CUtensorMap tm_kc,
              const __grid_constant__ CUtensorMap tm_vc, const __grid_constant__ CUtensorMap tm_kt,
              const __grid_constant__ CUtensorMap tm_vt) {
  constexpr int D = FEW_D;
  constexpr int HALF_BYTES = KV_TILE * 128;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023));
  const AttnArgs& a = args.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Ctl ctl{&sm.abort_flag, a.wait_limit_ns};
  const int cta = blockIdx.x;
  const int chain0 = args.runs.chain[cta];
  const int chain1 = args.runs.chain[cta + 1] - (args.runs.tile[cta + 1] == 0 ? 1 : 0);
  const int R = a.N * a.G;

  if (threadIdx.x == 0) {
    sm.abort_flag = 0;
    sm.q_done = 0;
    sm.segs_done = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], CONVERT_THREADS);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.drain[i], 1);
    }
    for (int i = 0; i < Smem::NSK; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < Smem::NSV; ++i) {
      mbar_init(&sm.v_full[i], 1 + 32);                    // the tile, and each lane's scale bytes
      mbar_init(&sm.v_empty[i], CONVERT_THREADS + GROUP);  // widened, and the keys' scales read
    }
    for (int i = 0; i < NVB; ++i) {
      mbar_init(&sm.vb_full[i], CONVERT_THREADS);
      mbar_init(&sm.vb_empty[i], 1);
      mbar_init(&sm.vt_full[i], 1);
      mbar_init(&sm.p_full[i], GROUP);
    }
    for (int i = 0; i < NSB; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_free[i], GROUP / 32);
    }
    fence_barrier_init();
  }
  if (warp == V_WARP && lane == 0) {
    tma_prefetch_desc(&tm_kc);
    tma_prefetch_desc(&tm_vc);
    tma_prefetch_desc(&tm_kt);
    tma_prefetch_desc(&tm_vt);
    if (chain0 <= chain1) {
      // the first prefix length and table entry, into L2 (prefetches read no data; see sm100.cuh)
      const Seg I = make_seg(chain0, cta, 0, args);
      prefetch_l2(a.prefix_len + I.b);
      const int i = args.fd_bs.div(args.runs.tile[cta] * KV_TILE);
      prefetch_l2(a.block_table + (size_t)I.b * a.max_blocks + (i < a.max_blocks ? i : a.max_blocks - 1));
    }
  }
  if (threadIdx.x < FEW_ROWS) sm.tree_scale[threadIdx.x] = a.scale_log2;
  if (warp == K_WARP) tmem_alloc(&sm.tmem_base, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  pdl_wait();

  int issued = 0;               // K or V ring slots this warp filled
  int vt_issued[NVB] = {0, 0};  // tree V tiles, by buffer

  if (warp == K_WARP || warp == V_WARP) {
    load_codes<D>(sm, args, warp == V_WARP, warp == V_WARP ? &tm_vc : &tm_kc, &tm_kt, cta, chain0, chain1, ctl, issued);
  } else if (warp == QK_WARP) {
    if (lane == 0) {
      // ------------------------------------------------------------ QK issuer
      constexpr uint32_t ID_BF16 = idesc_bf16_f32(KV_TILE, COLS, 0, 0), ID_E4M3 = idesc_e4m3_f32(KV_TILE, COLS);
      int jg = 0, kq = 0, sg = 0;  // tiles, K ring slots, segments
      bool ok = true;
      int p_next = chain0 <= chain1 ? a.prefix_len[seq_of(chain0, args)] : 0;
      for (int chain = chain0; ok && chain <= chain1; ++chain) {
        const Seg I = make_seg(chain, cta, p_next, args);
        if (chain < chain1) p_next = a.prefix_len[seq_of(chain + 1, args)];
        if (I.n_tiles == 0) continue;
        const int qb = sg & 1;
        if (!(ok = wait_bar(&sm.q_full[qb], (sg >> 1) & 1, ctl))) break;
        publish(&sm.q_done, ++sg);
        const uint64_t q8_desc = smem_desc_sw128(smem_u32(sm.q8[qb]), 16, 1024);
        for (int j = 0; j < I.n_tiles; ++j, ++jg) {
          const bool tree = j < I.n_tree;
          const int s0 = kq % Smem::NSK, s1 = (kq + 1) % Smem::NSK;
          ok = wait_bar(&sm.k_full[s0], (kq / Smem::NSK) & 1, ctl);
          if (ok && tree) ok = wait_bar(&sm.k_full[s1], ((kq + 1) / Smem::NSK) & 1, ctl);
          if (ok && jg >= NSB) ok = wait_bar(&sm.s_free[jg % NSB], ((jg / NSB) - 1) & 1, ctl);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d_tmem = tmem + TMEM_S0 + (jg % NSB) * COLS;
          const uint32_t k0 = smem_u32(sm.k[s0]);
          if (tree) {
            const uint32_t k1 = smem_u32(sm.k[s1]), q = smem_u32(sm.q[qb]);
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
              mma_ss(d_tmem, smem_desc_sw128((i >> 2 ? k1 : k0) + (i & 3) * 32, 16, 1024),
                     smem_desc_sw128(q + (i >> 2) * (COLS * 128) + (i & 3) * 32, 16, 1024), ID_BF16, i > 0);
          } else {
            const uint64_t k_desc = smem_desc_sw128(k0, 16, 1024);
#pragma unroll
            for (int i = 0; i < D / 32; ++i) mma_ss_f8(d_tmem, k_desc + 2 * i, q8_desc + 2 * i, ID_E4M3, i > 0);
          }
          mma_commit(&sm.s_full[jg % NSB]);
          mma_commit(&sm.k_empty[s0]);
          if (tree) mma_commit(&sm.k_empty[s1]);
          kq += tree ? 2 : 1;
        }
        if (ok) mma_commit(&sm.q_empty[qb]);
      }
    }
  } else if (warp == PV_WARP) {
    if (lane == 0) {
      // ------------------------------------------------------------ PV issuer
      constexpr uint32_t ID_PV = idesc_bf16_f32(D, P_ROWS, 1, 0);
      int jg = 0;
      bool ok = true;
      int p_next = chain0 <= chain1 ? a.prefix_len[seq_of(chain0, args)] : 0;
      for (int chain = chain0; ok && chain <= chain1; ++chain) {
        const Seg I = make_seg(chain, cta, p_next, args);
        if (chain < chain1) p_next = a.prefix_len[seq_of(chain + 1, args)];
        for (int j = 0; j < I.n_tiles; ++j, ++jg) {
          const int buf = jg % NVB;
          ok = wait_bar(&sm.vb_full[buf], (jg / NVB) & 1, ctl) && wait_bar(&sm.p_full[buf], (jg / NVB) & 1, ctl);
          if (!ok) break;
          tc_fence_after();
          const uint64_t v_desc = smem_desc_sw128(smem_u32(sm.vb[buf]), HALF_BYTES, 1024);
          const uint32_t p = smem_u32(sm.p[buf]);
#pragma unroll
          for (int i = 0; i < KV_TILE / 16; ++i)
            mma_ss(tmem + TMEM_O + buf * O_STRIDE, v_desc + ((i * 2048) >> 4),
                   smem_desc_sw128(p + (i >> 2) * (P_ROWS * 128) + (i & 3) * 32, 16, 1024), ID_PV, j > 1 || i > 0);
          mma_commit(&sm.vb_empty[buf]);
        }
      }
    }
  } else if (warp >= CONVERT_WARP0 && warp < SOFTMAX_WARP0) {
    // ------------------------------------------------------------ conversion
    const int ct = threadIdx.x - CONVERT_WARP0 * 32;
    const int t = ct & 127, hf = ct >> 7, swz = ct & 7;  // a tile's token, its half of the channels
    const int qr = ct >> 4, qc = ct & 15;                // a query row, its 16-byte chunk
    int jg = 0, vq = 0, sg = 0;
    int vt_seen[NVB] = {0, 0};
    bool ok = true;
    uint64_t anc_next = 0;  // of thread qc = 0: its row's ancestry word
    const auto load_q = [&](int chain) -> uint4 {
      if (qr >= R) return make_uint4(0, 0, 0, 0);
      const int b = args.fd_hkv.div(chain), g = chain - b * a.Hkv;
      const int node = args.fd_g.div(qr);
      if (qc == 0) anc_next = a.anc_mask[((size_t)b * a.N + node) * a.W];
      return *reinterpret_cast<const uint4*>(a.q + (((size_t)b * a.N + node) * a.Hq + g * a.G + (qr - node * a.G)) * D + qc * 8);
    };
    int p_next = chain0 <= chain1 ? a.prefix_len[seq_of(chain0, args)] : 0;
    uint4 q_next = chain0 <= chain1 ? load_q(chain0) : make_uint4(0, 0, 0, 0);
    for (int chain = chain0; ok && chain <= chain1; ++chain) {
      const Seg I = make_seg(chain, cta, p_next, args);
      const uint4 x = q_next;
      const uint64_t anc = anc_next;
      if (chain < chain1) {  // on their way while this one runs
        p_next = a.prefix_len[seq_of(chain + 1, args)];
        q_next = load_q(chain + 1);
        if (ct == 0) {
          const Seg nx = make_seg(chain + 1, cta, 0, args);
          for (int h = 0; h < 2; ++h) tma_prefetch_4d(&tm_vt, 64 * h, nx.g, 0, nx.b);
        }
      }
      if (I.n_tiles == 0) continue;
      {
        // The queries: as they are for the tree, and for the prefix scaled to
        // within 448, hi and lo.
        const int qb = sg & 1;
        ok = sg < 2 || wait_bar(&sm.q_empty[qb], ((sg >> 1) - 1) & 1, ctl);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        uint32_t m = q8_max2(q8_max2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), q8_max2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) m = q8_max2(m, __shfl_xor_sync(0xffffffffu, m, d));
        m = q8_max2(m, m >> 16) & 0xffffu;
        const int s = q8_scale_byte(m);
        const float inv = pow2_of(254 - s);
        uint32_t hi[2], lo[2];
        split4(x.x, x.y, inv, hi[0], lo[0]);
        split4(x.z, x.w, inv, hi[1], lo[1]);
        if (qr < FEW_ROWS) {  // column qr; lo's is FEW_ROWS further
          uint8_t* to8 = sm.q8[qb] + qr * 128 + (((qc >> 1) ^ qr) << 4) + (qc & 1) * 8;
          *reinterpret_cast<uint2*>(to8) = make_uint2(hi[0], hi[1]);
          *reinterpret_cast<uint2*>(to8 + FEW_ROWS * 128) = make_uint2(lo[0], lo[1]);
          uint8_t* to = sm.q[qb] + (qc >> 3) * (COLS * 128) + qr * 128 + (((qc & 7) ^ qr) << 4);
          *reinterpret_cast<uint4*>(to) = x;
          *reinterpret_cast<uint4*>(to + FEW_ROWS * 128) = make_uint4(0, 0, 0, 0);
          // an infinite query has no finite logits
          if (qc == 0) {
            sm.row_scale[sg & 3][qr] = m == 0x7f80u ? __uint_as_float(0x7fffffffu) : fmaxf(pow2_of(s) * a.scale_log2, LEAST);
            sm.anc[sg & 3][qr] = anc;
          }
        }
        fence_proxy_async();
        mbar_arrive(&sm.q_full[qb]);
        ++sg;
      }
      for (int j = 0; j < I.n_tiles; ++j, ++jg) {
        const int buf = jg % NVB;
        uint8_t* row = sm.vb[buf] + t * 128;
        if (jg >= NVB && !(ok = wait_bar(&sm.vb_empty[buf], ((jg / NVB) - 1) & 1, ctl))) break;
        if (j < I.n_tree) {
          if (ct == 0) {
            mbar_arrive_expect_tx(&sm.vt_full[buf], 2 * HALF_BYTES);
            for (int h = 0; h < 2; ++h)
              tma_load_4d(sm.vb[buf] + h * HALF_BYTES, &tm_vt, &sm.vt_full[buf], 64 * h, I.g, j * KV_TILE, I.b);
            if (buf) ++vt_issued[1];
            else ++vt_issued[0];
          }
          if (!(ok = wait_bar(&sm.vt_full[buf], (buf ? vt_seen[1] : vt_seen[0]) & 1, ctl))) break;
          if (buf) ++vt_seen[1];
          else ++vt_seen[0];
          if (hf == 0 && t < a.N) clear_unseen<D>(row, a.anc_mask + (size_t)I.b * a.N * a.W, t, a.N, a.W);
        } else {
          const int slot = vq % Smem::NSV;
          if (!(ok = wait_bar(&sm.v_full[slot], (vq / Smem::NSV) & 1, ctl))) break;
          const bool inside = (I.t_begin + j - I.n_tree) * KV_TILE + t < I.P;
          const WideScale ws(inside ? sm.v_scale[slot][t] >> 8 : 0u, inside);
          const uint8_t* src = sm.v[slot] + t * D;
          row += hf * HALF_BYTES;
          uint4 y[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) y[c] = *reinterpret_cast<const uint4*>(src + (((4 * hf + c) ^ swz) << 4));
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint4 lo, hi;
            widen16(y[c], ws.m1, lo, hi);
            *reinterpret_cast<uint4*>(row + (((2 * c) ^ swz) << 4)) = lo;
            *reinterpret_cast<uint4*>(row + (((2 * c + 1) ^ swz) << 4)) = hi;
          }
          if (inside && ws.m2 != 0x3f803f80u) {  // (a row beyond 2^15: the rest of its power of two)
#pragma unroll 1
            for (int e = 0; e < 32; ++e) {
              uint32_t* w = reinterpret_cast<uint32_t*>(row) + e;
              *w = mul_bf16x2(*w, ws.m2);
            }
          }
          mbar_arrive(&sm.v_empty[slot]);
          ++vq;
          fence_proxy_async();
        }
        mbar_arrive(&sm.vb_full[buf]);
      }
      if (!(ok = __all_sync(0xffffffffu, ok))) break;  // (lanes whose waits gave up, and the others, leave together)
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int grp = (warp - SOFTMAX_WARP0) >> 2;   // takes every other tile
    const int t = threadIdx.x & (GROUP - 1);       // token of a tile, channel of the output
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_tmem = tmem + lane_base + TMEM_O;
    int jg = 0, vq = 0, sg = 0;  // of the segment's first tile
    bool ok = true;
    int p_next = chain0 <= chain1 ? a.prefix_len[seq_of(chain0, args)] : 0;
    for (int chain = chain0; ok && chain <= chain1; ++chain) {
      const Seg I = make_seg(chain, cta, p_next, args);
      if (chain < chain1) p_next = a.prefix_len[seq_of(chain + 1, args)];
      if (!I.p_ok && grp == 0 && t == 0 && a.status) a.status[I.b] = TS_ERR_SHAPE;
      const int slot_out = 2 * cta + (chain != chain0 ? 1 : 0);
      const int j0 = (jg ^ grp) & 1;
      uint32_t see = 0;  // rows that see node t
      float m[FEW_ROWS], l[FEW_ROWS], lw[FEW_ROWS];  // reference; sums of the weights and of the rounded ones
#pragma unroll
      for (int r = 0; r < FEW_ROWS; ++r) {
        m[r] = r < R ? NEG_INF : 0.f;  // (rows of the padding need no reference)
        l[r] = lw[r] = 0.f;
      }
      const bool split = I.n_tiles == 0 || wait_count(&sm.q_done, sg + 1, ctl);  // (voted on with the first tile)
      if (I.n_tree > 0 && j0 == 0 && t < a.N) {
        for (int r = 0; r < R; ++r) see |= (uint32_t)((sm.anc[sg & 3][r] >> t) & 1) << r;
      }
      for (int j = j0; ok && j < I.n_tiles; j += 2) {
        const int tile = jg + j, sb = tile % NSB, uses = tile / NVB;
        float key = 1.f;
        uint32_t vis = see;
        bool got = split;
        if (j >= I.n_tree) {
          const int v = vq + j - I.n_tree, slot = v % Smem::NSV;
          got = got && wait_bar(&sm.v_full[slot], (v / Smem::NSV) & 1, ctl);
          const bool inside = (I.t_begin + j - I.n_tree) * KV_TILE + t < I.P;
          key = inside ? pow2_of(sm.v_scale[slot][t] & 0xff) : 0.f;
          vis = inside ? 0xffu : 0u;
          mbar_arrive(&sm.v_empty[slot]);
        }
        got = got && wait_bar(&sm.s_full[sb], (tile / NSB) & 1, ctl);
        if (uses > 0) got = got && wait_bar(&sm.vb_empty[grp], (uses - 1) & 1, ctl);  // the group's P buffer and O
        got = __all_sync(0xffffffffu, got);
        tc_fence_after();
        const float* scale = j < I.n_tree ? sm.tree_scale : sm.row_scale[sg & 3];
        float p[FEW_ROWS];
        // logits before the row's scale
        const auto logits = [&]() {
          uint32_t u[16];
          tmem_ld16(tmem + lane_base + TMEM_S0 + sb * COLS, u);
          tmem_ld_wait();
          reg_fence16(u);
#pragma unroll
          for (int r = 0; r < 8; ++r)
            p[r] = (vis >> r) & 1u ? (__uint_as_float(u[r]) + __uint_as_float(u[r + 8])) * key : NEG_INF;
        };
        // weights; no maximum is taken while they stay below 2^40
        bool fine = true;
        const auto weights = [&]() {
#pragma unroll
          for (int r = 0; r < FEW_ROWS; ++r) {
            const float y = fmaf(p[r], scale[r], m[r] == NEG_INF ? 0.f : -m[r]);
            const bool first = m[r] == NEG_INF && p[r] > NEG_INF;
            p[r] = ex2(y);
            fine = fine && !(p[r] > HIGH_WEIGHT || first);
          }
        };
        logits();
        weights();
        if (!named_barrier_and(VOTE_BARRIER + grp, GROUP, got && fine)) {
          if (!(ok = named_barrier_and(VOTE_BARRIER + grp, GROUP, got))) break;
          // A row whose weights are too high, or that has no reference yet, moves it up to
          // its largest logit of the tile; the others keep theirs, whatever their neighbours do.
          logits();
#pragma unroll
          for (int r = 0; r < FEW_ROWS; ++r) {
            if (r >= R) break;
            float top = p[r];
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            if (lane == 0) sm.warp_max[grp][warp & 3][r] = top;
          }
          named_barrier_and(VOTE_BARRIER + grp, GROUP, true);
          uint32_t u[16];
          if (j > 1) {  // (the group's PVs so far are done)
            tmem_ld16(o_tmem + grp * O_STRIDE, u);
            tmem_ld_wait();
            reg_fence16(u);
          }
#pragma unroll
          for (int r = 0; r < FEW_ROWS; ++r) {
            if (r >= R) break;
            float top = NEG_INF;
#pragma unroll
            for (int w = 0; w < 4; ++w) top = fmaxf(top, sm.warp_max[grp][w][r]);
            const bool high = ex2(fmaf(top, scale[r], -m[r])) > HIGH_WEIGHT;  // (as weights() takes it)
            top = (m[r] == NEG_INF ? top > NEG_INF : high) ? top * scale[r] : m[r];
            const float f = m[r] == NEG_INF ? 0.f : ex2(m[r] - top);  // what earlier weights are then worth
            m[r] = top;
            l[r] *= f;
            lw[r] *= f;
            u[r] = f == 0.f ? 0u : __float_as_uint(__uint_as_float(u[r]) * f);
          }
          if (j > 1) {
            tmem_st16(o_tmem + grp * O_STRIDE, u);
            tmem_st_wait();
          }
          weights();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.s_free[sb]);
        uint8_t* to = sm.p[grp] + (t >> 6) * (P_ROWS * 128) + (t & 7) * 2;
        const int chunk = (t & 63) >> 3;
#pragma unroll
        for (int r = 0; r < FEW_ROWS; ++r) {
          const __nv_bfloat16 w = __float2bfloat16_rn(p[r]);
          l[r] += p[r];
          lw[r] += __bfloat162float(w);
          *reinterpret_cast<__nv_bfloat16*>(to + r * 128 + ((chunk ^ r) << 4)) = w;
        }
        fence_proxy_async();
        mbar_arrive(&sm.p_full[grp]);
      }
      // End of the segment: both groups' sums and O, each at its references, are
      // joined, normalised and stored, every other row by a group.
      if (ok) {
        for (int k = max(0, I.n_tiles - 2); k < I.n_tiles; ++k)
          ok = ok && wait_bar(&sm.vb_empty[(jg + k) % NVB], ((jg + k) / NVB) & 1, ctl);
      }
#pragma unroll
      for (int r = 0; r < FEW_ROWS; ++r) {
        if (r >= R) break;
        float2 y = make_float2(l[r], lw[r]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          y.x += __shfl_xor_sync(0xffffffffu, y.x, d);
          y.y += __shfl_xor_sync(0xffffffffu, y.y, d);
        }
        if (lane == 0) sm.warp_sum[grp][warp & 3][r] = y;
        if (t == 0) sm.ref[grp][r] = m[r];
      }
      if (!(ok = named_barrier_and(SEG_BARRIER, 2 * GROUP, ok))) break;
      tc_fence_after();
      if (I.n_tiles > 0) ++sg;
      jg += I.n_tiles;
      vq += I.n_prefix;
      uint32_t u[2][16];
#pragma unroll
      for (int k = 0; k < 2; ++k) tmem_ld16(o_tmem + k * O_STRIDE, u[k]);
      tmem_ld_wait();
      reg_fence16(u[0]);
      reg_fence16(u[1]);
#pragma unroll
      for (int r = 0; r < FEW_ROWS; ++r) {
        if (r >= R) break;
        if ((r & 1) != grp) continue;
        const float top = fmaxf(sm.ref[0][r], sm.ref[1][r]);
        float acc = 0.f, den = 0.f, norm = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float w = sm.ref[k][r] == NEG_INF ? 0.f : ex2(sm.ref[k][r] - top);
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            sum.x += sm.warp_sum[k][q][r].x;
            sum.y += sm.warp_sum[k][q][r].y;
          }
          den = fmaf(sum.x, w, den);
          norm = fmaf(sum.y, w, norm);
          if (w != 0.f) acc = fmaf(__uint_as_float(u[k][r]), w, acc);  // (a group without a weight: whatever its O holds)
        }
        const bool none = den == 0.f;  // the row saw no key
        const float y = none ? 0.f : acc * (1.f / norm);
        const float lse2 = none ? NEG_INF : top + __log2f(den);
        if (I.whole) {
          const int node = args.fd_g.div(r);
          const size_t orow = ((size_t)I.b * a.N + node) * a.Hq + I.g * a.G + (r - node * a.G);
          a.out[orow * D + t] = __float2bfloat16_rn(y);
          if (t == 0 && a.lse) a.lse[orow] = lse2 * 0.69314718055994531f;
        } else {
          args.part_o[((size_t)slot_out * FEW_ROWS + r) * D + t] = y;
          if (t == 0) args.part_lse[slot_out * FEW_ROWS + r] = lse2;
        }
      }
      // all have read O, the sums and this segment's scales before the next one's
      tc_fence_before();
      named_barrier_and(SEG_BARRIER, 2 * GROUP, true);
      if (grp == 0 && t == 0) publish(&sm.segs_done, chain - chain0 + 1);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (*ctl.flag) {
    // A wait gave up: as in attn_q8.cu, what is in flight lands first.
    if (warp == V_WARP) asm volatile("cp.async.wait_all;" ::: "memory");
    if ((warp == K_WARP || warp == V_WARP) && lane == 0) {
      uint64_t* full = warp == V_WARP ? sm.v_full : sm.k_full;
      const int nst = warp == V_WARP ? Smem::NSV : Smem::NSK;
      for (int j = max(0, issued - nst); j < issued; ++j) mbar_wait(&full[j % nst], (j / nst) & 1, a.wait_limit_ns);
    } else if ((warp == QK_WARP || warp == PV_WARP) && lane == 0) {
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

// Joins the parts of a chain, as k_merge_q8: block (c, i), rows 4 i .. 4 i + 3,
// a warp a row.
constexpr int MERGE_THREADS = 128;
__global__ void __launch_bounds__(MERGE_THREADS)
k_merge_q8_few(const __grid_constant__ Q8Args args) {
  const AttnArgs& a = args.a;
  const Runs& runs = args.runs;
  const int c = blockIdx.x, chain = runs.chain[c + 1];
  if (runs.tile[c + 1] == 0 || (runs.chain[c] == chain && runs.tile[c] > 0)) return;  // nothing cut, or not begun here
  const int r = blockIdx.y * (MERGE_THREADS / 32) + (int)(threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= a.N * a.G) return;
  const int b = args.fd_hkv.div(chain), g = chain - b * a.Hkv;
  int last = c + 1;
  while (last + 1 < runs.n && runs.chain[last + 1] == chain && runs.tile[last + 1] > 0) ++last;
  pdl_wait();
  pdl_trigger();
  // the parts' weights, 32 at a time a lane each, then their values, several on their way
  float m = NEG_INF, den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = c; p0 <= last; p0 += 32) {
    const int p = p0 + lane, slot = 2 * p + (p == c && runs.chain[c] != chain ? 1 : 0);
    const float lse = p <= last ? args.part_lse[(size_t)slot * FEW_ROWS + r] : NEG_INF;
    float top = lse;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    top = fmaxf(top, m);
    const float f = m == NEG_INF ? 0.f : exp2f(m - top);
    const float w = lse == NEG_INF ? 0.f : exp2f(lse - top);
    m = top;
    den *= f;
    acc = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
    const int n = min(32, last - p0 + 1);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
      const int si = __shfl_sync(0xffffffffu, slot, i);
      const float4 o = reinterpret_cast<const float4*>(args.part_o + ((size_t)si * FEW_ROWS + r) * FEW_D)[lane];
      den += wi;
      if (wi != 0.f) acc = make_float4(fmaf(o.x, wi, acc.x), fmaf(o.y, wi, acc.y), fmaf(o.z, wi, acc.z), fmaf(o.w, wi, acc.w));
    }
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  const int node = args.fd_g.div(r);
  const size_t orow = ((size_t)b * a.N + node) * a.Hq + g * a.G + (r - node * a.G);
  reinterpret_cast<uint2*>(a.out + orow * FEW_D)[lane] =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (a.lse && lane == 0) a.lse[orow] = den == 0.f ? NEG_INF : (m + log2f(den)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t attn_q8_few_prepare() {
  return cudaFuncSetAttribute(k_attn_q8_few, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem) + 1024);
}

cudaError_t launch_attn_q8_few(const Q8Args& t, bool cut, const CUtensorMap& kc, const CUtensorMap& vc,
                               const CUtensorMap& kt, const CUtensorMap& vt, cudaStream_t s) {
  cudaError_t e = launch_pdl(k_attn_q8_few, dim3(t.runs.n), dim3(THREADS), sizeof(Smem) + 1024, s, t, kc, vc, kt, vt);
  if (e != cudaSuccess || !cut) return e;
  const dim3 grid(t.runs.n, ceil_div(t.a.N * t.a.G, MERGE_THREADS / 32));
  return launch_pdl(k_merge_q8_few, grid, dim3(MERGE_THREADS), 0, s, t);
}

}  // namespace ts
