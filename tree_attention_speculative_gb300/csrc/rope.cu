// Rotary positions of the tree's queries and keys.
//
// For a token at position p and each pair i < R/2 of the R rotated channels,
//   (x, y) -> m (x cos a - y sin a, y cos a + x sin a),  a = p f_i,
// the pair being channels (i, i + R/2), or (2i, 2i + 1) when interleaved; the
// other D - R channels are copied.
//
// The angle.  Only its fraction of a turn matters, and p is whole, so the host
// passes f_i / (2 pi) as a 64-bit fixed-point fraction F_i of a turn and the
// kernel takes p * F_i modulo 2^64: the turns drop out by themselves (a product
// in fp32 would be off by whole radians past p = 2^24).  The fraction that is
// left goes to sincospif in fp32, within 2^-26 of a turn.  F_i comes from
// doubles and is off by up to 2^-55.2 (f_i up to 1; theta from 1e4 to 1e7 against
// 70 digits), p times that in the angle: 2^-24.2 of a turn at p = 2^31.
//
// Memory-bound: every value is read and written once, 3 flops each.  A CTA
// takes whole tokens: its R/2 sines and cosines a token are computed once,
// into shared memory, and every head of the token reads them.  The first
// loads of the values are issued before the table, so that the sines hide
// behind them.  A thread's item is two 16-byte chunks, 8 pairs; rotary widths
// that are no multiple of 16 (and only those) go pair by pair, two bytes at a
// time.
#include "internal.cuh"

namespace ts {
namespace {

constexpr int ROPE_THREADS = 256;  // at most: a CTA has as many as leave no part of a round idle
constexpr int ROPE_MAX_TOK = 16;  // tokens a CTA: the table then holds 16 x 64 pairs, 8 KB

__device__ __forceinline__ float2 rope_sincos(int32_t pos, uint64_t turn, float mscale) {
  const uint64_t a = (uint64_t)(int64_t)pos * turn;
  const float half_turns = (float)(int32_t)(a >> 32) * 4.656612873077393e-10f;  // 2^-31: in [-1, 1]
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * mscale, s * mscale);
}

__device__ __forceinline__ float2 rope_turn(float x, float y, float2 cs) {
  return make_float2(x * cs.x - y * cs.y, y * cs.x + x * cs.y);
}

__device__ __forceinline__ float2 up(uint32_t w) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
__device__ __forceinline__ uint32_t down(float lo, float hi) {
  const __nv_bfloat162 t = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&t);
}

// Where head `h` of token `t` lies (heads: Hq of q, then Hkv of k).
struct RopeRow {
  const __nv_bfloat16* src;
  __nv_bfloat16* dst;
};
__device__ __forceinline__ RopeRow rope_row(const RopeArgs& a, int t, int h) {
  RopeRow r;
  if (h < a.Hq) {
    r.src = a.q + (size_t)t * a.q_token + (size_t)h * a.q_head;
    r.dst = a.q_out + ((size_t)t * a.Hq + h) * a.D;
  } else {
    h -= a.Hq;
    r.src = a.k + (size_t)t * a.k_token + (size_t)h * a.k_head;
    r.dst = a.k_out + ((size_t)t * a.Hkv + h) * a.D;
  }
  return r;
}

// Tables of cos, sin of the CTA's tokens: pair i of token k at [k * half + i].
__device__ __forceinline__ void rope_table(const RopeArgs& a, float2* table, int t0, int ntok) {
  const int half = a.R / 2;
  for (int e = threadIdx.x; e < ntok * half; e += blockDim.x) {
    const int k = e / half;
    table[e] = rope_sincos(a.pos[t0 + k], a.turn[e - k * half], a.mscale);
  }
}

// R a multiple of 16.  Item e of a CTA: item e % per of head e / per of its
// tokens' heads; items below R/16 of a head rotate, the rest copy.
//
// One item in flight a thread and eight CTAs an SM (32 registers): 4096 tokens
// of 72 heads of 128 in 26.1 us, 5.8 TB/s (two items, 40 registers: 28.3 us), 16384
// tokens in 90 us, 6.7 TB/s (98 us).
template <bool INTERLEAVED>
__global__ void __launch_bounds__(ROPE_THREADS, 8)
k_rope_vec(const __grid_constant__ RopeArgs a, FastDiv heads) {
  __shared__ __align__(16) float2 table[ROPE_MAX_TOK * 64];
  const int t0 = blockIdx.x * a.tok;
  const int ntok = min(a.tok, a.tokens - t0);
  const int lg = a.D == 128 ? 3 : 2;  // items a head: D / 16
  const int n = (ntok * heads.d) << lg;
  const int rot = a.R / 16, half = a.R / 2;
  pdl_wait();
  pdl_trigger();
  // item e: token k, place i in its head, channels cx and cy of its chunks (beyond
  // the rotated channels, copied, two chunks one after the other, as when interleaved)
  const auto at = [&](int e, RopeRow& r, int& k, int& i, int& cx, int& cy) {
    const int row = e >> lg;
    k = heads.div(row);
    r = rope_row(a, t0 + k, row - k * heads.d);
    i = e & ((1 << lg) - 1);
    cx = i >= rot || INTERLEAVED ? 16 * i : 8 * i;
    cy = i >= rot || INTERLEAVED ? cx + 8 : cx + half;
  };
  uint4 x, y;
  const auto load = [&](int e) {
    RopeRow r;
    int k, i, cx, cy;
    at(e, r, k, i, cx, cy);
    x = *reinterpret_cast<const uint4*>(r.src + cx);
    y = *reinterpret_cast<const uint4*>(r.src + cy);
  };
  if ((int)threadIdx.x < n) load(threadIdx.x);
  rope_table(a, table, t0, ntok);
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += blockDim.x) {
    if (e != (int)threadIdx.x) load(e);
    RopeRow r;  // (worked out again: kept over the table, it would not fit the registers)
    int k, i, cx, cy;
    at(e, r, k, i, cx, cy);
    if (i < rot) {
      uint32_t* wx = &x.x;
      uint32_t* wy = &y.x;
      const float4* cs = reinterpret_cast<const float4*>(table + k * half + 8 * i);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if (INTERLEAVED) {  // a word is a pair: pairs 8i + w in x, 8i + 4 + w in y
          const float4 c0 = cs[w / 2], c1 = cs[2 + w / 2];
          const float2 a0 = up(wx[w]), a1 = up(wy[w]);
          const float2 r0 = rope_turn(a0.x, a0.y, (w & 1) ? make_float2(c0.z, c0.w) : make_float2(c0.x, c0.y));
          const float2 r1 = rope_turn(a1.x, a1.y, (w & 1) ? make_float2(c1.z, c1.w) : make_float2(c1.x, c1.y));
          wx[w] = down(r0.x, r0.y);
          wy[w] = down(r1.x, r1.y);
        } else {  // words w of x and y hold pairs 8i + 2w and 8i + 2w + 1
          const float4 c = cs[w];
          const float2 p = up(wx[w]), q = up(wy[w]);
          const float2 r0 = rope_turn(p.x, q.x, make_float2(c.x, c.y));
          const float2 r1 = rope_turn(p.y, q.y, make_float2(c.z, c.w));
          wx[w] = down(r0.x, r1.x);
          wy[w] = down(r0.y, r1.y);
        }
      }
    } else if (r.src == r.dst) {
      continue;  // in place: the copied channels stay
    }
    *reinterpret_cast<uint4*>(r.dst + cx) = x;
    *reinterpret_cast<uint4*>(r.dst + cy) = y;
  }
}

// Any even R: an item is one pair (or two copied channels), two bytes a load, so
// that 4096 tokens of 72 heads of 128 take 61 us (R = 10, 20, 24 or 40, either
// layout; R = 32 through k_rope_vec 24 us).
__global__ void __launch_bounds__(ROPE_THREADS)
k_rope_pairs(const __grid_constant__ RopeArgs a, FastDiv heads) {
  __shared__ __align__(16) float2 table[ROPE_MAX_TOK * 64];
  const int t0 = blockIdx.x * a.tok;
  const int ntok = min(a.tok, a.tokens - t0);
  const int lg = a.D == 128 ? 6 : 5;  // items a head: D / 2
  const int n = (ntok * heads.d) << lg;
  const int half = a.R / 2;
  pdl_wait();
  pdl_trigger();
  rope_table(a, table, t0, ntok);
  __syncthreads();
  for (int e = threadIdx.x; e < n; e += blockDim.x) {
    const int row = e >> lg;
    const int k = heads.div(row);
    const RopeRow r = rope_row(a, t0 + k, row - k * heads.d);
    const int i = e & ((1 << lg) - 1);
    const int cx = i >= half || a.interleaved ? 2 * i : i;
    const int cy = i >= half || a.interleaved ? cx + 1 : i + half;
    const __nv_bfloat16 x = r.src[cx], y = r.src[cy];
    if (i < half) {
      const float2 z = rope_turn(__bfloat162float(x), __bfloat162float(y), table[k * half + i]);
      r.dst[cx] = __float2bfloat16_rn(z.x);
      r.dst[cy] = __float2bfloat16_rn(z.y);
    } else {
      r.dst[cx] = x;
      r.dst[cy] = y;
    }
  }
}

// a / b rounded up, for every a >= 1 (ceil_div's a + b - 1 passes 2^31 for the last few a).
constexpr int rope_ceil_div(int a, int b) { return (a - 1) / b + 1; }

// Tokens a CTA: enough for an item a thread, but no fewer CTAs than SMs (300
// tokens of 3 heads of 64: 2.4 us, without that 2.7).
// 16384 tokens of 9 heads of 128: 16.8 us (one token a CTA 20.1); of 2 heads of
// 64: 6.4 us (one token a CTA 17.2).
constexpr int rope_tokens_a_cta(int tokens, int items_a_token) {
  int tok = rope_ceil_div(ROPE_THREADS, items_a_token);
  const int spread = rope_ceil_div(tokens, PLAN_SMS);
  if (tok > spread) tok = spread;
  return tok < ROPE_MAX_TOK ? tok : ROPE_MAX_TOK;
}
// The most tokens a call takes, and the fewest.
static_assert(rope_tokens_a_cta(0x7fffffff, 4) == ROPE_MAX_TOK && rope_tokens_a_cta(0x7fffffff, 8192 * 64) == 1, "");
static_assert(rope_ceil_div(0x7fffffff, ROPE_MAX_TOK) == 1 << 27 && rope_ceil_div(0x7fffffff, 1) == 0x7fffffff, "");
static_assert(rope_tokens_a_cta(1, 4) == 1 && rope_tokens_a_cta(300, 12) == 2, "");

}  // namespace

cudaError_t launch_rope(RopeArgs a, cudaStream_t s) {
  const int heads = a.Hq + a.Hkv;
  const bool vec = a.R % 16 == 0;
  const int per = vec ? a.D / 16 : a.D / 2;
  a.tok = rope_tokens_a_cta(a.tokens, heads * per);
  const dim3 grid(rope_ceil_div(a.tokens, a.tok));
  // Threads: the items of a CTA in whole rounds (576 items of 72 heads of 128:
  // 192 threads, 26.1 us for 4096 tokens; 256 threads, 27.1 us).
  const int items = a.tok * heads * per;
  const int rounds = ceil_div(items, ROPE_THREADS);
  const dim3 block(32 * ceil_div(ceil_div(items, rounds), 32));
  const FastDiv fd = FastDiv::make(heads);
  if (!vec) return launch_pdl(k_rope_pairs, grid, block, 0, s, a, fd);
  return a.interleaved ? launch_pdl(k_rope_vec<true>, grid, block, 0, s, a, fd)
                       : launch_pdl(k_rope_vec<false>, grid, block, 0, s, a, fd);
}

}  // namespace ts
