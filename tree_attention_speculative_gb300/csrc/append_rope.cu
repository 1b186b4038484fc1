// New tokens appended to a paged cache with their rotary positions: token i of a
// sequence of P cached tokens is at position P + i; its queries and keys turn by
// that (rope.cuh), the queries go to a dense array, the keys and values to rows of
// the sequence's blocks, as bf16 or, quantised row by row (quant_row.cuh), as e4m3
// codes and a scale byte.
//
// Memory-bound: every value is read and written once.  A CTA takes whole tokens:
// one thread a token finds its sequence, position and pool row (append.cuh) while
// the first values are on their way, then the CTA makes a table of the tokens'
// sines and cosines in shared memory, which every head reads.  A thread's item is
// 16 channels of a head, two 16-byte chunks: 8 pairs of a turning one, or 16
// channels copied.  Rotary widths that are no multiple of 16 take 16 channels in
// a row as well and fetch the other half of each pair two bytes at a time.
//
// Measured: 16 prompts of 1-16K, 32 + 2 x 8 heads of 128, bf16: 500 us, 6.8 TB/s, the copy
// rate.  One token of each of 32 sequences 3.8 us, 450 tokens of 64 + 2 x 8 heads into the
// 8-bit cache 6.5 us (2.6 us of bytes): a launch and a chain of three loads (lengths, the
// table's entry, then the stores), beside which the values load.
#include "append.cuh"
#include "quant_row.cuh"
#include "rope.cuh"

namespace ts {
namespace {

constexpr int AR_THREADS = 256;
constexpr int AR_MAX_TOK = 16;
enum { HALVES_VEC = 0, ADJACENT_VEC = 1, ANY_WIDTH = 2 };

template <int D, bool Q8, int MODE>
__global__ void __launch_bounds__(AR_THREADS, Q8 || MODE == ANY_WIDTH ? 5 : 8)
k_append_rope(const __grid_constant__ AppendRopeArgs a, FastDiv heads) {
  constexpr int LANES = D / 16;  // items a head
  __shared__ __align__(16) float2 table[AR_MAX_TOK * 64];
  __shared__ long long dest[AR_MAX_TOK];  // pool row of KV head 0, or -1
  __shared__ int pos[AR_MAX_TOK];         // or -1: no sequence's
  pdl_wait();
  pdl_trigger();
  if ((int)blockIdx.x < a.len_ctas) {
    const int b = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
    if (b < a.B) {
      const int longer = append_sequence(a, b, threadIdx.x & 31);
      if (a.appended && (threadIdx.x & 31) == 0) a.appended[b] = longer;
    }
    return;
  }
  const int t0 = (blockIdx.x - a.len_ctas) * a.tok;
  const int ntok = min(a.tok, a.T - t0);
  const int n = ntok * heads.d * LANES;
  const int half = a.R / 2;
  const int i = threadIdx.x % LANES;  // the same place in every head: threads are a multiple of LANES

  // item e: its head's values, and channels cx and cy of the chunks
  int k, h, cx, cy;
  bool turns;
  const __nv_bfloat16* src;
  const auto at = [&](int e) {
    const int row = e / LANES;
    k = heads.div(row);
    h = row - k * heads.d;
    const size_t t = t0 + k;
    if (h < a.Hq) src = a.q + t * a.q_token + (size_t)h * a.q_head;
    else if (h < a.Hq + a.Hkv) src = a.k + t * a.k_token + (size_t)(h - a.Hq) * a.k_head;
    else src = a.v + t * a.v_token + (size_t)(h - a.Hq - a.Hkv) * a.v_head;
    turns = h < a.Hq + a.Hkv && 16 * i < a.R;
    cx = MODE == HALVES_VEC && turns ? 8 * i : 16 * i;
    cy = MODE == HALVES_VEC && turns ? cx + half : cx + 8;
  };
  uint4 x = make_uint4(0, 0, 0, 0), y = x;
  const auto load = [&]() {
    x = *reinterpret_cast<const uint4*>(src + cx);
    y = *reinterpret_cast<const uint4*>(src + cy);
  };
  if ((int)threadIdx.x < n) {
    at(threadIdx.x);
    load();
  }
  // (the last threads' loads run beside those of the first, which find the places)
  const bool ordered = append_ordered(a, blockDim.x - 1 - threadIdx.x, blockDim.x);
  if ((int)threadIdx.x < ntok) {
    const AppendPlace p = append_place(a, t0 + threadIdx.x);
    dest[threadIdx.x] = p.row;
    pos[threadIdx.x] = p.pos;
  }
  if (!__syncthreads_and(ordered)) {
    // some sequence's rows are not its own: such a one gets nothing
    if ((int)threadIdx.x < ntok && !append_owns(a, t0 + threadIdx.x)) dest[threadIdx.x] = pos[threadIdx.x] = -1;
    __syncthreads();
  }
  for (int e = threadIdx.x; e < ntok * half; e += blockDim.x) {
    const int kk = e / half;
    table[e] = rope_sincos(pos[kk], a.turn[e - kk * half], a.mscale);
  }
  __syncthreads();
  const int rounds = (n + blockDim.x - 1) / blockDim.x;  // the same on every lane: the shuffles need them all
  for (int it = 0; it < rounds; ++it) {
    const int e = threadIdx.x + it * blockDim.x;
    const bool valid = e < n;
    if (valid) {
      at(e);
      if (it > 0) load();
    }
    if (valid && turns) {
      if constexpr (MODE == ANY_WIDTH) {
        uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int c2 = 0; c2 < 8; ++c2) {
          const int c = 16 * i + 2 * c2;  // R is even: both channels turn or neither
          if (c >= a.R) break;
          const float2 f = up(w[c2]);
          if (a.interleaved) {
            const float2 z = rope_turn(f.x, f.y, table[k * half + c / 2]);
            w[c2] = down(z.x, z.y);
          } else {
            float z[2];
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const int ch = c + o;
              const bool first = ch < half;
              const float other = __bfloat162float(src[first ? ch + half : ch - half]);
              const float own = o ? f.y : f.x;
              const float2 cs = table[k * half + (first ? ch : ch - half)];
              const float2 r = first ? rope_turn(own, other, cs) : rope_turn(other, own, cs);
              z[o] = first ? r.x : r.y;
            }
            w[c2] = down(z[0], z[1]);
          }
        }
        x = make_uint4(w[0], w[1], w[2], w[3]);
        y = make_uint4(w[4], w[5], w[6], w[7]);
      } else {
        rope_chunks<MODE == ADJACENT_VEC>(x, y, table + k * half + 8 * i);
      }
    }
    int s = 0;
    if constexpr (Q8) {
      const uint32_t m = q8_row_max<LANES>(q8_max2_nan(q8_fold(x), q8_fold(y)));
      s = m > 0x7f80u ? Q8_NAN_SCALE : q8_scale_byte(m);
    }
    if (!valid) continue;
    if (h < a.Hq) {
      if (pos[k] >= 0) {
        __nv_bfloat16* dst = a.q_out + ((size_t)(t0 + k) * a.Hq + h) * D;
        *reinterpret_cast<uint4*>(dst + cx) = x;
        *reinterpret_cast<uint4*>(dst + cy) = y;
      }
      continue;
    }
    const long long base = dest[k];
    if (base < 0) continue;
    const int is_v = h >= a.Hq + a.Hkv;
    const size_t row = (size_t)base + (size_t)(h - a.Hq - (is_v ? a.Hkv : 0)) * a.bs;
    void* cache = is_v ? a.v_cache : a.k_cache;
    if constexpr (Q8) {
      uint8_t* dst = static_cast<uint8_t*>(cache) + row * D;
      const uint2 nan = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
      *reinterpret_cast<uint2*>(dst + cx) = s == Q8_NAN_SCALE ? nan : q8_codes(x, s);
      *reinterpret_cast<uint2*>(dst + cy) = s == Q8_NAN_SCALE ? nan : q8_codes(y, s);
      if (i == 0) a.kv_scale[2 * row + is_v] = (uint8_t)s;
    } else {
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(cache) + row * D;
      *reinterpret_cast<uint4*>(dst + cx) = x;
      *reinterpret_cast<uint4*>(dst + cy) = y;
    }
  }
}

template <int D, bool Q8>
cudaError_t launch(const AppendRopeArgs& a, unsigned ctas, unsigned threads, FastDiv fd, cudaStream_t s) {
  if (a.R % 16) return launch_pdl(k_append_rope<D, Q8, ANY_WIDTH>, dim3(ctas), dim3(threads), 0, s, a, fd);
  return a.interleaved ? launch_pdl(k_append_rope<D, Q8, ADJACENT_VEC>, dim3(ctas), dim3(threads), 0, s, a, fd)
                       : launch_pdl(k_append_rope<D, Q8, HALVES_VEC>, dim3(ctas), dim3(threads), 0, s, a, fd);
}

}  // namespace

cudaError_t launch_append_rope(AppendRopeArgs a, cudaStream_t s) {
  const int heads = a.Hq + 2 * a.Hkv, per = a.D / 16;
  // Tokens a CTA: two items a thread, but no fewer CTAs than SMs.  Prompts of 1-16K 497 us
  // (one item a thread 514, four 498), 450 tokens of 80 heads 6.4 (6.7, 8.5); 32 tokens,
  // one a CTA 3.9, two 4.6.
  a.tok = 2 * ceil_div(AR_THREADS, heads * per);
  const int spread = a.T ? (a.T - 1) / PLAN_SMS + 1 : 1;
  a.tok = a.tok > spread ? spread : a.tok;
  a.tok = a.tok > AR_MAX_TOK ? AR_MAX_TOK : a.tok;
  // threads: the items of a CTA in whole rounds
  const int items = a.tok * heads * per;
  const unsigned threads = 32 * ceil_div(ceil_div(items, ceil_div(items, AR_THREADS)), 32);
  a.len_ctas = ceil_div(a.B, threads / 32);
  const long long ctas = (a.T ? (a.T - 1) / a.tok + 1ll : 0ll) + a.len_ctas;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  const FastDiv fd = FastDiv::make(heads);
  if (a.D == 128)
    return a.kv_scale ? launch<128, true>(a, ctas, threads, fd, s) : launch<128, false>(a, ctas, threads, fd, s);
  return a.kv_scale ? launch<64, true>(a, ctas, threads, fd, s) : launch<64, false>(a, ctas, threads, fd, s);
}

}  // namespace ts
