// Tree attention over the 8-bit paged cache: one warp a query row, one key at
// a time, with a running maximum and sum.
#include <cuda_fp8.h>

#include "internal.cuh"

namespace ts {
namespace {

__device__ __forceinline__ float e4m3(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}
__device__ __forceinline__ float scale_of(uint8_t s) { return __uint_as_float((uint32_t)s << 23); }

template <int D>
__global__ void __launch_bounds__(256)
k_attn_q8_rows(const __grid_constant__ AttnQ8Args q) {
  constexpr int C = D / 32;
  const AttnArgs& a = q.a;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (long long)a.B * a.N * a.Hq) return;
  const int h = (int)(row % a.Hq), g = h / a.G;
  const int node = (int)(row / a.Hq % a.N), b = (int)(row / a.Hq / a.N);
  const int P_dev = a.prefix_len[b];
  const long long cap = (long long)a.max_blocks * a.bs;
  const int P = (int)min((long long)max(P_dev, 0), cap);
  if (P != P_dev && lane == 0 && a.status) a.status[b] = TS_ERR_SHAPE;
  float x[C], o[C], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    x[c] = __bfloat162float(a.q[(size_t)row * D + lane * C + c]) * a.scale_log2;
    o[c] = 0.f;
  }
  const auto step = [&](const float (&k)[C], const float (&v)[C]) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) s = fmaf(x[c], k[c], s);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float mn = fmaxf(m, s);
    const float f = exp2f(m - mn), p = exp2f(s - mn);
    l = l * f + p;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = fmaf(p, v[c], o[c] * f);
    m = mn;
  };
  for (int t = 0; t < P; ++t) {
    int blk = a.block_table[(size_t)b * a.max_blocks + t / a.bs];
    if (blk < 0 || blk >= a.num_blocks) {
      if (lane == 0 && a.status) a.status[b] = TS_ERR_BAD_BLOCK;
      blk = 0;
    }
    const size_t r = ((size_t)blk * a.Hkv + g) * a.bs + t % a.bs;
    const float ks = scale_of(q.kv_scale[2 * r]), vs = scale_of(q.kv_scale[2 * r + 1]);
    float k[C], v[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      k[c] = e4m3(q.k_codes[r * D + lane * C + c]) * ks;
      v[c] = e4m3(q.v_codes[r * D + lane * C + c]) * vs;
    }
    step(k, v);
  }
  for (int j = 0; j < a.N; ++j) {
    if (!((a.anc_mask[((size_t)b * a.N + node) * a.W + j / 64] >> (j % 64)) & 1)) continue;
    const size_t r = ((size_t)b * a.N + j) * a.Hkv + g;
    float k[C], v[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      k[c] = __bfloat162float(a.k_tree[r * D + lane * C + c]);
      v[c] = __bfloat162float(a.v_tree[r * D + lane * C + c]);
    }
    step(k, v);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) a.out[(size_t)row * D + lane * C + c] = __float2bfloat16_rn(o[c] * inv);
  if (a.lse && lane == 0) a.lse[row] = (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t launch_attn_q8(const AttnQ8Args& q, cudaStream_t s) {
  const long long rows = (long long)q.a.B * q.a.N * q.a.Hq;
  const dim3 grid((unsigned)((rows + 7) / 8));
  return q.a.D == 128 ? launch_pdl(k_attn_q8_rows<128>, grid, dim3(256), 0, s, q)
                      : launch_pdl(k_attn_q8_rows<64>, grid, dim3(256), 0, s, q);
}

}  // namespace ts
