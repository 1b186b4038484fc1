// Rotary positions: the angle of a pair at a position, and its turn.
//
// The angle.  Only its fraction of a turn matters, and p is whole, so the host
// passes f_i / (2 pi) as a 64-bit fixed-point fraction F_i of a turn and the
// kernel takes p * F_i modulo 2^64: the turns drop out by themselves (a product
// in fp32 would be off by whole radians past p = 2^24).  The fraction that is
// left goes to sincospif in fp32, within 2^-26 of a turn.  F_i comes from
// doubles and is off by up to 2^-55.2 (f_i up to 1; theta from 1e4 to 1e7 against
// 70 digits), p times that in the angle: 2^-24.2 of a turn at p = 2^31.
#pragma once

#include "internal.cuh"

namespace ts {

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

// Two 16-byte chunks x and y of a head turn in place, 8 pairs whose cosines and
// sines are at cs: pair k of them is words of x (first of the pair) and y, or
// with adjacent pairs one word, of x for k < 4 and of y after.
template <bool INTERLEAVED>
__device__ __forceinline__ void rope_chunks(uint4& x, uint4& y, const float2* pairs) {
  uint32_t* wx = &x.x;
  uint32_t* wy = &y.x;
  const float4* cs = reinterpret_cast<const float4*>(pairs);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (INTERLEAVED) {  // pairs w in x, 4 + w in y
      const float4 c0 = cs[w / 2], c1 = cs[2 + w / 2];
      const float2 a0 = up(wx[w]), a1 = up(wy[w]);
      const float2 r0 = rope_turn(a0.x, a0.y, (w & 1) ? make_float2(c0.z, c0.w) : make_float2(c0.x, c0.y));
      const float2 r1 = rope_turn(a1.x, a1.y, (w & 1) ? make_float2(c1.z, c1.w) : make_float2(c1.x, c1.y));
      wx[w] = down(r0.x, r0.y);
      wy[w] = down(r1.x, r1.y);
    } else {  // words w of x and y hold pairs 2w and 2w + 1
      const float4 c = cs[w];
      const float2 p = up(wx[w]), q = up(wy[w]);
      const float2 r0 = rope_turn(p.x, q.x, make_float2(c.x, c.y));
      const float2 r1 = rope_turn(p.y, q.y, make_float2(c.z, c.w));
      wx[w] = down(r0.x, r1.x);
      wy[w] = down(r0.y, r1.y);
    }
  }
}

}  // namespace ts
