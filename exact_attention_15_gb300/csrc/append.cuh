// What the appending kernels share: 16-element parts of a head, the rotary position
// embedding's angles and turns, and the conversions.
//
// A pair (a, b) of a query or key at position p turns into
// (a cos t - b sin t, a sin t + b cos t) with t = p * inv_freq[i]. Far positions
// make t large (10^6 radians at a million tokens), where 32-bit products lose
// the angle: the turn count p * inv_freq / 2 pi is kept as a 64-bit binary
// fraction, whose integer product with p drops whole turns exactly; its top 24
// bits after that are the angle.
#pragma once

#include "paged.cuh"

namespace attn {

__device__ __forceinline__ void widen8(uint4 w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo_to_f32(u[i]);
    x[2 * i + 1] = bf16hi_to_f32(u[i]);
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                            pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
// Two values to e4m3, nearest-even, what lies beyond 448 to 448 (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// 16 elements of a head: two runs of 8.
struct Part {
  uint4 a, b;
};

// A frequency (radians per position) as a fraction of a turn, in units of 2^-64.
__device__ __forceinline__ unsigned long long turn_fraction(double inv_freq) {
  double turns = inv_freq * 0.15915494309189533577;  // 1 / 2 pi
  turns -= floor(turns);
  return static_cast<unsigned long long>(turns * 18446744073709551616.0);
}
// Cosine and sine of its angle at position `pos`.
__device__ __forceinline__ float2 turn_at(unsigned long long f, int pos) {
  const long long whole = static_cast<long long>(f * static_cast<unsigned long long>(pos));
  // half turns in [-1, 1)
  const float half = static_cast<float>(static_cast<int>(whole >> 32)) * (1.0f / 2147483648.0f);
  float sn, c;
  sincospif(half, &sn, &c);
  return make_float2(c, sn);
}
// Turns pairs (x0[e], x1[e]), or pairs of neighbours.
__device__ __forceinline__ void turn_halves(float (&x0)[8], float (&x1)[8], const float2 (&turn)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 r = turn[e];
    const float a = x0[e], c = x1[e];
    x0[e] = a * r.x - c * r.y;
    x1[e] = a * r.y + c * r.x;
  }
}
__device__ __forceinline__ void turn_neighbours(float (&x0)[8], float (&x1)[8], const float2 (&turn)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 r = turn[e], u = turn[4 + e];
    const float a = x0[2 * e], c = x0[2 * e + 1], a1 = x1[2 * e], c1 = x1[2 * e + 1];
    x0[2 * e] = a * r.x - c * r.y;
    x0[2 * e + 1] = a * r.y + c * r.x;
    x1[2 * e] = a1 * u.x - c1 * u.y;
    x1[2 * e + 1] = a1 * u.y + c1 * u.x;
  }
}

}  // namespace attn
