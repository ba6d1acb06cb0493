// The 8-bit integer codec: one fp32 scale per row,
//   s = fp32(max|v| / 127),   q = clamp(RNE(v / s), -127, 127)
// of the exact real quotient (ties to even); s == 0 gives codes 0; a row that
// holds an infinity or a NaN gets the scale NaN and codes 0, so that what is
// computed from it is NaN.
//
// The quotient is taken as v * fp32(1/s), which is off the exact one by at most
// 127 * 2^-23 < 2^-16. Where it lands within 2^-15 of a midpoint (one value in
// 16000) the code is settled exactly: with the candidate q, e = v - q s comes
// from one fused multiply-add, and 2|e| against s decides. For q = 0 and
// |q| >= 2 that e is exact (v and q s are multiples of ulp(s), |e| is near
// s / 2 and has at most 24 bits). For |q| = 1 a v just below s / 2 can need 25
// bits; then |e| > s / 2 rounds to s / 2 at the least, which an odd q treats
// alike.
#pragma once

#include <cstdint>

#include "svdq_f32x2.cuh"

namespace svdq {

struct Int8Scale {
  float s;       // what is stored
  float rcp;     // fp32(1/s); 0: codes 0, or
  bool small;    // s is too small for the quick quotient
};

__device__ __forceinline__ Int8Scale int8_scale(float amax) {
  Int8Scale r;
  if (!(amax <= 3.4028235e38f)) return Int8Scale{__int_as_float(0x7FC00000), 0.f, false};
  r.s = __fdiv_rn(amax, 127.f);
  r.small = r.s < 1e-30f && r.s > 0.f;
  r.rcp = r.s > 0.f && !r.small ? __frcp_rn(r.s) : 0.f;
  return r;
}

// The code of v from the candidate q, |q - v/s| < 1.
__device__ __forceinline__ float int8_settle(float v, float q, float s) {
  const float e = fmaf(-q, s, v), d = fabsf(e) + fabsf(e);
  const bool odd = (__float2int_rn(q) & 1) != 0;
  if (d > s || (d == s && odd)) q += e > 0.f ? 1.f : -1.f;
  return q;
}

// Codes of v for scales too small for fp32 products: the quotient of two fp32
// values differs from a midpoint by more than 2^-34, or is one, so fp64
// rounds it right.
__device__ __forceinline__ float int8_code_small(float v, float s) {
  const double q = rint((double)v / (double)s);
  return (float)fmin(fmax(q, -127.0), 127.0);
}

constexpr float kInt8Magic = 12582912.f;   // 1.5 * 2^23: adding it rounds to an integer, left in the low bits

// Candidate codes of two values, still carrying kInt8Magic; `far` collects how
// far the quotients are from them.
__device__ __forceinline__ float2 int8_quick(float2 v, const Int8Scale& sc, float& far) {
  const float2 r = make_float2(sc.rcp, sc.rcp), magic = make_float2(kInt8Magic, kInt8Magic);
  const float2 b = fma2_rn(v, r, magic);
  const float2 d = fma2_rn(v, r, fma2_rn(b, make_float2(-1.f, -1.f), magic));
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(far) : "f"(far), "f"(d.x), "f"(d.y));
  return b;
}

__device__ __forceinline__ float int8_careful(float v, float b, const Int8Scale& sc) {
  if (sc.rcp == 0.f) return (sc.small ? int8_code_small(v, sc.s) : 0.f) + kInt8Magic;
  return int8_settle(v, b - kInt8Magic, sc.s) + kInt8Magic;
}

// N = 4 or 8 consecutive codes (the address is a multiple of N).
template <int N>
__device__ __forceinline__ void int8_store(int8_t* out, const float2 (&v)[N / 2], const Int8Scale& sc) {
  float2 b[N / 2];
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) b[i] = int8_quick(v[i], sc, far);
  if (far > 0.5f - 0x1p-15f || sc.rcp == 0.f) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) b[i] = make_float2(int8_careful(v[i].x, b[i].x, sc), int8_careful(v[i].y, b[i].y, sc));
  }
  uint32_t w[N / 4];
#pragma unroll
  for (int j = 0; j < N / 4; ++j) {
    const uint32_t lo = __byte_perm(__float_as_uint(b[2 * j].x), __float_as_uint(b[2 * j].y), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(b[2 * j + 1].x), __float_as_uint(b[2 * j + 1].y), 0x0040);
    w[j] = __byte_perm(lo, hi, 0x5410);
  }
  if constexpr (N == 4) *reinterpret_cast<uint32_t*>(out) = w[0];
  else *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
}

// The same for an array of single values, N = 1 too.
template <int N>
__device__ __forceinline__ void int8_store(int8_t* out, const float (&v)[N], const Int8Scale& sc) {
  if constexpr (N == 1) {
    float far = 0.f;
    float b = int8_quick(make_float2(v[0], 0.f), sc, far).x;
    if (far > 0.5f - 0x1p-15f || sc.rcp == 0.f) b = int8_careful(v[0], b, sc);
    out[0] = (int8_t)(__float_as_uint(b) & 0xFFu);
  } else {
    float2 p[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) p[i] = make_float2(v[2 * i], v[2 * i + 1]);
    int8_store<N>(out, p, sc);
  }
}

}  // namespace svdq
