// The 8-bit integer codec: one fp32 scale per row,
//   s = fp32(max|v| * fp32(1/127)),   q = clamp(RNE(v / s), -127, 127)
// of the exact real quotient (ties to even); s == 0 gives codes 0; a row that
// holds an infinity or a NaN gets the scale NaN and codes 0, so that what is
// computed from it is NaN.
//
// The scale is a product and not the quotient max|v| / 127, so that scales and codes
// are those which elementary tensor operations give on a GPU, where a division by a
// number multiplies by its fp32 reciprocal. That costs a sixteenth of a step:
// fp32(1/127) is (1/127) (1 - 2^-28), so s is within 1/2 + 1/16 of its steps of
// max|v| / 127 (the rounded quotient within 1/2; they differ in 4 to 5 % of the
// rows, by one step), and v / s within 127 * (2^-24 + 2^-28) of 127 v / max|v|.
//
// The quotient is taken as v * fp32(1/s), its product rounded only with the sum
// that makes an integer of it, so it is off the exact one by at most
// 127 * 2^-24 < 2^-17. Pieces in which one lands within 2^-16 of a midpoint are
// settled exactly: with the candidate q, e = v - q s comes from one fused
// multiply-add, and 2|e| against s decides. For q = 0 and |q| >= 2 that e is
// exact (v and q s are multiples of ulp(s), |e| is near s / 2 and has at most 24
// bits). For |q| = 1 a v just below s / 2 can need 25 bits; then |e| > s / 2
// rounds to s / 2 at the least, which an odd q treats alike. Settling is no rare
// case: 16-bit values over their own maximum are ratios of small integers, and in
// rows whose maximum has a short significand many of 127 v / max fall on a
// midpoint (all 256 values of a warp's piece are settled when one of them does).
#pragma once

#include <cstdint>

#include "svdq_int4.cuh"   // fma2_rn

namespace svdq {

struct Int8Scale {
  float s;        // what is stored
  float rcp;      // fp32(1/s); 0: codes 0
  bool special;   // the row is not finite, or s too small for fp32 quotients
};

__device__ __forceinline__ Int8Scale int8_scale(float amax) {
  if (!(amax <= 3.4028235e38f)) return Int8Scale{__int_as_float(0x7FC00000), 0.f, true};
  Int8Scale r;
  r.s = amax * (1.f / 127.f);
  r.special = r.s < 1e-30f && r.s > 0.f;
  r.rcp = r.s >= 1e-30f ? __frcp_rn(r.s) : 0.f;
  return r;
}

constexpr float kInt8Magic = 12582912.f;   // 1.5 * 2^23: adding it rounds to an integer, left in the low bits
constexpr float kInt8Near = 0.5f - 0x1p-16f;

// Candidate codes of two values, still carrying kInt8Magic; `far` collects how
// far the quotients are from them.
__device__ __forceinline__ float2 int8_quick(float2 v, float rcp, float& far) {
  const float2 r = make_float2(rcp, rcp), magic = make_float2(kInt8Magic, kInt8Magic);
  const float2 b = fma2_rn(v, r, magic);
  const float2 d = fma2_rn(v, r, fma2_rn(b, make_float2(-1.f, -1.f), magic));
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(far) : "f"(far), "f"(d.x), "f"(d.y));
  return b;
}

// One step from candidate b towards v where 2|e| > s, or where they are equal
// and the code is odd (b's last bit): d = 2|e| - s as an integer is then positive
// with that bit added.
__device__ __forceinline__ float int8_step(float b, float e, float s) {
  const float d = fmaf(2.f, fabsf(e), -s);
  return __float_as_int(d) + (__float_as_int(b) & 1) > 0 ? b + copysignf(1.f, e) : b;
}

__device__ __forceinline__ float2 int8_settle(float2 v, float2 b, float s) {
  const float2 q = fma2_rn(b, make_float2(-1.f, -1.f), make_float2(kInt8Magic, kInt8Magic));   // -q
  const float2 e = fma2_rn(q, make_float2(s, s), v);
  return make_float2(int8_step(b.x, e.x, s), int8_step(b.y, e.y, s));
}

// Codes of a special row: 0 where it is not finite; else v and s are brought
// into range by 2^100, and the code is clamped (s has so few bits that max / s
// can pass 127).
__device__ __noinline__ float2 int8_special(float2 v, float s) {
  if (!(s < 1.f)) return make_float2(kInt8Magic, kInt8Magic);
  const float k = 0x1p100f, t = s * k;
  float far = 0.f;
  v = make_float2(fminf(fmaxf(v.x * k, -127.f * t), 127.f * t), fminf(fmaxf(v.y * k, -127.f * t), 127.f * t));
  return int8_settle(v, int8_quick(v, __frcp_rn(t), far), t);
}

// N = 4 or 8 consecutive codes (the address is a multiple of N).
template <int N>
__device__ __forceinline__ void int8_store(int8_t* out, const float2 (&v)[N / 2], const Int8Scale& sc) {
  float2 b[N / 2];
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < N / 2; ++i) b[i] = int8_quick(v[i], sc.rcp, far);
  if (far > kInt8Near) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) b[i] = int8_settle(v[i], b[i], sc.s);
  }
  if (sc.special) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) b[i] = int8_special(v[i], sc.s);
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
    const float2 one = make_float2(v[0], 0.f);
    float far = 0.f;
    float2 b = int8_quick(one, sc.rcp, far);
    if (far > kInt8Near) b = int8_settle(one, b, sc.s);
    if (sc.special) b = int8_special(one, sc.s);
    out[0] = (int8_t)(__float_as_uint(b.x) & 0xFFu);
  } else {
    float2 p[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) p[i] = make_float2(v[2 * i], v[2 * i + 1]);
    int8_store<N>(out, p, sc);
  }
}

}  // namespace svdq
