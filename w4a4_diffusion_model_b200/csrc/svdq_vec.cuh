// 16-byte vectors of bf16, fp16 or fp32 values in global memory, as fp32
// registers and back; and the row reductions of the kernels that keep a row
// in a team of threads (norm, 8-bit quantizer).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

namespace svdq {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Values of type T in 16 bytes.
template <typename T>
inline constexpr int kVecN = 16 / (int)sizeof(T);

__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b, __nv_bfloat16) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b, __half) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  a = f.x;
  b = f.y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 p = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

template <typename T>
__device__ __forceinline__ void unpack_vec(const uint4& r, float (&f)[kVecN<T>]) {
  if constexpr (sizeof(T) == 4) {
    f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y); f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
  } else {
    unpack2(r.x, f[0], f[1], T());
    unpack2(r.y, f[2], f[3], T());
    unpack2(r.z, f[4], f[5], T());
    unpack2(r.w, f[6], f[7], T());
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack_vec(const float (&f)[kVecN<T>]) {
  if constexpr (sizeof(T) == 4) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  } else {
    return make_uint4(pack2(f[0], f[1], T()), pack2(f[2], f[3], T()), pack2(f[4], f[5], T()), pack2(f[6], f[7], T()));
  }
}

// A value that this kernel reads once: not kept in L1. (Not the read-only
// path: an output may be the input's own memory.)
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// A thread's piece of a row: one 16-byte vector (VEC) or one value.
template <typename T, bool VEC>
struct Piece {
  static constexpr int kN = VEC ? kVecN<T> : 1;
  using Raw = std::conditional_t<VEC, uint4, T>;
  __device__ static Raw zero() {
    if constexpr (VEC) return make_uint4(0, 0, 0, 0);
    else return from_float<T>(0.f);
  }
  __device__ static Raw load(const T* p) {
    if constexpr (VEC) return load_once(p);
    else return *p;
  }
  __device__ static void unpack(const Raw& r, float (&f)[kN]) {
    if constexpr (VEC) unpack_vec<T>(r, f);
    else f[0] = to_float(r);
  }
  __device__ static void store(T* p, const float (&f)[kN]) {
    if constexpr (VEC) *reinterpret_cast<uint4*>(p) = pack_vec<T>(f);
    else *p = from_float<T>(f[0]);
  }
};

// N consecutive parameters of type WT (bf16, fp16 or fp32) as fp32.
template <typename WT, int N>
__device__ __forceinline__ void load_params(const WT* p, float (&f)[N]) {
  if constexpr (N == 1) {
    f[0] = to_float(p[0]);
  } else {
    constexpr int W = kVecN<WT>;
    static_assert(N % W == 0, "parameter vector");
#pragma unroll
    for (int j = 0; j < N / W; ++j) {
      float t[W];
      unpack_vec<WT>(*reinterpret_cast<const uint4*>(p + j * W), t);
#pragma unroll
      for (int i = 0; i < W; ++i) f[j * W + i] = t[i];
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The larger of two values, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// Reductions over the team that shares a row; every thread gets the result. The
// team is the block's blockDim.x threads: a power of two up to a warp (several
// teams in the block: blockDim.y), or several warps (blockDim.y == 1). Then
// `slot` is shared memory for a value per warp, and calls that follow each other
// take alternate slots, so that one barrier per call is enough (a warp can be at
// most one call behind any other). All lanes of a warp take part, rows or not.
__device__ __forceinline__ float lanes_sum(float v) {
  if (blockDim.x >= 32) return warp_sum(v);
  for (int o = (int)blockDim.x >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

__device__ __forceinline__ float lanes_max_nan(float v) {
  if (blockDim.x >= 32) return warp_max_nan(v);
  for (int o = (int)blockDim.x >> 1; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

__device__ __forceinline__ float2 team_sum2(float a, float b, float2* slot) {
  a = lanes_sum(a);
  b = lanes_sum(b);
  if (blockDim.x <= 32) return make_float2(a, b);
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) slot[w] = make_float2(a, b);
  __syncthreads();
  const float2 v = lane < warps ? slot[lane] : make_float2(0.f, 0.f);
  return make_float2(warp_sum(v.x), warp_sum(v.y));
}

__device__ __forceinline__ float team_sum(float a, float2* slot) {
  a = lanes_sum(a);
  if (blockDim.x <= 32) return a;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) slot[w].x = a;
  __syncthreads();
  return warp_sum(lane < warps ? slot[lane].x : 0.f);
}

__device__ __forceinline__ float team_max_nan(float a, float2* slot) {
  a = lanes_max_nan(a);
  if (blockDim.x <= 32) return a;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0) slot[w].x = a;
  __syncthreads();
  return warp_max_nan(lane < warps ? slot[lane].x : 0.f);
}

}  // namespace svdq
