// Rotary positions with several axes (time, height, width, ...).
//
// A head's first R = sum of axis_dims elements form R/2 pairs; pair i belongs
// to the axis whose section of axis_dims / 2 pairs holds i, and turns by
//   angle(t, i) = position[t][axis(i)] * freq[i]
//   (a, b) -> (a cos - b sin, a sin + b cos),
// the same angle for every head of token t. Elements past R pass unchanged.
// Pairs are neighbours (2i, 2i+1) or halves (i, i + R/2). The gradient of the
// rotation is the rotation by the opposite angle (`inverse`).
//
// Angles of far positions: the angle is formed and reduced to half turns in
// fp64 (a position of 10^6 at frequency 1 leaves fp32 an error of 0.06 rad),
// then sincospif works on a value in [-1, 1].
//
// Bound: HBM, 2 bytes read and 2 written per 16-bit element and nothing reused
// but the angles. A block takes one token at a time (or a share of its heads
// when tokens are few): its threads first fill a table of R/2 (cos, sin) in
// shared memory, once for all heads, then stream the heads, 16 bytes of each
// operand per thread.
#pragma once

#include "svdq_ptx.cuh"
#include "svdq_vec.cuh"

namespace svdq {

constexpr int kRopeMaxAxes = 8;
constexpr int kRopeMaxD = 512;

struct RopeArgs {
  const void* x;
  void* y;
  long long xt, xh, yt, yh;      // token and head strides, in elements
  const void* pos;               // [pos_rows][axes], int32 or fp32
  const double* freq;            // [R/2]
  long long T, pos_rows;
  int heads, heads_per_block, D, R, axes;
  int axis_end[kRopeMaxAxes];    // last pair + 1 of each axis
  int pos_fp32, inverse;
};

// Position of token row `p` on the axis of pair i.
__device__ __forceinline__ double rope_position(const RopeArgs& a, long long p, int i) {
  int axis = 0;
#pragma unroll
  for (int k = 0; k < kRopeMaxAxes - 1; ++k) axis += (k < a.axes - 1 && i >= a.axis_end[k]) ? 1 : 0;
  const long long at = p * a.axes + axis;
  return a.pos_fp32 ? (double)static_cast<const float*>(a.pos)[at] : (double)static_cast<const int*>(a.pos)[at];
}


// N values at p as fp32 and back: one 16-byte vector, or one value.
template <typename T, int N>
__device__ __forceinline__ void rope_load(const T* p, float (&f)[N]) {
  if constexpr (N == 1) f[0] = to_float(*p);
  else unpack_vec<T>(load_once(p), f);
}

template <typename T, int N>
__device__ __forceinline__ void rope_store(T* p, const float (&f)[N]) {
  if constexpr (N == 1) *p = from_float<T>(f[0]);
  else *reinterpret_cast<uint4*>(p) = pack_vec<T>(f);
}

// HALVES: pairs (i, i + R/2), else (2i, 2i+1). VEC: 16-byte pieces (every
// address, stride and section boundary is a multiple of 16 bytes), else one
// pair per thread.
template <typename T, bool HALVES, bool VEC>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a) {
  __shared__ float2 cs[kRopeMaxD / 2];
  constexpr int V = VEC ? kVecN<T> : 1;
  const int half = a.R / 2;
  grid_dependency_wait();
  grid_launch_dependents();
  const int h0 = blockIdx.y * a.heads_per_block;
  const int nh = min(a.heads_per_block, a.heads - h0);
  for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
    const long long p = t % a.pos_rows;
    for (int i = threadIdx.x; i < half; i += blockDim.x) {
      // angle in half turns, reduced to [-1, 1]
      double turn = rope_position(a, p, i) * a.freq[i] * 0.31830988618379067154;
      turn -= 2.0 * rint(0.5 * turn);
      float s, c;
      sincospif((float)turn, &s, &c);
      cs[i] = make_float2(c, a.inverse ? -s : s);
    }
    __syncthreads();
    const T* x = static_cast<const T*>(a.x) + t * a.xt + h0 * a.xh;
    T* y = static_cast<T*>(a.y) + t * a.yt + h0 * a.yh;
    // items of a head: pieces of pairs, then pieces of what passes unchanged
    const int turned = HALVES ? half / V : (VEC ? a.R / V : half);
    const int items = turned + (a.D - a.R) / V;
    for (int j = threadIdx.x; j < nh * items; j += blockDim.x) {
      const int h = j / items, i = j - h * items;
      const T* xr = x + h * a.xh;
      T* yr = y + h * a.yh;
      if (i >= turned) {
        float f[V];
        const int e = a.R + (i - turned) * V;
        rope_load<T, V>(xr + e, f);
        rope_store<T, V>(yr + e, f);
      } else if constexpr (HALVES) {
        float u[V], v[V], p0[V], p1[V];
        rope_load<T, V>(xr + i * V, u);
        rope_load<T, V>(xr + half + i * V, v);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float2 w = cs[i * V + k];
          p0[k] = u[k] * w.x - v[k] * w.y;
          p1[k] = v[k] * w.x + u[k] * w.y;
        }
        rope_store<T, V>(yr + i * V, p0);
        rope_store<T, V>(yr + half + i * V, p1);
      } else if constexpr (VEC) {
        float u[V], o[V];
        rope_load<T, V>(xr + i * V, u);
#pragma unroll
        for (int k = 0; k < V; k += 2) {
          const float2 w = cs[(i * V + k) / 2];
          o[k] = u[k] * w.x - u[k + 1] * w.y;
          o[k + 1] = u[k + 1] * w.x + u[k] * w.y;
        }
        rope_store<T, V>(yr + i * V, o);
      } else {
        const float u = to_float(xr[2 * i]), v = to_float(xr[2 * i + 1]);
        const float2 w = cs[i];
        yr[2 * i] = from_float<T>(u * w.x - v * w.y);
        yr[2 * i + 1] = from_float<T>(v * w.x + u * w.y);
      }
    }
    __syncthreads();
  }
}

}  // namespace svdq
