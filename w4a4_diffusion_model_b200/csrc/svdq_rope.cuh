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
// but the angles. A block takes a few tokens (or a share of one token's heads
// when tokens are few): its threads first fill a table of (cos, sin) in shared
// memory, once for all heads, then stream the heads. A thread keeps one 16-byte
// place of the head and walks the (token, head) rows, the next rows' loads always
// ahead of the present rows' arithmetic, the first ones ahead of the angles.
// 32760 x 40 x 128 bf16 halves 111 us (6.0 TB/s), 4608 x 48 x 128 inside a merged
// projection 22.9 us (4.9 TB/s).
#pragma once

#include "svdq_ptx.cuh"
#include "svdq_rows.cuh"
#include "svdq_vec.cuh"

namespace svdq {

constexpr int kRopeMaxAxes = 8;
constexpr int kRopeMaxD = 512;
constexpr int kRopeTable = 512;    // (cos, sin) of a block's tokens
constexpr int kRopeThreads = 256;

struct RopeArgs {
  const void* x;
  void* y;
  long long xt, xh, yt, yh;      // token and head strides, in elements
  const void* pos;               // [pos_rows][axes], int32 or fp32
  const double* freq;            // [R/2]
  int T, pos_rows;
  int heads, heads_per_block, tokens_per_block, D, R, axes;
  int axis_end[kRopeMaxAxes];    // last pair + 1 of each axis; past every pair where there is no axis
  int pos_fp32, inverse;
};

// Position of row `p` on the axis of pair i.
__device__ __forceinline__ double rope_position(const RopeArgs& a, unsigned p, int i) {
  int axis = 0;
#pragma unroll
  for (int k = 0; k < kRopeMaxAxes - 1; ++k) axis += i >= a.axis_end[k] ? 1 : 0;
  const size_t at = (size_t)p * a.axes + axis;
  return a.pos_fp32 ? (double)static_cast<const float*>(a.pos)[at] : (double)static_cast<const int*>(a.pos)[at];
}

// A place of the head: what a thread loads, turns and stores of it.
// Interleaved pairs: one piece of V values, V / 2 pairs; halves: V values of
// each half, V pairs. The paired fp32 instructions fit halves (two pairs' first
// elements beside each other); interleaved pairs would have to be swapped for
// them, which costs what they save.
template <typename T, bool HALVES, bool VEC>
struct RopePlace {
  static constexpr int V = VEC ? kVecN<T> : HALVES ? 1 : 2;
  static constexpr int kPairs = HALVES ? V : V / 2;
  struct Raw {
    uint4 a, b;
    T s, t;
  };
  struct Turn {
    float c[kPairs], s[kPairs];
  };
  __device__ static void load(Raw& r, const T* p, int half) {
    if constexpr (VEC) {
      r.a = load_once(p);
      if constexpr (HALVES) r.b = load_once(p + half);
    } else {
      r.s = p[0];
      r.t = p[HALVES ? half : 1];
    }
  }
  __device__ static void turn(const Raw& r, const Turn& w, T* p, int half) {
    if constexpr (!VEC) {
      const float a = to_float(r.s), b = to_float(r.t);
      p[0] = from_float<T>(fmaf(-b, w.s[0], a * w.c[0]));
      p[HALVES ? half : 1] = from_float<T>(fmaf(a, w.s[0], b * w.c[0]));
    } else if constexpr (!HALVES) {
      float f[V], o[V];
      unpack_vec<T>(r.a, f);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        o[2 * i] = fmaf(-f[2 * i + 1], w.s[i], f[2 * i] * w.c[i]);
        o[2 * i + 1] = fmaf(f[2 * i], w.s[i], f[2 * i + 1] * w.c[i]);
      }
      *reinterpret_cast<uint4*>(p) = pack_vec<T>(o);
    } else {
      float2 a[V / 2], b[V / 2], o[V / 2];
      unpack_pairs<T>(r.a, a);
      unpack_pairs<T>(r.b, b);
#pragma unroll
      for (int i = 0; i < V / 2; ++i)
        o[i] = fma2_rn(b[i], make_float2(-w.s[2 * i], -w.s[2 * i + 1]),
                       mul2_rn(a[i], make_float2(w.c[2 * i], w.c[2 * i + 1])));
      *reinterpret_cast<uint4*>(p) = pack_pairs<T>(o);
#pragma unroll
      for (int i = 0; i < V / 2; ++i)
        o[i] = fma2_rn(a[i], make_float2(w.s[2 * i], w.s[2 * i + 1]),
                       mul2_rn(b[i], make_float2(w.c[2 * i], w.c[2 * i + 1])));
      *reinterpret_cast<uint4*>(p + half) = pack_pairs<T>(o);
    }
  }
};

// Walks the rows (token, head) of a block in steps of `per_pass` heads.
template <typename P>
struct RopeCursor {
  P* p;
  int k, h;                      // token and head within the block
  long long step, wrap;          // elements per step, and from a token's heads to the next token's
  __device__ void next(int per_pass, int nh) {
    p += step;
    h += per_pass;
    while (h >= nh) {
      h -= nh;
      ++k;
      p += wrap;
    }
  }
};

// HALVES: pairs (i, i + R/2), else (2i, 2i+1). VEC: 16-byte pieces (every
// address, stride and section boundary is a multiple of 16 bytes), else one
// pair per thread.
template <typename T, bool HALVES, bool VEC>
__global__ void __launch_bounds__(kRopeThreads, HALVES ? 3 : 4) rope_kernel(const RopeArgs a) {
  using Place = RopePlace<T, HALVES, VEC>;
  constexpr int NP = Place::kPairs;
  constexpr int kRows = HALVES ? 1 : 2;   // loaded at a time (two loads; twice as many measured no faster)
  __shared__ __align__(16) float table[2][kRopeTable];   // cos and sin, [token][pair]
  const int half = a.R / 2;
  const int h0 = blockIdx.y * a.heads_per_block;
  const int nh = min(a.heads_per_block, a.heads - h0);
  const int t0 = blockIdx.x * a.tokens_per_block;
  const int nt = min(a.tokens_per_block, a.T - t0);
  // places of a head that turn, then 16-byte (or single) pieces that do not
  const int turned = half / NP;
  constexpr int kCopy = VEC ? kVecN<T> : 1;
  const int items = turned + (a.D - a.R) / kCopy;
  const int per_pass = max(1, (int)blockDim.x / items);       // heads a pass of the block covers
  const int first = (int)threadIdx.x / items;
  int item = (int)threadIdx.x - first * items;
  const bool works = first < per_pass;
  const int at = HALVES ? item * NP : 2 * item * NP;
  RopeCursor<const T> in = {static_cast<const T*>(a.x) + t0 * a.xt + (h0 + first) * a.xh, 0, first, per_pass * a.xh,
                            a.xt - nh * a.xh};
  RopeCursor<T> out = {static_cast<T*>(a.y) + t0 * a.yt + (h0 + first) * a.yh, 0, first, per_pass * a.yh,
                       a.yt - nh * a.yh};
  while (in.h >= nh) {           // more heads a pass than the block's tokens have
    in.h -= nh;
    ++in.k;
    in.p += in.wrap;
    out.h -= nh;
    ++out.k;
    out.p += out.wrap;
  }
  const RopeCursor<const T> in0 = in;
  const RopeCursor<T> out0 = out;
  grid_dependency_wait();
  grid_launch_dependents();
  // the first rows are on their way while the angles are formed
  typename Place::Raw r[kRows];
  auto fetch = [&](typename Place::Raw (&r)[kRows]) {
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      if (in.k < nt) {
        Place::load(r[u], in.p + at, half);
        in.next(per_pass, nh);
      }
  };
  const bool turns = works && item < turned;
  if (turns) fetch(r);
  for (int j = threadIdx.x; j < nt * half; j += blockDim.x) {
    const unsigned k = (unsigned)j / (unsigned)half, i = (unsigned)j - k * (unsigned)half;
    unsigned p = (unsigned)t0 + k;
    if (a.pos_rows != a.T) p %= (unsigned)a.pos_rows;
    // angle in half turns, reduced to [-1, 1]
    double turn = rope_position(a, p, (int)i) * a.freq[i] * 0.31830988618379067154;
    turn -= 2.0 * rint(0.5 * turn);
    float s, c;
    sincospif((float)turn, &s, &c);
    table[0][j] = c;
    table[1][j] = a.inverse ? -s : s;
  }
  __syncthreads();
  while (turns && out.k < nt) {
    typename Place::Raw ahead[kRows];
    fetch(ahead);
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      if (out.k < nt) {
        typename Place::Turn w;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          w.c[i] = table[0][out.k * half + item * NP + i];
          w.s[i] = table[1][out.k * half + item * NP + i];
        }
        Place::turn(r[u], w, out.p + at, half);
        out.next(per_pass, nh);
        r[u] = ahead[u];
      }
  }
  if (!works) return;
  // what passes unchanged, and (single pairs of a head wider than the block) the places past the block's threads
  for (; item < items; item += blockDim.x) {
    in = in0;
    out = out0;
    for (; out.k < nt; in.next(per_pass, nh), out.next(per_pass, nh)) {
      if (item >= turned) {
        const int c = a.R + (item - turned) * kCopy;
        if constexpr (VEC) *reinterpret_cast<uint4*>(out.p + c) = load_once(in.p + c);
        else out.p[c] = in.p[c];
      } else if (item >= (int)blockDim.x) {
        const int c = HALVES ? item * NP : 2 * item * NP;
        typename Place::Raw raw;
        typename Place::Turn w;
        Place::load(raw, in.p + c, half);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          w.c[i] = table[0][out.k * half + item * NP + i];
          w.s[i] = table[1][out.k * half + item * NP + i];
        }
        Place::turn(raw, w, out.p + c, half);
      } else {
        break;
      }
    }
  }
}

}  // namespace svdq
