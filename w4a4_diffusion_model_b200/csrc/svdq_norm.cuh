// Layer norm over the channels of each row, its gradient, and the same norm
// with the 8-bit quantizer of the next product behind it.
//
//   y[m][c] = (x[m][c] - mean[m]) rstd[m] w[g][c] + b[g][c],   g = m / rows_per_group
//   rstd = 1 / sqrt(var + eps), var = mean of (x - mean)^2
// The rows of a group share their weight and bias: one group is the affine
// norm, a group per image is the modulated norm of a diffusion transformer
// (add_one: w = 1 + scale, added in fp32). Backward, with h = dy w and
// xhat = (x - mean) rstd:
//   dx = rstd (h - mean_c(h) - xhat mean_c(h xhat))
//   dw[g] = sum over the group's rows of dy xhat,   db[g] = sum of dy
//
// All sums are fp32. The variance is taken around the mean in a second sweep
// over the row's registers (E[x^2] - mean^2 loses the digits of rows whose
// mean is large). Bound: HBM (2 or 3 row passes of 2 or 4 bytes).
#pragma once

#include "svdq_int8_codec.cuh"
#include "svdq_ptx.cuh"
#include "svdq_rows.cuh"
#include "svdq_vec.cuh"

namespace svdq {

struct NormArgs {
  const void* x;
  long long ldx;
  const void* w;         // [groups][C] or null (1)
  const void* b;         // [groups][C] or null (0)
  float* mean;           // [M]; written by the forward pass if non-null, read by the backward pass
  float* rstd;
  long long M, rows_per_group;
  int C;
  float eps, add;        // added to w: 1 with add_one
  // forward
  void* y;
  long long ldy;
  // forward with the 8-bit quantizer
  const float* inv_lambda;   // [C] or null
  int8_t* q;                 // [M][C]
  float* s;                  // [M]
  // backward
  const void* dy;
  long long lddy;
  void* dx;
  long long lddx;
  float* dw;             // [groups][C] or null
  float* db;
  float* part;           // [chunks][2][groups][C] partial sums of dw and db, null: one chunk, straight to dw and db
  int chunks;            // row chunks per group
  int depth;             // stages of the row ring
};

template <typename WT, int N>
__device__ __forceinline__ void norm_gain(const NormArgs& a, long long g, int c, float (&w)[N]) {
  if (a.w) {
    load_params<WT, N>(static_cast<const WT*>(a.w) + g * a.C + c, w);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] += a.add;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = 1.f;
  }
}

// A team of blockDim.x threads takes a row at a time: a warp (several teams
// in the block: blockDim.y) or the whole block (blockDim.y == 1). A thread
// holds NV pieces of the row.
template <typename T, typename WT, int NV, int MAXT, bool VEC, bool QUANT>
__global__ void __launch_bounds__(MAXT, 1) layernorm_kernel(const NormArgs a) {
  using P = Piece<T, VEC>;
  constexpr int N = P::kN;
  __shared__ float2 slots[3][32];
  const int warps = blockDim.x >> 5, tid = threadIdx.x;
  const float inv_c = 1.f / (float)a.C;
  grid_dependency_wait();
  grid_launch_dependents();
  const long long teams = (long long)gridDim.x * blockDim.y;
  for (long long m = (long long)blockIdx.x * blockDim.y + threadIdx.y; m < a.M; m += teams) {
    const T* x = static_cast<const T*>(a.x) + m * a.ldx;
    typename P::Raw r[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * (int)blockDim.x + tid) * N;
      r[v] = c < a.C ? P::load(x + c) : P::zero();
    }
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float f[N];
      P::unpack(r[v], f);
#pragma unroll
      for (int i = 0; i < N; ++i) sum += f[i];
    }
    const float mean = team_sum(sum, warps, slots[0]) * inv_c;
    float sq = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if ((v * (int)blockDim.x + tid) * N < a.C) {
        float f[N];
        P::unpack(r[v], f);
#pragma unroll
        for (int i = 0; i < N; ++i) sq = fmaf(f[i] - mean, f[i] - mean, sq);
      }
    }
    const float rstd = 1.f / sqrtf(team_sum(sq, warps, slots[1]) * inv_c + a.eps);
    if (tid == 0) {
      if (a.mean) a.mean[m] = mean;
      if (a.rstd) a.rstd[m] = rstd;
    }
    const long long g = m / a.rows_per_group;
    auto value = [&](int v, int c, float (&f)[N]) {
      float w[N], b[N];
      P::unpack(r[v], f);
      norm_gain<WT, N>(a, g, c, w);
      if (a.b) load_params<WT, N>(static_cast<const WT*>(a.b) + g * a.C + c, b);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = fmaf((f[i] - mean) * rstd, w[i], a.b ? b[i] : 0.f);
    };
    if constexpr (!QUANT) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * (int)blockDim.x + tid) * N;
        if (c < a.C) {
          float f[N];
          value(v, c, f);
          P::store(static_cast<T*>(a.y) + m * a.ldy + c, f);
        }
      }
    } else {
      float q[NV][N], amax = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * (int)blockDim.x + tid) * N;
        if (c < a.C) {
          value(v, c, q[v]);
          if (a.inv_lambda) {
            float l[N];
            load_params<float, N>(a.inv_lambda + c, l);
#pragma unroll
            for (int i = 0; i < N; ++i) q[v][i] *= l[i];
          }
#pragma unroll
          for (int i = 0; i < N; ++i) amax = max_nan(amax, fabsf(q[v][i]));
        }
      }
      const Int8Scale sc = int8_scale(team_max_nan(amax, warps, slots[2]));
      if (tid == 0) a.s[m] = sc.s;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * (int)blockDim.x + tid) * N;
        if (c < a.C) int8_store<N>(a.q + m * a.C + c, q[v], sc);
      }
    }
  }
}

// Forward for rows of more than one warp: a block per row, rows streamed through
// the ring, weight and bias of the group kept in registers. Thread t holds the
// pieces t, t + blockDim.x, ... of a row (kRowElems values).
//
// Mean and variance take one barrier: each warp forms its own mean and its own
// sum of squares around that mean, and the block joins them,
//   M2 = sum_w (M2_w + n_w (mean_w - mean)^2).
template <typename T, typename WT, int MAXT, bool QUANT>
__global__ void __launch_bounds__(MAXT, 1) layernorm_rows_kernel(const NormArgs a) {
  constexpr int N = kVecN<T>, NV = kRowPieces<T>;
  extern __shared__ __align__(16) unsigned char norm_ring[];
  __shared__ float2 slots[2][32];
  __shared__ float2 counts[32];                  // n_w and 1 / n_w
  __shared__ uint64_t full[kRingMaxStages];
  const int warps = blockDim.x >> 5, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float inv_c = 1.f / (float)a.C;
  RowRing<1> ring = {norm_ring, full, {static_cast<const unsigned char*>(a.x)}, {a.ldx * (long long)sizeof(T)},
                     (uint32_t)(a.C * (int)sizeof(T)), a.depth};
  if (tid == 0) ring.init();
  bool in[NV];
  int mine = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    in[v] = (v * (int)blockDim.x + tid) * N < a.C;
    mine += in[v] ? N : 0;
  }
  mine = __reduce_add_sync(0xFFFFFFFFu, mine);
  if (lane == 0) counts[warp] = make_float2((float)mine, mine ? 1.f / (float)mine : 0.f);
  __syncthreads();
  const float inv_n = counts[warp].y;
  const float lane_n = lane < warps ? counts[lane].x : 0.f, lane_inv_n = lane < warps ? counts[lane].y : 0.f;
  grid_dependency_wait();
  grid_launch_dependents();
  if (tid == 0)
    for (int s = 0; s < a.depth; ++s) {
      const long long m = blockIdx.x + (long long)s * gridDim.x;
      if (m < a.M) ring.fetch(s, m);
    }
  float w[NV][N], b[NV][N];
  long long group = -1;
  int stage = 0, turn = 0;
  uint32_t parity = 0;
  for (long long m = blockIdx.x; m < a.M; m += gridDim.x, turn ^= 1) {
    const long long g = (unsigned)m / (unsigned)a.rows_per_group;
    if (g != group) {
      group = g;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * (int)blockDim.x + tid) * N;
        if (in[v]) {
          norm_gain<WT, N>(a, g, c, w[v]);
          if (a.b) load_params<WT, N>(static_cast<const WT*>(a.b) + g * a.C + c, b[v]);
        }
        if (!a.b) {
#pragma unroll
          for (int i = 0; i < N; ++i) b[v][i] = 0.f;
        }
      }
    }
    ring.wait(stage, parity);
    float f[NV][N], sum = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const uint4 r = in[v] ? *reinterpret_cast<const uint4*>(ring.row(stage, 0) + (v * (int)blockDim.x + tid) * 16)
                            : make_uint4(0, 0, 0, 0);
      unpack_vec<T>(r, f[v]);
#pragma unroll
      for (int i = 0; i < N; ++i) sum += f[v][i];
    }
    sum = warp_sum(sum);
    const float own = sum * inv_n;
    float sq = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (in[v]) {
#pragma unroll
        for (int i = 0; i < N; ++i) sq = fmaf(f[v][i] - own, f[v][i] - own, sq);
      }
    sq = warp_sum(sq);
    if (lane == 0) slots[turn][warp] = make_float2(sum, sq);
    __syncthreads();
    if (tid == 0 && m + (long long)a.depth * gridDim.x < a.M) ring.fetch(stage, m + (long long)a.depth * gridDim.x);
    const float2 t = lane < warps ? slots[turn][lane] : make_float2(0.f, 0.f);
    const float mean = warp_sum(t.x) * inv_c;
    const float d = t.x * lane_inv_n - mean;
    const float rstd = 1.f / sqrtf(warp_sum(fmaf(lane_n * d, d, t.y)) * inv_c + a.eps);
    if (++stage == a.depth) {
      stage = 0;
      parity ^= 1u;
    }
    if (tid == 0) {
      if (a.mean) a.mean[m] = mean;
      if (a.rstd) a.rstd[m] = rstd;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < N; ++i) f[v][i] = fmaf((f[v][i] - mean) * rstd, w[v][i], b[v][i]);
    if constexpr (!QUANT) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (in[v]) Piece<T, true>::store(static_cast<T*>(a.y) + m * a.ldy + (v * (int)blockDim.x + tid) * N, f[v]);
    } else {
      float amax = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (in[v]) {
          if (a.inv_lambda) {
            float l[N];
            load_params<float, N>(a.inv_lambda + (v * (int)blockDim.x + tid) * N, l);
#pragma unroll
            for (int i = 0; i < N; ++i) f[v][i] *= l[i];
          }
#pragma unroll
          for (int i = 0; i < N; ++i) amax = max_nan(amax, fabsf(f[v][i]));
        }
      __shared__ float2 tops[2][32];
      const Int8Scale sc = int8_scale(team_max_nan(amax, warps, tops[turn]));
      if (tid == 0) a.s[m] = sc.s;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * (int)blockDim.x + tid) * N;
        if (in[v]) int8_store<N>(a.q + m * a.C + c, f[v], sc);
      }
    }
  }
}

// Backward. blockIdx.x = group * chunks + chunk; a block's teams (blockDim.y of
// them) take the chunk's rows in turn and add dy xhat and dy of their columns
// in registers; the block then adds its teams' sums in team order and writes
// one partial row of dw and db. Every order is fixed, so are the results.
template <typename T, typename WT, int NV, int MAXT, bool VEC>
__global__ void __launch_bounds__(MAXT, 1) layernorm_backward_kernel(const NormArgs a) {
  using P = Piece<T, VEC>;
  constexpr int N = P::kN;
  extern __shared__ float norm_smem[];      // [NV * N][blockDim.x]: the teams' sums, one team at a time
  __shared__ float2 slots[2][32];
  const int tid = threadIdx.x, team = threadIdx.y, teams = blockDim.y;
  const int warps = blockDim.x >> 5;
  const float inv_c = 1.f / (float)a.C;
  const long long g = blockIdx.x / a.chunks;
  const int chunk = (int)(blockIdx.x % a.chunks);
  const long long groups = gridDim.x / a.chunks;
  const long long row0 = g * a.rows_per_group;
  const long long rows = min(a.rows_per_group, a.M - row0);
  const bool sums = a.dw != nullptr || a.db != nullptr;
  float dw[NV][N], db[NV][N];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int i = 0; i < N; ++i) dw[v][i] = db[v][i] = 0.f;
  grid_dependency_wait();
  grid_launch_dependents();
  int turn = 0;
  // every team makes the same number of turns: the team's reduction has a barrier of the block
  for (long long k = (long long)chunk * teams; k < rows; k += (long long)a.chunks * teams, turn ^= 1) {
    const bool live = k + team < rows;
    const long long m = row0 + (live ? k + team : k);
    const T* x = static_cast<const T*>(a.x) + m * a.ldx;
    const T* dy = static_cast<const T*>(a.dy) + m * a.lddy;
    typename P::Raw rx[NV], ry[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * (int)blockDim.x + tid) * N;
      const bool in = live && c < a.C;
      rx[v] = in ? P::load(x + c) : P::zero();
      ry[v] = in ? P::load(dy + c) : P::zero();
    }
    const float mean = a.mean[m], rstd = a.rstd[m];
    // xhat and h of piece v, from its registers
    auto values = [&](int v, int c, float (&xh)[N], float (&dyv)[N], float (&h)[N]) {
      P::unpack(rx[v], xh);
      P::unpack(ry[v], dyv);
      norm_gain<WT, N>(a, g, c, h);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        xh[i] = (xh[i] - mean) * rstd;
        h[i] *= dyv[i];
      }
    };
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * (int)blockDim.x + tid) * N;
      if (live && c < a.C) {
        float xh[N], dyv[N], h[N];
        values(v, c, xh, dyv, h);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          dw[v][i] = fmaf(dyv[i], xh[i], dw[v][i]);
          db[v][i] += dyv[i];
          s1 += h[i];
          s2 = fmaf(h[i], xh[i], s2);
        }
      }
    }
    float2 s;
    if (teams == 1 || warps == 1) {
      s = team_sum2(s1, s2, warps, slots[turn]);
    } else {   // several teams of several warps: every warp leaves its sums, a team adds its own
      s1 = warp_sum(s1);
      s2 = warp_sum(s2);
      const int w = team * warps + (tid >> 5), lane = tid & 31;
      if (lane == 0) slots[turn][w] = make_float2(s1, s2);
      __syncthreads();
      const float2 t = lane < warps ? slots[turn][team * warps + lane] : make_float2(0.f, 0.f);
      s = make_float2(warp_sum(t.x), warp_sum(t.y));
    }
    const float m1 = s.x * inv_c, m2 = s.y * inv_c;
    if (live) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * (int)blockDim.x + tid) * N;
        if (c < a.C) {
          float xh[N], dyv[N], h[N];
          values(v, c, xh, dyv, h);
#pragma unroll
          for (int i = 0; i < N; ++i) h[i] = rstd * (h[i] - m1 - xh[i] * m2);
          P::store(static_cast<T*>(a.dx) + m * a.lddx + c, h);
        }
      }
    }
  }
  if (!sums) return;
  // the teams' sums, in team order, by way of shared memory
  for (int which = 0; which < 2; ++which) {
    for (int t = 1; t < teams; ++t) {
      __syncthreads();
      if (team == t) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int i = 0; i < N; ++i) norm_smem[(v * N + i) * blockDim.x + tid] = which ? db[v][i] : dw[v][i];
      }
      __syncthreads();
      if (team == 0) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int i = 0; i < N; ++i) (which ? db[v][i] : dw[v][i]) += norm_smem[(v * N + i) * blockDim.x + tid];
      }
    }
  }
  if (team != 0) return;
  const long long cols = groups * a.C;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * (int)blockDim.x + tid) * N;
    if (c >= a.C) continue;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (a.part) {
        a.part[(2ll * chunk) * cols + g * a.C + c + i] = dw[v][i];
        a.part[(2ll * chunk + 1) * cols + g * a.C + c + i] = db[v][i];
      } else {
        if (a.dw) a.dw[g * a.C + c + i] = dw[v][i];
        if (a.db) a.db[g * a.C + c + i] = db[v][i];
      }
    }
  }
}

// Backward for rows of more than one warp: as above with one team, the rows of
// x and dy streamed through the ring.
template <typename T, typename WT, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) layernorm_backward_rows_kernel(const NormArgs a) {
  constexpr int N = kVecN<T>, NV = kRowPieces<T>;
  extern __shared__ __align__(16) unsigned char norm_ring[];
  __shared__ float2 slots[2][32];
  __shared__ uint64_t full[kRingMaxStages];
  const int warps = blockDim.x >> 5, tid = threadIdx.x;
  const float inv_c = 1.f / (float)a.C;
  RowRing<2> ring = {norm_ring, full,
                     {static_cast<const unsigned char*>(a.x), static_cast<const unsigned char*>(a.dy)},
                     {a.ldx * (long long)sizeof(T), a.lddy * (long long)sizeof(T)},
                     (uint32_t)(a.C * (int)sizeof(T)), a.depth};
  if (tid == 0) ring.init();
  const long long g = blockIdx.x / a.chunks, groups = gridDim.x / a.chunks;
  const int chunk = (int)(blockIdx.x % a.chunks);
  const long long row0 = g * a.rows_per_group, rows = min(a.rows_per_group, a.M - row0);
  bool in[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) in[v] = (v * (int)blockDim.x + tid) * N < a.C;
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  if (tid == 0)
    for (int s = 0; s < a.depth; ++s) {
      const long long k = chunk + (long long)s * a.chunks;
      if (k < rows) ring.fetch(s, row0 + k);
    }
  float w[NV][N], dw[NV][N], db[NV][N];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (in[v]) norm_gain<WT, N>(a, g, (v * (int)blockDim.x + tid) * N, w[v]);
#pragma unroll
    for (int i = 0; i < N; ++i) dw[v][i] = db[v][i] = 0.f;
  }
  int stage = 0, turn = 0;
  uint32_t parity = 0;
  float mean = 0.f, rstd = 0.f;
  if (chunk < rows) {
    mean = a.mean[row0 + chunk];
    rstd = a.rstd[row0 + chunk];
  }
  for (long long k = chunk; k < rows; k += a.chunks, turn ^= 1) {
    // the next row's statistics, ahead of their use
    const long long next = min(k + a.chunks, rows - 1);
    const float mean1 = a.mean[row0 + next], rstd1 = a.rstd[row0 + next];
    ring.wait(stage, parity);
    float xh[NV][N], h[NV][N], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (in[v]) {
        unpack_vec<T>(*reinterpret_cast<const uint4*>(ring.row(stage, 0) + (v * (int)blockDim.x + tid) * 16), xh[v]);
        unpack_vec<T>(*reinterpret_cast<const uint4*>(ring.row(stage, 1) + (v * (int)blockDim.x + tid) * 16), h[v]);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          xh[v][i] = (xh[v][i] - mean) * rstd;
          dw[v][i] = fmaf(h[v][i], xh[v][i], dw[v][i]);
          db[v][i] += h[v][i];
          h[v][i] *= w[v][i];
          s1 += h[v][i];
          s2 = fmaf(h[v][i], xh[v][i], s2);
        }
      }
    }
    const float2 s = team_sum2(s1, s2, warps, slots[turn]);
    if (tid == 0 && k + (long long)a.depth * a.chunks < rows) ring.fetch(stage, row0 + k + (long long)a.depth * a.chunks);
    if (++stage == a.depth) {
      stage = 0;
      parity ^= 1u;
    }
    const float m1 = s.x * inv_c, m2 = s.y * inv_c;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (in[v]) {
#pragma unroll
        for (int i = 0; i < N; ++i) h[v][i] = rstd * (h[v][i] - m1 - xh[v][i] * m2);
        Piece<T, true>::store(static_cast<T*>(a.dx) + (row0 + k) * a.lddx + (v * (int)blockDim.x + tid) * N, h[v]);
      }
    mean = mean1;
    rstd = rstd1;
  }
  if (!a.dw && !a.db) return;
  const long long cols = groups * a.C;
  float* pw = a.part ? a.part + 2ll * chunk * cols : a.dw;
  float* pb = a.part ? a.part + (2ll * chunk + 1) * cols : a.db;
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if (in[v]) {
      const long long c = g * a.C + (v * (int)blockDim.x + tid) * N;
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        if (pw) *reinterpret_cast<float4*>(pw + c + i) = make_float4(dw[v][i], dw[v][i + 1], dw[v][i + 2], dw[v][i + 3]);
        if (pb) *reinterpret_cast<float4*>(pb + c + i) = make_float4(db[v][i], db[v][i + 1], db[v][i + 2], db[v][i + 3]);
      }
    }
}

// dw and db from the chunks' partial rows: a block takes 32 columns, its warp
// w adds the chunks w, w + 8, ... in order, then the eight sums in order.
__global__ void __launch_bounds__(256) layernorm_partials_kernel(const float* __restrict__ part,
                                                                 float* __restrict__ dw, float* __restrict__ db,
                                                                 long long cols, int chunks) {
  __shared__ float sums[8][33];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int which = blockIdx.y;
  const long long c = (long long)blockIdx.x * 32 + lane;
  grid_dependency_wait();
  grid_launch_dependents();
  float s = 0.f;
  if (c < cols)
    for (int k = w; k < chunks; k += 8) s += part[(2ll * k + which) * cols + c];
  sums[w][lane] = s;
  __syncthreads();
  float* out = which ? db : dw;
  if (w == 0 && c < cols && out) {
#pragma unroll
    for (int j = 1; j < 8; ++j) s += sums[j][lane];
    out[c] = s;
  }
}

}  // namespace svdq
