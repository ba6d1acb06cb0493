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
  int strip_blocks;      // few rows: blocks that sum columns, ahead of those that form dx
  int first_block;       // few rows: number of the launch's first block
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

// A team of blockDim.x threads takes a row at a time: some lanes of a warp or a
// warp (several teams in the block: blockDim.y) or the whole block. A thread
// holds NV pieces of the row.
template <typename T, typename WT, int NV, int MAXT, bool VEC, bool QUANT>
__global__ void __launch_bounds__(MAXT, 1) layernorm_kernel(const NormArgs a) {
  using P = Piece<T, VEC>;
  constexpr int N = P::kN;
  __shared__ float2 slots[3][32];
  const int tid = threadIdx.x;
  const float inv_c = 1.f / (float)a.C;
  grid_dependency_wait();
  grid_launch_dependents();
  const long long teams = (long long)gridDim.x * blockDim.y;
  // the lanes of a warp make the same number of turns, rows or not
  for (long long first = (long long)blockIdx.x * blockDim.y; first < a.M; first += teams) {
    const long long m = first + threadIdx.y;
    const bool live = m < a.M;
    const T* x = static_cast<const T*>(a.x) + m * a.ldx;
    typename P::Raw r[NV];
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * (int)blockDim.x + tid) * N;
      r[v] = live && c < a.C ? P::load(x + c) : P::zero();
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float f[N];
      P::unpack(r[v], f);
#pragma unroll
      for (int i = 0; i < N; ++i) sum += f[i];
    }
    const float mean = team_sum(sum, slots[0]) * inv_c;
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
    const float rstd = __frsqrt_rn(fmaf(team_sum(sq, slots[1]), inv_c, a.eps));
    if (live && tid == 0) {
      if (a.mean) a.mean[m] = mean;
      if (a.rstd) a.rstd[m] = rstd;
    }
    const long long g = (unsigned)(live ? m : first) / (unsigned)a.rows_per_group;
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
        if (live && c < a.C) {
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
        if (live && c < a.C) {
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
      const Int8Scale sc = int8_scale(team_max_nan(amax, slots[2]));
      if (live && tid == 0) a.s[m] = sc.s;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * (int)blockDim.x + tid) * N;
        if (live && c < a.C) int8_store<N>(a.q + m * a.C + c, q[v], sc);
      }
    }
  }
}

// Forward for rows off 16-byte boundaries, single values: NV of them a thread, a
// team of warps per row (blockDim.y teams), blockIdx.x = group * chunks + chunk.
// Bound: instructions, so weight and bias of the group stay in registers, addresses
// advance by a row's stride, columns are tested once, and the next row is loaded
// across the reductions. A warp takes the mean and the squares around it of its own
// columns; warps are joined behind one barrier as in the kernel below. bf16, one
// row a block without the next row's loads against this: 16384 x 1151 59 / 34.6 us,
// 40000 x 777 110 / 64, 16384 x 3001 138 / 95 (a ring with copies of the aligned span
// around each row: 55 at 1151). Rows loaded ahead of the weights: 38.7 -> 34.6.
template <typename T, typename WT, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > 256 ? 1 : 3) layernorm_values_kernel(const NormArgs a) {
  constexpr int W = MAXT / 32;
  __shared__ float2 slots[2][W];
  const int tid = threadIdx.x, team = threadIdx.y, teams = blockDim.y, lanes = blockDim.x;
  const int warps = lanes >> 5;
  const float inv_c = 1.f / (float)a.C;
  const long long g = blockIdx.x / a.chunks;
  const int chunk = (int)(blockIdx.x % a.chunks);
  const long long row0 = g * a.rows_per_group;
  const long long rows = min(a.rows_per_group, a.M - row0);
  const long long step = (long long)a.chunks * teams, first = (long long)chunk * teams;
  // columns of warp w
  auto columns = [&](int w) {
    int n = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v) n += min(max(a.C - v * lanes - 32 * w, 0), 32);
    return (float)n;
  };
  const float inv_n = 1.f / columns(tid >> 5);
  const int joined = tid & (W - 1);   // every W lanes join the team's warps
  const float joined_n = joined < warps ? columns(joined) : 0.f;
  bool in[NV];
  float gain[NV], bias[NV];
  grid_dependency_wait();
  grid_launch_dependents();
#pragma unroll
  for (int v = 0; v < NV; ++v) in[v] = v * lanes + tid < a.C;
  long long m = row0 + first + team;
  const T* x = static_cast<const T*>(a.x) + m * a.ldx + tid;
  T* y = static_cast<T*>(a.y) + m * a.ldy + tid;
  T r[NV];
  auto fetch = [&](bool live) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      r[v] = from_float<T>(0.f);
      if (live && in[v]) r[v] = x[v * lanes];
    }
  };
  bool live = first + team < rows;
  fetch(live);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = v * lanes + tid;
    float w[1] = {0.f}, b[1] = {0.f};
    if (in[v]) {
      norm_gain<WT, 1>(a, g, c, w);
      if (a.b) load_params<WT, 1>(static_cast<const WT*>(a.b) + g * a.C + c, b);
    }
    gain[v] = w[0];
    bias[v] = b[0];
  }
  int turn = 0;
  // every team makes the same number of turns: the reduction has a barrier of the block
  for (long long k = first; k < rows; k += step, turn ^= 1) {
    float f[NV], sum = 0.f, sq = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      f[v] = to_float(r[v]);
      sum += f[v];
    }
    const bool store = live;
    const long long row = m;
    live = k + step + team < rows;
    m += step;
    x += step * a.ldx;
    fetch(live);
    float mean = warp_sum(sum) * inv_n;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (in[v]) sq = fmaf(f[v] - mean, f[v] - mean, sq);
    sq = warp_sum(sq);
    if (warps > 1) {
      float2* slot = slots[turn] + team * warps;
      if ((tid & 31) == 0) slot[tid >> 5] = make_float2(mean, sq);
      __syncthreads();
      const float2 w = joined < warps ? slot[joined] : make_float2(0.f, 0.f);
      mean = w.x * joined_n;
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) mean += __shfl_xor_sync(0xFFFFFFFFu, mean, o);
      mean *= inv_c;
      sq = joined < warps ? fmaf((w.x - mean) * (w.x - mean), joined_n, w.y) : 0.f;
#pragma unroll
      for (int o = W / 2; o > 0; o >>= 1) sq += __shfl_xor_sync(0xFFFFFFFFu, sq, o);
    }
    const float rstd = __frsqrt_rn(fmaf(sq, inv_c, a.eps));
    if (store) {
      if (tid == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (in[v]) y[v * lanes] = from_float<T>(fmaf((f[v] - mean) * rstd, gain[v], bias[v]));
    }
    y += step * a.ldy;
  }
}

// Forward for rows of more than one warp, many of them: a block per row, rows
// streamed through the ring, weight and bias of the group in registers. Thread
// t holds the pieces t, t + blockDim.x, ... of a row, E elements: 32 of them
// where the row has enough, so that what a row costs a thread besides its
// elements (the wait, shuffles, the join) is shared by more. W: warps the block
// may have; the join runs over all of them, unrolled (absent ones hold zeros).
//
// Mean and variance take one barrier: each thread forms its own mean and its sum
// of squares around that, a warp joins its threads' and every thread joins the
// warps', each time by
//   M2 = sum_i (M2_i + n_i (mean_i - mean)^2).
// FULL: the row fills every piece of every thread. 9216 x 4096 bf16 26 us (5.8 TB/s;
// one row per block, no ring 54), 65536 x 1024 46 us.
template <typename T, typename WT, int E, int W, bool QUANT, bool FULL>
__global__ void __launch_bounds__(32 * W, 16 / W) layernorm_rows_kernel(const NormArgs a) {
  constexpr int N = kVecN<T>, NV = E / N, H = N / 2;
  extern __shared__ __align__(16) unsigned char norm_ring[];
  __shared__ float4 moments[2][W];   // of each warp: sum, sum of squares around its own mean, values, mean
  __shared__ float tops[2][W];
  __shared__ uint64_t full[kRingMaxStages];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float inv_c = 1.f / (float)a.C;
  const int M = (int)a.M, step = (int)gridDim.x;
  const uint32_t row_bytes = (uint32_t)(a.C * (int)sizeof(T));
  RowRing<1> ring = {norm_ring, full, {static_cast<const unsigned char*>(a.x)}, {a.ldx * (long long)sizeof(T)},
                     row_bytes, a.depth};
  if (tid == 0) ring.init();
  if (tid < 2 * W) {
    (&moments[0][0])[tid] = make_float4(0.f, 0.f, 0.f, 0.f);
    (&tops[0][0])[tid] = 0.f;
  }
  bool in[NV];
  int mine = 0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    in[v] = FULL || (v * (int)blockDim.x + tid) * N < a.C;
    mine += in[v] ? N : 0;
  }
  const int warp_has = __reduce_add_sync(0xFFFFFFFFu, mine);
  const float own_n = (float)mine, inv_own = mine ? 1.f / (float)mine : 0.f;          // elements of this thread
  const float n = (float)warp_has, inv_n = warp_has ? 1.f / (float)warp_has : 0.f;   // and of this warp
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  if (tid == 0)
    for (int s = 0; s < a.depth; ++s) {
      const long long m = blockIdx.x + (long long)s * step;
      if (m < M) ring.fetch(s, m);
    }
  float2 w[NV][H], b[NV][H];
  const int ahead = a.depth * step;
  long long group_end = 0;                       // row at which the next group begins
  int stage = 0, turn = 0;
  uint32_t parity = 0;
  const unsigned char* piece = norm_ring + tid * 16;
  T* y = static_cast<T*>(a.y) + blockIdx.x * a.ldy + tid * N;
  for (int m = blockIdx.x; m < M; m += step, turn ^= 1) {
    if (m >= group_end) {
      const long long g = (unsigned)m / (unsigned)a.rows_per_group;
      group_end = (g + 1) * a.rows_per_group;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const long long c = g * a.C + (v * (int)blockDim.x + tid) * N;
#pragma unroll
        for (int i = 0; i < H; ++i) {
          w[v][i] = pair(1.f);
          b[v][i] = pair(0.f);
        }
        if (in[v] && a.w) {
          load_pairs<WT, N>(static_cast<const WT*>(a.w) + c, w[v]);
#pragma unroll
          for (int i = 0; i < H; ++i) w[v][i] = add2_rn(w[v][i], pair(a.add));
        }
        if (in[v] && a.b) load_pairs<WT, N>(static_cast<const WT*>(a.b) + c, b[v]);
      }
    }
    ring.wait(stage, parity);
    float2 f[NV][H], sum2 = pair(0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      uint4 r = make_uint4(0, 0, 0, 0);
      if (in[v]) r = *reinterpret_cast<const uint4*>(piece + v * (int)blockDim.x * 16);
      unpack_pairs<T>(r, f[v]);
#pragma unroll
      for (int i = 0; i < H; ++i) sum2 = add2_rn(sum2, f[v][i]);
    }
    // around the thread's own mean first: this sweep does not wait for a shuffle
    const float mine_sum = sum2.x + sum2.y, mine_mean = mine_sum * inv_own;
    float2 sq2 = pair(0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (in[v]) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
          const float2 d = add2_rn(f[v][i], pair(-mine_mean));
          sq2 = fma2_rn(d, d, sq2);
        }
      }
    const float sum = warp_sum(mine_sum);
    const float own = sum * inv_n;
    const float off = mine_mean - own;
    const float sq = warp_sum(fmaf(own_n * off, off, sq2.x + sq2.y));
    if (lane == 0) moments[turn][warp] = make_float4(sum, sq, n, own);
    __syncthreads();
    if (tid == 0 && m < M - ahead) ring.fetch(stage, m + ahead);
    piece += row_bytes;
    if (++stage == a.depth) {
      stage = 0;
      parity ^= 1u;
      piece = norm_ring + tid * 16;
    }
    float mean = 0.f, m2 = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) mean += moments[turn][i].x;
    mean *= inv_c;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float4 t = moments[turn][i];
      const float d = t.w - mean;
      m2 += fmaf(t.z * d, d, t.y);
    }
    const float rstd = __frsqrt_rn(fmaf(m2, inv_c, a.eps));
    if (tid == 0) {
      if (a.mean) a.mean[m] = mean;
      if (a.rstd) a.rstd[m] = rstd;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < H; ++i)
        f[v][i] = fma2_rn(mul2_rn(add2_rn(f[v][i], pair(-mean)), pair(rstd)), w[v][i], b[v][i]);
    if constexpr (!QUANT) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (in[v]) *reinterpret_cast<uint4*>(y + v * (int)blockDim.x * N) = pack_pairs<T>(f[v]);
      y += step * a.ldy;
    } else {
      float amax = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (in[v]) {
          if (a.inv_lambda) {
            float2 l[H];
            load_pairs<float, N>(a.inv_lambda + (v * (int)blockDim.x + tid) * N, l);
#pragma unroll
            for (int i = 0; i < H; ++i) f[v][i] = mul2_rn(f[v][i], l[i]);
          }
#pragma unroll
          for (int i = 0; i < H; ++i) amax = amax3_nan(amax, f[v][i].x, f[v][i].y);
        }
      amax = warp_amax_nan(amax);
      if (lane == 0) tops[turn][warp] = amax;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < W; ++i) amax = max_nan(amax, tops[turn][i]);
      const Int8Scale sc = int8_scale(amax);
      if (tid == 0) a.s[m] = sc.s;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (in[v]) int8_store<N>(a.q + (long long)m * a.C + (v * (int)blockDim.x + tid) * N, f[v], sc);
    }
  }
  if (tid == 0) ring.leave();
}

// The sums of a block's teams, piece v of thread t at column (v blockDim.x + t) N,
// added in team order by way of shared memory ([teams][C]) into row g of out.
template <int NV, int N>
__device__ __forceinline__ void join_teams(const float (&sum)[NV][N], float* smem, float* out, long long g, int C) {
  const int tid = threadIdx.x, team = threadIdx.y, teams = blockDim.y;
  const int threads = blockDim.x * blockDim.y, thread = team * blockDim.x + tid;
  __syncthreads();
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * (int)blockDim.x + tid) * N;
    if (c < C) {
#pragma unroll
      for (int i = 0; i < N; ++i) smem[team * C + c + i] = sum[v][i];
    }
  }
  __syncthreads();
  if (out)
    for (int c = thread; c < C; c += threads) {
      float t = smem[c];
      for (int k = 1; k < teams; ++k) t += smem[k * C + c];
      out[g * C + c] = t;
    }
}

// Backward. blockIdx.x = group * chunks + chunk; a block's teams (blockDim.y of
// them) take the chunk's rows in turn and add dy xhat and dy of their columns
// in registers; the block then adds its teams' sums in team order and writes
// one partial row of dw and db. Every order is fixed, so are the results.
//
// Rows of up to 512 channels in 16-byte pieces: a team is some lanes of a warp.
template <typename T, typename WT, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) layernorm_backward_kernel(const NormArgs a) {
  using P = Piece<T, true>;
  constexpr int N = P::kN;
  extern __shared__ float norm_smem[];      // [teams][C]: the teams' sums
  const int tid = threadIdx.x, team = threadIdx.y, teams = blockDim.y;
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
  // every team makes the same number of turns: its lanes' shuffles take the whole warp
  for (long long k = (long long)chunk * teams; k < rows; k += (long long)a.chunks * teams) {
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
    const float m1 = lanes_sum(s1) * inv_c, m2 = lanes_sum(s2) * inv_c;
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
  float* const out[2] = {a.part ? a.part + 2ll * chunk * groups * a.C : a.dw,
                         a.part ? a.part + (2ll * chunk + 1) * groups * a.C : a.db};
#pragma unroll
  for (int which = 0; which < 2; ++which)
    join_teams<NV, N>(which ? db : dw, norm_smem, out[which], g, a.C);
}

// The same for rows off 16-byte boundaries, single values: NV of them a thread, a
// team of warps per row. Bound: instructions, so addresses advance by a row's
// stride, columns are tested once, xhat and h stay in registers between the
// row's sums and its dx, and the next row is loaded across the sums' reduction.
// bf16, without these against with them: 16384 x 1151 118 / 57.6 us, 40000 x 777
// 246 / 91, 17060 x 434 57.6 / 25.5.
template <typename T, typename WT, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, 512 / MAXT) layernorm_backward_values_kernel(const NormArgs a) {
  extern __shared__ float norm_smem[];      // [teams][C]: the teams' sums
  __shared__ float2 slots[2][MAXT / 32];
  const int tid = threadIdx.x, team = threadIdx.y, teams = blockDim.y, lanes = blockDim.x;
  const int warps = lanes >> 5, lane = tid & 31;
  const float inv_c = 1.f / (float)a.C;
  const long long g = blockIdx.x / a.chunks;
  const int chunk = (int)(blockIdx.x % a.chunks);
  const long long groups = gridDim.x / a.chunks;
  const long long row0 = g * a.rows_per_group;
  const long long rows = min(a.rows_per_group, a.M - row0);
  const long long step = (long long)a.chunks * teams, first = (long long)chunk * teams;
  bool in[NV];
  float gain[NV], dw[NV][1], db[NV][1];
  grid_dependency_wait();
  grid_launch_dependents();
#pragma unroll
  for (int v = 0; v < NV; ++v) in[v] = v * lanes + tid < a.C;
  // the team's row and its statistics; rows behind the group's last read as zeros
  long long m = row0 + first + team;
  const T* x = static_cast<const T*>(a.x) + m * a.ldx + tid;
  const T* dy = static_cast<const T*>(a.dy) + m * a.lddy + tid;
  T* dx = static_cast<T*>(a.dx) + m * a.lddx + tid;
  T rx[NV], ry[NV];
  float mean, rstd;
  auto fetch = [&](bool live) {
    mean = live ? a.mean[m] : 0.f;
    rstd = live ? a.rstd[m] : 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      rx[v] = ry[v] = from_float<T>(0.f);
      if (live && in[v]) {
        rx[v] = x[v * lanes];
        ry[v] = dy[v * lanes];
      }
    }
  };
  bool live = first + team < rows;
  fetch(live);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = v * lanes + tid;
    float w[1] = {0.f};
    if (in[v]) norm_gain<WT, 1>(a, g, c, w);
    gain[v] = w[0];
    dw[v][0] = db[v][0] = 0.f;
  }
  int turn = 0;
  // every team makes the same number of turns: the reduction has a barrier of the block
  for (long long k = first; k < rows; k += step, turn ^= 1) {
    float xh[NV], h[NV], s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const float d = to_float(ry[v]);
      xh[v] = in[v] ? (to_float(rx[v]) - mean) * rstd : 0.f;
      h[v] = gain[v] * d;
      dw[v][0] = fmaf(d, xh[v], dw[v][0]);
      db[v][0] += d;
      s1 += h[v];
      s2 = fmaf(h[v], xh[v], s2);
    }
    const float row_rstd = rstd;
    const bool store = live;
    live = k + step + team < rows;
    m += step;
    x += step * a.ldx;
    dy += step * a.lddy;
    fetch(live);
    // both sums at once: the lower lanes reduce s1, the upper ones s2
    float t = lane < 16 ? s1 : s2;
    t += __shfl_xor_sync(0xFFFFFFFFu, lane < 16 ? s2 : s1, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    float m1, m2;
    if (warps == 1) {
      m1 = __shfl_sync(0xFFFFFFFFu, t, 0);
      m2 = __shfl_sync(0xFFFFFFFFu, t, 16);
    } else {
      float2* slot = slots[turn] + team * warps;
      if ((lane & 15) == 0) reinterpret_cast<float*>(slot + (tid >> 5))[lane >> 4] = t;
      __syncthreads();
      m1 = m2 = 0.f;
      for (int i = 0; i < warps; ++i) {
        const float2 w = slot[i];
        m1 += w.x;
        m2 += w.y;
      }
    }
    m1 *= inv_c;
    m2 *= inv_c;
    if (store) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (in[v]) dx[v * lanes] = from_float<T>(row_rstd * (h[v] - m1 - xh[v] * m2));
    }
    dx += step * a.lddx;
  }
  if (!a.dw && !a.db) return;
  float* const out[2] = {a.part ? a.part + 2ll * chunk * groups * a.C : a.dw,
                         a.part ? a.part + (2ll * chunk + 1) * groups * a.C : a.db};
#pragma unroll
  for (int which = 0; which < 2; ++which)
    join_teams<NV, 1>(which ? db : dw, norm_smem, out[which], g, a.C);
}

// Backward for rows of more than one warp: a block per chunk of a group's rows,
// rows of x and dy streamed through the ring, the chunk's dw and db in
// registers (2 E of them). The weight is in registers too where two blocks of 8
// warps fit beside each other with it, else in shared memory (each thread its own
// columns, read back once a row). HOLD: xhat and h stay in registers between the row's
// two sweeps; else (E = 32, rows of more than 8192) the second sweep forms them
// again from the stage, which then waits for one more barrier. FULL as above.
// With the join of the chunks: 9216 x 4096 bf16 42.6 us (5.3 TB/s), 32760 x 5120
// 153 us (6.6 TB/s).
template <typename T, typename WT, int E, int W, int BLOCKS, bool HOLD, bool FULL>
__global__ void __launch_bounds__(32 * W, BLOCKS) layernorm_backward_rows_kernel(const NormArgs a) {
  constexpr int N = kVecN<T>, NV = E / N, H = N / 2;
  extern __shared__ __align__(16) unsigned char norm_ring[];
  __shared__ __align__(16) float2 slots[2][W];
  __shared__ uint64_t full[kRingMaxStages];
  const int tid = threadIdx.x, lane = tid & 31;
  const float inv_c = 1.f / (float)a.C;
  const uint32_t row_bytes = (uint32_t)(a.C * (int)sizeof(T));
  RowRing<2> ring = {norm_ring, full,
                     {static_cast<const unsigned char*>(a.x), static_cast<const unsigned char*>(a.dy)},
                     {a.ldx * (long long)sizeof(T), a.lddy * (long long)sizeof(T)}, row_bytes, a.depth};
  constexpr bool kGainRegs = HOLD && W <= 8;
  float* gain = reinterpret_cast<float*>(norm_ring + 2 * (size_t)a.depth * row_bytes);   // [C]
  float2 gr[kGainRegs ? NV : 1][H];
  if (tid == 0) ring.init();
  if (tid < 2 * W) (&slots[0][0])[tid] = pair(0.f);
  const long long g = blockIdx.x / a.chunks, groups = gridDim.x / a.chunks;
  const int chunk = (int)(blockIdx.x % a.chunks);
  const long long row0 = g * a.rows_per_group;
  const int rows = (int)min(a.rows_per_group, a.M - row0), ahead = a.depth * a.chunks;
  bool in[NV];
  float2 dw[NV][H], db[NV][H];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    in[v] = FULL || (v * (int)blockDim.x + tid) * N < a.C;
#pragma unroll
    for (int i = 0; i < H; ++i) dw[v][i] = db[v][i] = pair(0.f);
  }
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  if (tid == 0)
    for (int s = 0; s < a.depth; ++s) {
      const int k = chunk + s * a.chunks;
      if (k < rows) ring.fetch(s, row0 + k);
    }
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if (in[v]) {
      const int c = (v * (int)blockDim.x + tid) * N;
      float w[N];
      norm_gain<WT, N>(a, g, c, w);
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        if constexpr (kGainRegs) {
          gr[v][i / 2] = make_float2(w[i], w[i + 1]);
          gr[v][i / 2 + 1] = make_float2(w[i + 2], w[i + 3]);
        } else {
          *reinterpret_cast<float4*>(gain + c + i) = make_float4(w[i], w[i + 1], w[i + 2], w[i + 3]);
        }
      }
    }
  int stage = 0, turn = 0;
  uint32_t parity = 0;
  float mean = 0.f, rstd = 0.f;
  if (chunk < rows) {
    mean = a.mean[row0 + chunk];
    rstd = a.rstd[row0 + chunk];
  }
  const unsigned char* at_x = norm_ring + tid * 16;
  T* dx = static_cast<T*>(a.dx) + (row0 + chunk) * a.lddx + tid * N;
  const long long dx_step = a.chunks * a.lddx;
  const float* stat_mean = a.mean + row0;
  const float* stat_rstd = a.rstd + row0;
  for (int k = chunk; k < rows; k += a.chunks, turn ^= 1) {
    // the next row's statistics, ahead of their use
    const int next = min(k + a.chunks, rows - 1);
    const float mean1 = stat_mean[next], rstd1 = stat_rstd[next];
    ring.wait(stage, parity);
    // xhat, dy and h = dy w of piece v
    auto piece = [&](int v, float2 (&xh)[H], float2 (&dy)[H], float2 (&h)[H]) {
      const unsigned char* at = at_x + v * (int)blockDim.x * 16;
      unpack_pairs<T>(*reinterpret_cast<const uint4*>(at), xh);
      unpack_pairs<T>(*reinterpret_cast<const uint4*>(at + row_bytes), dy);
#pragma unroll
      for (int i = 0; i < H; i += 2) {
        if constexpr (kGainRegs) {
          h[i] = mul2_rn(dy[i], gr[v][i]);
          h[i + 1] = mul2_rn(dy[i + 1], gr[v][i + 1]);
        } else {
          const float4 w = *reinterpret_cast<const float4*>(gain + (v * (int)blockDim.x + tid) * N + 2 * i);
          h[i] = mul2_rn(dy[i], make_float2(w.x, w.y));
          h[i + 1] = mul2_rn(dy[i + 1], make_float2(w.z, w.w));
        }
      }
#pragma unroll
      for (int i = 0; i < H; ++i) xh[i] = mul2_rn(add2_rn(xh[i], pair(-mean)), pair(rstd));
    };
    float2 xh[HOLD ? NV : 1][H], h[HOLD ? NV : 1][H], s1 = pair(0.f), s2 = pair(0.f);
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (in[v]) {
        float2 dy[H];
        constexpr bool K = HOLD;
        float2(&x)[H] = xh[K ? v : 0], (&hh)[H] = h[K ? v : 0];
        piece(v, x, dy, hh);
#pragma unroll
        for (int i = 0; i < H; ++i) {
          dw[v][i] = fma2_rn(dy[i], x[i], dw[v][i]);
          db[v][i] = add2_rn(db[v][i], dy[i]);
          s1 = add2_rn(s1, hh[i]);
          s2 = fma2_rn(hh[i], x[i], s2);
        }
      }
    const float s = warp_sum_halves(s1.x + s1.y, s2.x + s2.y, lane);
    if ((lane & 15) == 0) reinterpret_cast<float*>(&slots[turn][tid >> 5])[lane >> 4] = s;
    __syncthreads();
    if (HOLD && tid == 0 && k + ahead < rows) ring.fetch(stage, row0 + k + ahead);
    float2 t = pair(0.f);
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      const float4 u = *reinterpret_cast<const float4*>(&slots[turn][i]);
      t = add2_rn(t, add2_rn(make_float2(u.x, u.y), make_float2(u.z, u.w)));
    }
    // dx = rstd h - rstd m1 - xhat rstd m2
    const float2 r1 = pair(-rstd * (t.x * inv_c)), r2 = pair(-rstd * (t.y * inv_c));
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (in[v]) {
        constexpr bool K = HOLD;
        float2(&x)[H] = xh[K ? v : 0], (&hh)[H] = h[K ? v : 0];
        if constexpr (!HOLD) {
          float2 dy[H];
          piece(v, x, dy, hh);
        }
#pragma unroll
        for (int i = 0; i < H; ++i) hh[i] = fma2_rn(x[i], r2, fma2_rn(hh[i], pair(rstd), r1));
        *reinterpret_cast<uint4*>(dx + v * (int)blockDim.x * N) = pack_pairs<T>(hh);
      }
    if (!HOLD) {
      __syncthreads();
      if (tid == 0 && k + ahead < rows) ring.fetch(stage, row0 + k + ahead);
    }
    dx += dx_step;
    at_x += 2 * row_bytes;
    if (++stage == a.depth) {
      stage = 0;
      parity ^= 1u;
      at_x = norm_ring + tid * 16;
    }
    mean = mean1;
    rstd = rstd1;
  }
  if (tid == 0) ring.leave();
  if (!a.dw && !a.db) return;
  const long long cols = groups * a.C;
  float* pw = a.part ? a.part + 2ll * chunk * cols : a.dw;
  float* pb = a.part ? a.part + (2ll * chunk + 1) * cols : a.db;
#pragma unroll
  for (int v = 0; v < NV; ++v)
    if (in[v]) {
      const long long c = g * a.C + (v * (int)blockDim.x + tid) * N;
#pragma unroll
      for (int i = 0; i < H; i += 2) {
        if (pw) *reinterpret_cast<float4*>(pw + c + 2 * i) = make_float4(dw[v][i].x, dw[v][i].y, dw[v][i + 1].x, dw[v][i + 1].y);
        if (pb) *reinterpret_cast<float4*>(pb + c + 2 * i) = make_float4(db[v][i].x, db[v][i].y, db[v][i + 1].x, db[v][i + 1].y);
      }
    }
}

// Backward for few rows, in one launch: dw and db need no reduction over a row
// (the statistics are given), so the first strip_blocks blocks each sum a strip
// of 32 columns over a group's rows, a warp every 16th row, while the others form
// dx. Both read x and dy, from L2 the second time, which is what few rows cost;
// nothing is kept in between. A row's dx takes a warp up to 1024 channels, else
// the block. 226 x 1151 fp32 4.7 us (with partial sums 9.3).
constexpr int kNormFewThreads = 512;

template <typename T, typename WT, bool VEC>
__global__ void __launch_bounds__(kNormFewThreads) layernorm_backward_few_kernel(const NormArgs a) {
  using P = Piece<T, VEC>;
  constexpr int N = P::kN, kWarps = kNormFewThreads / 32;
  __shared__ float sums[2][kWarps][33];
  __shared__ float2 slot[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int block = (int)blockIdx.x + a.first_block;
  grid_dependency_wait();
  grid_launch_dependents();
  if (block < a.strip_blocks) {
    const int strips = (a.C + 31) / 32;
    const long long g = block / strips;
    const int c = (block % strips) * 32 + lane;
    const long long row0 = g * a.rows_per_group;
    const int rows = (int)min(a.rows_per_group, a.M - row0);
    float w = 0.f, b = 0.f;
    if (c < a.C) {
      const T* x = static_cast<const T*>(a.x) + row0 * a.ldx + c;
      const T* dy = static_cast<const T*>(a.dy) + row0 * a.lddy + c;
#pragma unroll 8
      for (int r = warp; r < rows; r += kWarps) {
        const float d = to_float(dy[r * a.lddy]);
        w = fmaf(d, (to_float(x[r * a.ldx]) - a.mean[row0 + r]) * a.rstd[row0 + r], w);
        b += d;
      }
    }
    sums[0][warp][lane] = w;
    sums[1][warp][lane] = b;
    __syncthreads();
    if (warp < 2 && c < a.C) {
      float t = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) t += sums[warp][k][lane];
      float* out = warp ? a.db : a.dw;
      if (out) out[g * a.C + c] = t;
    }
    return;
  }
  const bool narrow = a.C <= 1024;
  const int tid = narrow ? lane : (int)threadIdx.x, team = narrow ? 32 : kNormFewThreads;
  const long long m = narrow ? (long long)(block - a.strip_blocks) * kWarps + warp : block - a.strip_blocks;
  if (m >= a.M) return;                       // a warp of its own, or no block at all
  const long long g = m / a.rows_per_group;
  const T* x = static_cast<const T*>(a.x) + m * a.ldx;
  const T* dy = static_cast<const T*>(a.dy) + m * a.lddy;
  const float mean = a.mean[m], rstd = a.rstd[m];
  auto piece = [&](int c, float (&xh)[N], float (&h)[N]) {
    float w[N];
    P::unpack(P::load(x + c), xh);
    P::unpack(P::load(dy + c), h);
    norm_gain<WT, N>(a, g, c, w);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      xh[i] = (xh[i] - mean) * rstd;
      h[i] *= w[i];
    }
  };
  float s1 = 0.f, s2 = 0.f;
#pragma unroll 4
  for (int c = tid * N; c < a.C; c += team * N) {
    float xh[N], h[N];
    piece(c, xh, h);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s1 += h[i];
      s2 = fmaf(h[i], xh[i], s2);
    }
  }
  float2 s = make_float2(warp_sum(s1), warp_sum(s2));
  if (!narrow) {
    if (lane == 0) slot[warp] = s;
    __syncthreads();
    s = lane < kWarps ? slot[lane] : make_float2(0.f, 0.f);
    s = make_float2(warp_sum(s.x), warp_sum(s.y));
  }
  const float m1 = s.x / (float)a.C, m2 = s.y / (float)a.C;
  T* dx = static_cast<T*>(a.dx) + m * a.lddx;
#pragma unroll 4
  for (int c = tid * N; c < a.C; c += team * N) {
    float xh[N], h[N];
    piece(c, xh, h);
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = rstd * (h[i] - m1 - xh[i] * m2);
    P::store(dx + c, h);
  }
}

// dw and db from the chunks' partial rows: a block takes 32 columns, its warp
// w adds the chunks w, w + 16, ... in order, then the warps' sums in order.
constexpr int kPartWarps = 16;

__global__ void __launch_bounds__(32 * kPartWarps) layernorm_partials_kernel(const float* part, float* dw, float* db,
                                                                             long long cols, int chunks) {
  __shared__ float sums[kPartWarps][33];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int which = blockIdx.y;
  const long long c = (long long)blockIdx.x * 32 + lane;
  grid_dependency_wait();
  grid_launch_dependents();
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int k = w; k < chunks; k += kPartWarps) s += part[(2ll * k + which) * cols + c];
  }
  sums[w][lane] = s;
  __syncthreads();
  float* out = which ? db : dw;
  if (w == 0 && c < cols && out) {
#pragma unroll
    for (int j = 1; j < kPartWarps; ++j) s += sums[j][lane];
    out[c] = s;
  }
}

}  // namespace svdq
