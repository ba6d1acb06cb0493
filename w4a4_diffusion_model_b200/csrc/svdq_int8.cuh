// The W8A8 linear layer: 8-bit integer codes with one scale per token of X and
// one per output channel of W,
//   Y[m][n] = sx[m] sw[n] sum_k qx[m][k] qw[n][k] + bias[n].
// The integer sum runs on the tensor cores (tcgen05 kind::i8, int32
// accumulators in tensor memory), so it is exact: |sum| <= 127^2 K < 2^31 for
// K <= 131072 (128 * 127 K too; 128^2 K is 2^31 at K = 131072). The epilogue rounds the sum to fp32, multiplies by sw and then by
// sx (in this order: a token's scale may lie anywhere in fp32's range, and the
// sum times it, or the product of the scales, could leave that range where Y
// does not), adds the bias in fp32 and rounds once to Y's type.
#pragma once

#include "svdq_int8_codec.cuh"
#include "svdq_ptx.cuh"
#include "svdq_rows.cuh"
#include "svdq_vec.cuh"

namespace svdq {

// ---------------------------------------------------------------- quantizer
struct Int8QuantArgs {
  const void* x;
  long long ldx;
  const float* mult;    // [K] or null: v = fp32(x * mult)
  int8_t* q;            // [M][K]
  float* s;             // [M]
  long long M;
  int K;
  int depth;            // stages of the row ring
};

template <typename T>
__device__ __forceinline__ void int8_values(const Int8QuantArgs& a, const uint4& r, int k, float (&f)[kVecN<T>]) {
  unpack_vec<T>(r, f);
  if (a.mult) {
    float l[kVecN<T>];
    load_params<float, kVecN<T>>(a.mult + k, l);
#pragma unroll
    for (int i = 0; i < kVecN<T>; ++i) f[i] *= l[i];
  }
}

// A team of blockDim.x threads (lanes of a warp, or the whole block) takes a row
// at a time and holds it in registers, NV vectors a thread: one read of X, one
// write of the codes, which is the bound (HBM). NV = 0: the row does not fit;
// it is read once for its maximum and once more, from L2, for its codes.
template <typename T, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) int8_quantize_kernel(const Int8QuantArgs a) {
  constexpr int N = kVecN<T>;
  constexpr int R = NV ? NV : 1;
  __shared__ float2 slots[2][32];
  const int tid = threadIdx.x;
  const int step = (int)blockDim.x * N;
  grid_dependency_wait();
  grid_launch_dependents();
  const long long teams = (long long)gridDim.x * blockDim.y;
  int turn = 0;
  // the lanes of a warp make the same number of turns, rows or not
  for (long long first = (long long)blockIdx.x * blockDim.y; first < a.M; first += teams, turn ^= 1) {
    const long long m = first + threadIdx.y;
    const int K = m < a.M ? a.K : 0;
    const T* x = static_cast<const T*>(a.x) + m * a.ldx;
    uint4 r[R];
    float amax = 0.f;
    auto look = [&](const uint4& v, int k) {
      float f[N];
      int8_values<T>(a, v, k, f);
#pragma unroll
      for (int i = 0; i < N; ++i) amax = max_nan(amax, fabsf(f[i]));
    };
    if constexpr (NV > 0) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int k = v * step + tid * N;
        r[v] = k < K ? load_once(x + k) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int k = v * step + tid * N;
        if (k < K) look(r[v], k);
      }
    } else {
      for (int k = tid * N; k < K; k += step) look(*reinterpret_cast<const uint4*>(x + k), k);
    }
    const Int8Scale sc = int8_scale(team_max_nan(amax, slots[turn]));
    if (tid == 0 && K > 0) a.s[m] = sc.s;
    int8_t* q = a.q + m * a.K;
    if constexpr (NV > 0) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int k = v * step + tid * N;
        if (k < K) {
          float f[N];
          int8_values<T>(a, r[v], k, f);
          int8_store<N>(q + k, f, sc);
        }
      }
    } else {
      for (int k = tid * N; k < K; k += step) {
        float f[N];
        int8_values<T>(a, *reinterpret_cast<const uint4*>(x + k), k, f);
        int8_store<N>(q + k, f, sc);
      }
    }
  }
}

// Many rows of more than one warp: a block per row, rows streamed through the
// ring, the factors in registers, E elements a thread; FULL: K fills them all.
// Bound: HBM, with the instructions of the codes close behind. 4608 x 4096 bf16
// smoothed 12 us (4.7 TB/s), 9001 x 13824 67 us (5.6 TB/s, 0.87 of a copy).
template <typename T, int E, int W, bool FULL>
__global__ void __launch_bounds__(32 * W, 16 / W) int8_quantize_rows_kernel(const Int8QuantArgs a) {
  constexpr int N = kVecN<T>, NV = E / N, H = N / 2;
  extern __shared__ __align__(16) unsigned char quant_ring[];
  __shared__ float tops[2][W];
  __shared__ uint64_t full[kRingMaxStages];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int M = (int)a.M, step = (int)gridDim.x, ahead = a.depth * step;
  const uint32_t row_bytes = (uint32_t)(a.K * (int)sizeof(T));
  RowRing<1> ring = {quant_ring, full, {static_cast<const unsigned char*>(a.x)}, {a.ldx * (long long)sizeof(T)},
                     row_bytes, a.depth};
  if (tid == 0) ring.init();
  if (tid < 2 * W) (&tops[0][0])[tid] = 0.f;
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  if (tid == 0)
    for (int s = 0; s < a.depth; ++s) {
      const long long m = blockIdx.x + (long long)s * step;
      if (m < M) ring.fetch(s, m);
    }
  bool in[NV];
  float2 l[NV][H];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int k = (v * (int)blockDim.x + tid) * N;
    in[v] = FULL || k < a.K;
#pragma unroll
    for (int i = 0; i < H; ++i) l[v][i] = pair(1.f);
    if (a.mult && in[v]) load_pairs<float, N>(a.mult + k, l[v]);
  }
  int stage = 0, turn = 0;
  uint32_t parity = 0;
  const unsigned char* piece = quant_ring + tid * 16;
  int8_t* q = a.q + (long long)blockIdx.x * a.K + tid * N;
  const long long q_step = (long long)step * a.K;
  for (int m = blockIdx.x; m < M; m += step, turn ^= 1) {
    ring.wait(stage, parity);
    float2 f[NV][H];
    float amax = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (in[v]) {
        unpack_pairs<T>(*reinterpret_cast<const uint4*>(piece + v * (int)blockDim.x * 16), f[v]);
#pragma unroll
        for (int i = 0; i < H; ++i) {
          f[v][i] = mul2_rn(f[v][i], l[v][i]);
          amax = amax3_nan(amax, f[v][i].x, f[v][i].y);
        }
      }
    amax = warp_amax_nan(amax);
    if (lane == 0) tops[turn][warp] = amax;
    __syncthreads();
    if (tid == 0 && m < M - ahead) ring.fetch(stage, m + ahead);
    piece += row_bytes;
    if (++stage == a.depth) {
      stage = 0;
      parity ^= 1u;
      piece = quant_ring + tid * 16;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) amax = max_nan(amax, tops[turn][i]);
    const Int8Scale sc = int8_scale(amax);
    if (tid == 0) a.s[m] = sc.s;
#pragma unroll
    for (int v = 0; v < NV; ++v)
      if (in[v]) int8_store<N>(q + v * (int)blockDim.x * N, f[v], sc);
    q += q_step;
  }
  if (tid == 0) ring.leave();
}

// ---------------------------------------------------------------- tensor-core pieces
// D(tmem, int32) (+)= A(smem) * B(smem)^T, signed 8-bit integers.
__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor, kind::i8: signed 8-bit A/B (K-major), int32 accumulator.
__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4)                       // D format: s32
         | (1u << 7)                     // A format: s8
         | (1u << 10)                    // B format: s8
         | ((uint32_t)(N >> 3) << 17)    // N / 8
         | ((uint32_t)(M >> 4) << 24);   // M / 16
}

struct Int8GemmArgs {
  const float* sx;     // [M]
  const float* sw;     // [N]
  const float* bias;   // [N] or null
  void* y;
  long long ldy;
  int M, N, K;
  int a_rows;          // single-CTA kernel: rows of the A box (8..128)
};

// ---------------------------------------------------------------- few tokens
// Y for at most 8 tokens: every weight is read once and used M times, so the
// product is bound by HBM and the integer dot-product instruction (dp4a: four
// products per lane) keeps up. A warp holds a 512-byte slice of kGvChannels
// rows of W (16 bytes a lane, all loads in flight at once) and the same slice
// of each token; a block's warps take `warps_k` slices of the same channels in
// turn, or several channel groups where K is short. Sums are integers, so any
// order gives the same bits. 2 x 4096 x 24576: 19.7 us, 5.1 TB/s (the single-CTA
// kernel below takes 21.1 for 9 tokens).
constexpr int kGvThreads = 256;
constexpr int kGvChannels = 8;

template <int MT, typename OT>
__global__ void __launch_bounds__(kGvThreads) int8_few_tokens_kernel(const int8_t* qx, const int8_t* qw,
                                                                     const Int8GemmArgs a, int warps_k) {
  __shared__ int sums[kGvThreads / 32][kGvChannels * MT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / warps_k, wk = warp - group * warps_k;      // channel group, slice of K
  const int groups = (kGvThreads / 32) / warps_k;
  const int n0 = (blockIdx.x * groups + group) * kGvChannels;
  int acc[kGvChannels][MT];
#pragma unroll
  for (int c = 0; c < kGvChannels; ++c)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[c][m] = 0;
  const int8_t* w = qw + (long long)n0 * a.K;
  grid_dependency_wait();
  grid_launch_dependents();
  for (int k = wk * 512 + lane * 16; k < a.K; k += warps_k * 512) {
    uint4 r[kGvChannels];
#pragma unroll
    for (int c = 0; c < kGvChannels; ++c)
      r[c] = n0 + c < a.N ? load_once(w + (long long)c * a.K + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint4 x = m < a.M ? *reinterpret_cast<const uint4*>(qx + (long long)m * a.K + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < kGvChannels; ++c) {
        int t = acc[c][m];
        t = __dp4a((int)r[c].x, (int)x.x, t);
        t = __dp4a((int)r[c].y, (int)x.y, t);
        t = __dp4a((int)r[c].z, (int)x.z, t);
        acc[c][m] = __dp4a((int)r[c].w, (int)x.w, t);
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int c = 0; c < kGvChannels; ++c)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int t = __reduce_add_sync(0xFFFFFFFFu, acc[c][m]);
      if (lane == 0) sums[warp][m * kGvChannels + c] = t;
    }
  __syncthreads();
  for (int j = threadIdx.x; j < groups * kGvChannels * MT; j += kGvThreads) {
    const int i = j % (kGvChannels * MT), g = j / (kGvChannels * MT);
    const int m = i / kGvChannels, n = (blockIdx.x * groups + g) * kGvChannels + i % kGvChannels;
    if (m >= a.M || n >= a.N) continue;
    int t = 0;
    for (int k = 0; k < warps_k; ++k) t += sums[g * warps_k + k][i];
    static_cast<OT*>(a.y)[(long long)m * a.ldy + n] =
        from_float<OT>(fmaf((float)t * a.sw[n], a.sx[m], a.bias ? a.bias[n] : 0.f));
  }
}

// ---------------------------------------------------------------- single-CTA kernel
// One 128 x 256 output tile per CTA and K slice; a cluster of gridDim.z CTAs
// splits K when there are too few tiles for the GPU. The tile is that wide
// because 128 bytes of K cost a CTA 0.28 us whatever the tile (measured over whole
// kernels: 128 x 64, 128 x 128 and 256 x 256 alike, one accumulator or four), so
// narrow tiles only repeat it; what shortens a small product is a shorter K slice.
// For pairs of 256 x 256 that is the tensor peak. For the narrow tiles these times do
// not tell the MMA's own time from the latency of the loads behind a ring of four
// stages; nothing here rests on which of the two it is.
//
// Warp 0 loads (TMA, 128 bytes of K per stage), warp 1 issues the MMAs, then all
// eight warps take the accumulator out of tensor memory (warp w: lanes
// 32 (w % 4).., half of the columns) into shared memory (the ring's, idle by
// then). The CTAs of a cluster read each other's tiles there: CTA z adds and
// writes the columns [z, z + 1) 256 / gridDim.z. A lane keeps its columns and
// their scales from row to row. Rows past M are neither loaded (the A box is cut
// to a_rows) nor written, so few tokens cost little traffic. 16 x 4096 x 4096 in
// quarters of K 8.8 us (pairs 15), 64 x 4096 x 24576 whole 23 us (4.4 TB/s).
constexpr int kI8KTile = 128;                        // K elements (= bytes) per stage row
constexpr int kI8StageA = 128 * kI8KTile;            // 16 KB
constexpr int kI8Threads = 256;
constexpr int kI8Cols = 256;
constexpr int kI8StageBytes = kI8StageA + kI8Cols * kI8KTile;   // 48 KB
constexpr int kI8Stages = 4;
constexpr int kI8Ld = kI8Cols + 4;                   // int32 per row of the staged tile
static_assert(kI8Stages * kI8StageBytes >= 128 * kI8Ld * 4, "the tile is staged in the ring");
constexpr int kI8ScaleOffset = kI8Stages * kI8StageBytes;   // sx of the rows, then (sw, bias) of the columns
constexpr int kI8BarOffset = kI8ScaleOffset + 128 * 4 + kI8Cols * 8;
constexpr int kI8Bytes = kI8BarOffset + 128 + 1024;

// Sum over a cluster's CTAs of the int32 at the same shared address; `first` is
// this CTA's.
__device__ __forceinline__ int4 sum_cluster(int4 first, uint32_t addr, int z, int splits) {
  for (int p = 1; p < splits; ++p) {
    int4 u;
    asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "r"(mapa_shared(addr, (uint32_t)((z + p) % splits)))
                 : "memory");
    first.x += u.x;
    first.y += u.y;
    first.z += u.z;
    first.w += u.w;
  }
  return first;
}

template <typename OT>
__global__ void __launch_bounds__(kI8Threads, 1) svdq_int8_gemm_kernel(const __grid_constant__ CUtensorMap tm_x,
                                                                       const __grid_constant__ CUtensorMap tm_w,
                                                                       const Int8GemmArgs a) {
  extern __shared__ __align__(1024) unsigned char i8_smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(i8_smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kI8BarOffset);
  uint64_t* empty = full + kI8Stages;
  uint64_t* done = empty + kI8Stages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles_n = (a.N + kI8Cols - 1) / kI8Cols;
  const int n0 = (int)(blockIdx.x % tiles_n) * kI8Cols, m0 = (int)(blockIdx.x / tiles_n) * 128;
  const int splits = gridDim.z, z = blockIdx.z;
  const int kts = (a.K + kI8KTile - 1) / kI8KTile;
  const int kt0 = kts * z / splits, kt1 = kts * (z + 1) / splits;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kI8Stages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    mbar_init(done, 1);
    fence_mbar_init();
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kI8Cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0 && lane == 0) {
    const uint32_t bytes = (uint32_t)((a.a_rows + kI8Cols) * kI8KTile);
    int s = 0, kt = kt0;
    uint32_t ph = 1;
    for (; kt < kt1; ++kt) {
      if (!mbar_wait(empty + s, ph, kDevErrTimeoutEmpty)) break;
      unsigned char* sa = smem + s * kI8StageBytes;
      mbar_arrive_expect_tx(full + s, bytes);
      tma_load_2d(sa + kI8StageA, &tm_w, full + s, kt * kI8KTile, n0);
      tma_load_2d(sa, &tm_x, full + s, kt * kI8KTile, m0);
      if (++s == kI8Stages) {
        s = 0;
        ph ^= 1u;
      }
    }
    if (device_error_set()) {   // let the copies this thread issued land before the CTA exits
      const int it = kt - kt0;
      for (int j = it > kI8Stages ? it - kI8Stages : 0; j < it; ++j) mbar_drain(full + j % kI8Stages, (j / kI8Stages) & 1);
    }
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = idesc_i8(128, kI8Cols);
    int s = 0;
    uint32_t ph = 0;
    for (int kt = kt0; kt < kt1; ++kt) {
      if (!mbar_wait(full + s, ph, kDevErrTimeoutFull)) break;
      tc_fence_after();
      const uint64_t ad = smem_desc(smem_u32(smem + s * kI8StageBytes), 16, 1024, kSwizzle128B);
      const uint64_t bd = smem_desc(smem_u32(smem + s * kI8StageBytes + kI8StageA), 16, 1024, kSwizzle128B);
      const int steps = min(kI8KTile, a.K - kt * kI8KTile + 31) / 32;   // of 32 K elements (32 bytes)
#pragma unroll
      for (int j = 0; j < kI8KTile / 32; ++j)
        if (j < steps) mma_i8(tmem, ad + 2u * j, bd + 2u * j, idesc, kt > kt0 || j > 0 ? 1u : 0u);
      tc_commit(empty + s);
      if (++s == kI8Stages) {
        s = 0;
        ph ^= 1u;
      }
    }
    tc_commit(done);
  }
  float* sxs = reinterpret_cast<float*>(smem + kI8ScaleOffset);
  float2* cols_s = reinterpret_cast<float2*>(smem + kI8ScaleOffset + 128 * 4);
  if (warp >= 2) {   // the scales, while the product runs
    for (int i = threadIdx.x - 64; i < 128 + kI8Cols; i += kI8Threads - 64) {
      if (i < 128) {
        sxs[i] = m0 + i < a.M ? a.sx[m0 + i] : 0.f;
      } else {
        const int n = n0 + i - 128;
        cols_s[i - 128] = n < a.N ? make_float2(a.sw[n], a.bias ? a.bias[n] : 0.f) : make_float2(0.f, 0.f);
      }
    }
  }
  __syncwarp();
  // every MMA has read its stages: the ring is free for the tile
  const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(done, 0, kDevErrTimeoutAccum) && !device_error_set());
  tc_fence_after();
  const int q = warp & 3;
  if (ok && 32 * q < a.M - m0) {
    int* tile = reinterpret_cast<int*>(smem) + (32 * q + lane) * kI8Ld;
#pragma unroll
    for (int i = 0; i < kI8Cols / 2; i += 32) {
      const int c = (warp >> 2) * (kI8Cols / 2) + i;
      uint32_t v[32];
      tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * q) << 16) + c, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 32; j += 4)
        *reinterpret_cast<uint4*>(tile + c + j) = make_uint4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
  }
  tc_fence_before();
  if (splits > 1) cluster_sync();
  else __syncthreads();
  if (ok) {
    // A warp takes up to 128 of the CTA's columns, four a lane: neighbours where
    // Y's rows allow wide stores, else a quarter of the columns apart, so that a
    // warp's single stores are dense (the cluster's sums, read four at a time,
    // then pass through this CTA's own columns of its tile, which no peer reads).
    const int rows = min(128, a.M - m0), cols = min(128, kI8Cols / splits), per_row = cols / 4;
    const bool wide = (a.ldy & 3) == 0;
    const int place = lane % per_row, dc = wide ? 1 : per_row;
    const int rows_per_warp = 32 / per_row, row_step = (kI8Threads / 32) * rows_per_warp;
    const int row0 = warp * rows_per_warp + lane / per_row;
    const uint32_t base = smem_u32(smem);
    for (int part = 0; part < kI8Cols / splits; part += cols) {
      const int first = z * (kI8Cols / splits) + part;
      if (!wide && splits > 1) {
#pragma unroll 4
        for (int r = row0; r < rows; r += row_step) {
          const uint32_t at = (uint32_t)(r * kI8Ld + first + 4 * place) * 4;
          *reinterpret_cast<int4*>(smem + at) =
              sum_cluster(*reinterpret_cast<const int4*>(smem + at), base + at, z, splits);
        }
        __syncwarp();
      }
      const int c0 = first + (wide ? 4 * place : place);
      float sw[4], bias[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 sb = cols_s[c0 + i * dc];
        sw[i] = sb.x;
        bias[i] = sb.y;
      }
      OT* y = static_cast<OT*>(a.y) + (long long)m0 * a.ldy + n0 + c0;
#pragma unroll 4
      for (int r = row0; r < rows; r += row_step) {
        const uint32_t at = (uint32_t)(r * kI8Ld + c0) * 4;
        int t[4];
        if (wide) {
          const int4 v = sum_cluster(*reinterpret_cast<const int4*>(smem + at), base + at, z, splits);
          t[0] = v.x; t[1] = v.y; t[2] = v.z; t[3] = v.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] = *reinterpret_cast<const int*>(smem + at + 4 * i * dc);
        }
        const float sx = sxs[r];
        float f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = fmaf((float)t[i] * sw[i], sx, bias[i]);
        OT* p = y + (long long)r * a.ldy;
        if (wide && n0 + c0 + 4 <= a.N) {
          if constexpr (sizeof(OT) == 4) *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
          else *reinterpret_cast<uint2*>(p) = make_uint2(pack2(f[0], f[1], OT()), pack2(f[2], f[3], OT()));
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n0 + c0 + i * dc < a.N) p[i * dc] = from_float<OT>(f[i]);
        }
      }
    }
  }
  if (splits > 1) cluster_sync();   // no CTA leaves while a peer may read its tile
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kI8Cols);
  }
}

// ---------------------------------------------------------------- CTA-pair kernel
// Large products: one tcgen05 MMA (cta_group::2) spans the two SMs of a cluster
// of 2 and computes a 256 x 256 tile; each CTA stages its own 128 rows of X and its
// own 128 rows of W (two thirds of the bytes that a 128 x 256 tile would fetch
// per product). Persistent: cluster c takes tiles c, c + clusters, ...; two
// accumulators alternate, so a tile's epilogue runs under the next tile's MMAs.
// Roles per CTA (320 threads):
//   warps 0-7  epilogue: warp (q, h) takes accumulator lanes 32q.. and columns
//              128 h..: scales, bias, rounding, 128B-swizzled boxes, TMA stores
//   warp 8     producer: TMA loads of this CTA's rows, counted on the even
//              CTA's stage barrier (both CTAs' bytes)
//   warp 9     the even CTA's lane 0 issues the MMAs; a multicast commit frees
//              each stage, and hands over each accumulator, in both CTAs
// Tiles go in bands of kP8Band tile rows, column by column: the clusters that
// run at one time then share few rows of X and of W, and L2 serves the rest.
constexpr int kP8Threads = 320;
constexpr int kP8EpiWarps = 8;
constexpr int kP8Band = 8;
constexpr int kP8StageBytes = 2 * 128 * kI8KTile;            // 32 KB: 128 rows of X, 128 rows of W
constexpr int kP8Stages = 5;
constexpr int kP8BoxBytes = 4096;                            // 32 rows x 128 bytes
constexpr int kP8Cols = 128;                                 // accumulator columns per epilogue warp
constexpr int kP8BoxOffset = kP8Stages * kP8StageBytes;
constexpr int kP8ColOffset = kP8BoxOffset + kP8EpiWarps * kP8BoxBytes;   // (sw, bias) of each warp's columns
constexpr int kP8BarOffset = kP8ColOffset + kP8EpiWarps * kP8Cols * 8;
constexpr int kP8Bytes = kP8BarOffset + 256 + 1024;

__device__ __forceinline__ void mma_i8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// TMA load into this CTA's shared memory, counted on a barrier of the pair's
// even CTA (`bar`: its shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const void* tmap, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
      ::"r"(smem_u32(dst)), "l"(tmap), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

struct Int8Tile {
  int m0, n0;
};

__device__ __forceinline__ Int8Tile int8_pair_tile(int tile, int tiles_m, int tiles_n) {
  const int band = tile / (kP8Band * tiles_n);
  const int rows = min(kP8Band, tiles_m - band * kP8Band);
  const int i = tile - band * kP8Band * tiles_n;
  return Int8Tile{(band * kP8Band + i % rows) * 256, (i / rows) * 256};
}

// A warp's 32 x 128 band of the int32 tile (tensor memory at taddr, row m0 + lane)
// to Y: `add` (this lane's 128 int32 in shared memory, or null) is added first;
// `drained` is told once the last column has left tensor memory.
template <typename OT, typename F>
__device__ __forceinline__ void int8_store_band(uint32_t taddr, const int* add, float sx, const float2* colv,
                                                unsigned char* box, const CUtensorMap& tm_y, int tma_y,
                                                const Int8GemmArgs& a, int m0, int n0, int lane, F drained) {
  constexpr int kBoxCols = 128 / (int)sizeof(OT);
  const bool live = m0 < a.M;
#pragma unroll
  for (int b = 0; b < kP8Cols / kBoxCols; ++b) {
    if (tma_y && lane == 0) bulk_wait_read<0>();   // the previous store from this box has read it
    __syncwarp();
#pragma unroll
    for (int c = 0; c < kBoxCols; c += 32) {
      const int col = b * kBoxCols + c;
      uint32_t v[32];
      tmem_ld_32x32b_x32(taddr + col, v);
      tmem_ld_wait();
      if (col + 32 == kP8Cols) drained();
      if (add) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          const uint4 u = *reinterpret_cast<const uint4*>(add + col + i);
          v[i] += u.x;
          v[i + 1] += u.y;
          v[i + 2] += u.z;
          v[i + 3] += u.w;
        }
      }
      float f[32];
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float4 sb = *reinterpret_cast<const float4*>(colv + col + i);
        f[i] = fmaf((float)(int)v[i] * sb.x, sx, sb.y);
        f[i + 1] = fmaf((float)(int)v[i + 1] * sb.z, sx, sb.w);
      }
      // row `lane` of the box: 16-byte chunk j at (j ^ (lane & 7)), the 128B swizzle
      constexpr int kChunks = 32 * (int)sizeof(OT) / 16;
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        float g[kVecN<OT>];
#pragma unroll
        for (int i = 0; i < kVecN<OT>; ++i) g[i] = f[j * kVecN<OT> + i];
        const int chunk = c * (int)sizeof(OT) / 16 + j;
        *reinterpret_cast<uint4*>(box + lane * 128 + ((chunk ^ (lane & 7)) << 4)) = pack_vec<OT>(g);
      }
    }
    const int col0 = n0 + b * kBoxCols;
    if (tma_y) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && live && col0 < a.N) {
        tma_store_2d_evict_first(&tm_y, box, col0 * (int)sizeof(OT), m0);   // x in bytes
        bulk_commit();
      }
    } else {
      __syncwarp();
      const int rows = min(32, a.M - m0);
      OT* y = static_cast<OT*>(a.y) + (long long)m0 * a.ldy + col0;
#pragma unroll
      for (int c = 0; c < kBoxCols; c += 32) {
        const int e = c + lane, byte = e * (int)sizeof(OT);
        if (col0 + e < a.N) {
#pragma unroll 8
          for (int r = 0; r < rows; ++r)
            y[r * a.ldy + e] = *reinterpret_cast<const OT*>(box + r * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15));
        }
      }
      __syncwarp();
    }
  }
}

// tm_y views Y as bytes, in boxes of 32 rows x 128; tma_y = 0 where Y's rows or their
// stride are no whole 16-byte pieces (then the staged boxes are written by plain
// stores).
//
// SPLIT: a cluster of two pairs shares one tile, each pair half of K (few tiles and
// a long K: twice as many SMs work, half as long). Pair p finishes the columns
// 128 p..; for the other columns each CTA writes its int32 sums into the shared
// memory of the CTA with the same rows in the other pair (the ring's, idle by
// then), which adds them to its own.
constexpr int kP8PartLd = kP8Cols + 4;   // int32 per row of the received half: rows 4 banks apart
static_assert(kP8Stages * kP8StageBytes >= 128 * kP8PartLd * 4, "the half tile is received in the ring");

template <typename OT, bool SPLIT>
__global__ void __launch_bounds__(kP8Threads, 1) svdq_int8_gemm_pair_kernel(const __grid_constant__ CUtensorMap tm_x,
                                                                            const __grid_constant__ CUtensorMap tm_w,
                                                                            const __grid_constant__ CUtensorMap tm_y,
                                                                            const Int8GemmArgs a, int tma_y) {
  extern __shared__ __align__(1024) unsigned char p8_smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(p8_smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kP8BarOffset);   // even CTA: both CTAs' loads
  uint64_t* empty = full + kP8Stages;
  uint64_t* acc_full = empty + kP8Stages;    // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2], even CTA: both CTAs' epilogue warps
  uint64_t* mma_drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank(), crank = rank & 1u, even = rank & ~1u;   // CTA of the pair, its even CTA
  const int part = SPLIT ? (int)(rank >> 1) : 0;
  constexpr int kCtas = SPLIT ? 4 : 2;
  const int cluster = blockIdx.x / kCtas, nclusters = gridDim.x / kCtas;
  const int tiles_m = (a.M + 255) / 256, tiles_n = (a.N + 255) / 256;
  const int ntiles = tiles_m * tiles_n;
  const int kts = (a.K + kI8KTile - 1) / kI8KTile;
  const int kt0 = SPLIT ? kts * part / 2 : 0, kt1 = SPLIT ? kts * (part + 1) / 2 : kts;
  const uint16_t both = (uint16_t)(3u << even);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kP8Stages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + b, 1);
      mbar_init(acc_empty + b, 2 * kP8EpiWarps);
    }
    mbar_init(mma_drain, 1);
    fence_mbar_init();
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
    if (tma_y) prefetch_tmap(&tm_y);
  }
  if (warp == 9) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();

  const int q = warp & 3, h = warp >> 2;      // epilogue warps
  unsigned char* box = smem + kP8BoxOffset + warp * kP8BoxBytes;
  float2* colv = reinterpret_cast<float2*>(smem + kP8ColOffset) + warp * kP8Cols;
  float sx = 0.f;
  // the scales of a band, ahead of its sums
  auto load_scales = [&](int m0, int n0) {
    sx = m0 + lane < a.M ? a.sx[m0 + lane] : 0.f;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kP8Cols / 32; ++i) {
      const int n = n0 + 32 * i + lane;
      colv[32 * i + lane] = n < a.N ? make_float2(a.sw[n], a.bias ? a.bias[n] : 0.f) : make_float2(0.f, 0.f);
    }
    __syncwarp();
  };
  bool done = false;                          // SPLIT: this warp's tile is complete

  if (warp == 8) {
    if (lane == 0) {
      const uint32_t full_even = mapa_shared(smem_u32(full), even);
      uint32_t it = 0;
      bool ok = true;
      for (int tile = cluster; tile < ntiles && ok; tile += nclusters) {
        const Int8Tile t = int8_pair_tile(tile, tiles_m, tiles_n);
        for (int kt = kt0; kt < kt1; ++kt, ++it) {
          const uint32_t s = it % kP8Stages;
          if (!mbar_wait(empty + s, ((it / kP8Stages) & 1u) ^ 1u, kDevErrTimeoutEmpty)) {
            ok = false;
            break;
          }
          unsigned char* sa = smem + s * kP8StageBytes;
          if (crank == 0) mbar_arrive_expect_tx(full + s, 2 * kP8StageBytes);
          tma_load_2d_pair(sa, &tm_x, full_even + 8 * s, kt * kI8KTile, t.m0 + 128 * (int)crank);
          tma_load_2d_pair(sa + kI8StageA, &tm_w, full_even + 8 * s, kt * kI8KTile, t.n0 + 128 * (int)crank);
        }
      }
      // After a failure, let this thread's loads land before the CTAs exit. The
      // odd CTA's are counted in the other CTA, so both wait a time that no load
      // in flight can outlast.
      if (device_error_set()) {
        const unsigned long long t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull) {
        }
      }
    }
  } else if (warp == 9) {
    if (lane == 0 && crank == 0) {
      const uint32_t idesc = idesc_i8(256, 256);
      const uint64_t dA0 = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
      const uint64_t dB0 = smem_desc(smem_u32(smem) + kI8StageA, 16, 1024, kSwizzle128B);
      uint32_t it = 0, tcount = 0;
      bool ok = true;
      for (int tile = cluster; tile < ntiles && ok; tile += nclusters, ++tcount) {
        const uint32_t buf = tcount & 1u;
        if (!mbar_wait(acc_empty + buf, ((tcount >> 1) & 1u) ^ 1u, kDevErrTimeoutAccum)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kt = kt0; kt < kt1; ++kt, ++it) {
          const uint32_t s = it % kP8Stages;
          if (!mbar_wait(full + s, (it / kP8Stages) & 1u, kDevErrTimeoutFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t off = (uint64_t)(s * ((uint32_t)kP8StageBytes >> 4));
#pragma unroll
          for (int j = 0; j < kI8KTile / 32; ++j)
            mma_i8_pair(tmem + 256 * buf, dA0 + off + 2u * j, dB0 + off + 2u * j, idesc, kt > kt0 || j > 0 ? 1u : 0u);
          tc_commit_pair(empty + s, both);
        }
        if (ok) tc_commit_pair(acc_full + buf, both);
      }
      if (!ok) {
        tc_commit_pair(mma_drain, (uint16_t)(1u << even));
        mbar_drain(mma_drain, 0);
      }
    }
  } else if constexpr (SPLIT) {
    const Int8Tile t = int8_pair_tile(cluster, tiles_m, tiles_n);
    if (h == part) load_scales(t.m0 + 128 * (int)crank + 32 * q, t.n0 + 128 * h);
    done = __all_sync(0xFFFFFFFFu, mbar_wait(acc_full, 0, kDevErrTimeoutAccum) && !device_error_set());
    tc_fence_after();
  } else {
    const uint32_t acc_empty_even = mapa_shared(smem_u32(acc_empty), even);
    uint32_t tcount = 0;
    for (int tile = cluster; tile < ntiles; tile += nclusters, ++tcount) {
      const Int8Tile t = int8_pair_tile(tile, tiles_m, tiles_n);
      const uint32_t buf = tcount & 1u;
      const int m0 = t.m0 + 128 * (int)crank + 32 * q, n0 = t.n0 + 128 * h;
      load_scales(m0, n0);
      const bool ok =
          __all_sync(0xFFFFFFFFu, mbar_wait(acc_full + buf, (tcount >> 1) & 1u, kDevErrTimeoutAccum) && !device_error_set());
      tc_fence_after();
      if (!ok) break;
      int8_store_band<OT>(tmem + ((uint32_t)(q * 32) << 16) + 256 * buf + (uint32_t)(h * 128), nullptr, sx, colv, box, tm_y,
                          tma_y, a, m0, n0, lane, [&] {
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_remote(acc_empty_even + 8 * buf);
                          });
    }
    if (lane == 0) bulk_wait<0>();
  }
  if constexpr (SPLIT) {
    __syncwarp();
    cluster_sync();   // every MMA of the cluster has read its stages: the rings are free
    const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * 128);
    const uint32_t row = smem_u32(smem) + (uint32_t)((32 * q + lane) * kP8PartLd * 4);
    if (done && h != part) {
      const uint32_t there = mapa_shared(row, rank ^ 2u);
#pragma unroll
      for (int c = 0; c < kP8Cols; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(taddr + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(there + 4 * (c + i)), "r"(v[i]),
                       "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3])
                       : "memory");
      }
      tc_fence_before();
    }
    cluster_sync();   // the halves are there
    if (done && h == part) {
      const Int8Tile t = int8_pair_tile(cluster, tiles_m, tiles_n);
      int8_store_band<OT>(taddr, reinterpret_cast<const int*>(smem) + (32 * q + lane) * kP8PartLd, sx, colv, box, tm_y,
                          tma_y, a, t.m0 + 128 * (int)crank + 32 * q, t.n0 + 128 * h, lane, [] {});
      if (lane == 0) bulk_wait<0>();
    }
  }
  tc_fence_before();
  cluster_sync();   // no CTA leaves while its peer may still signal its barriers
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace svdq
