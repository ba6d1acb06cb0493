// The W8A8 linear layer: 8-bit integer codes with one scale per token of X and
// one per output channel of W,
//   Y[m][n] = sx[m] sw[n] sum_k qx[m][k] qw[n][k] + bias[n].
// The integer sum runs on the tensor cores (tcgen05 kind::i8, int32
// accumulators in tensor memory), so it is exact: |sum| <= 127^2 K < 2^31 for
// K <= 131072. The epilogue rounds the sum to fp32, multiplies by sw and then by
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

// A team of blockDim.x threads (a warp, or the whole block) takes a row at a
// time and holds it in registers, NV vectors a thread: one read of X, one
// write of the codes, which is the bound (HBM). NV = 0: the row does not fit;
// it is read once for its maximum and once more, from L2, for its codes.
template <typename T, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) int8_quantize_kernel(const Int8QuantArgs a) {
  constexpr int N = kVecN<T>;
  constexpr int R = NV ? NV : 1;
  __shared__ float2 slots[2][32];
  const int warps = blockDim.x >> 5, tid = threadIdx.x;
  const int step = (int)blockDim.x * N;
  grid_dependency_wait();
  grid_launch_dependents();
  const long long teams = (long long)gridDim.x * blockDim.y;
  int turn = 0;
  for (long long m = (long long)blockIdx.x * blockDim.y + threadIdx.y; m < a.M; m += teams, turn ^= 1) {
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
        r[v] = k < a.K ? load_once(x + k) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int k = v * step + tid * N;
        if (k < a.K) look(r[v], k);
      }
    } else {
      for (int k = tid * N; k < a.K; k += step) look(*reinterpret_cast<const uint4*>(x + k), k);
    }
    const Int8Scale sc = int8_scale(team_max_nan(amax, warps, slots[turn]));
    if (tid == 0) a.s[m] = sc.s;
    int8_t* q = a.q + m * a.K;
    if constexpr (NV > 0) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int k = v * step + tid * N;
        if (k < a.K) {
          float f[N];
          int8_values<T>(a, r[v], k, f);
          int8_store<N>(q + k, f, sc);
        }
      }
    } else {
      for (int k = tid * N; k < a.K; k += step) {
        float f[N];
        int8_values<T>(a, *reinterpret_cast<const uint4*>(x + k), k, f);
        int8_store<N>(q + k, f, sc);
      }
    }
  }
}

// Many rows of more than one warp: a block per row, rows streamed through the
// ring, the factors in registers, E elements a thread.
template <typename T, int E, int W>
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
    in[v] = k < a.K;
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
  int a_rows;          // rows of the A box (8..128)
};

// ---------------------------------------------------------------- single-CTA kernel
// One 128 x NB output tile per CTA and K slice; a cluster of gridDim.z CTAs
// splits K when there are too few tiles for the GPU. Roles: warps 0-3 take the
// accumulator out of tensor memory, warp 4 loads (TMA, 128 bytes of K per
// stage), warp 5 issues the MMAs. The int32 tile then goes through shared
// memory (the ring's, idle by then), where the CTAs of a cluster read each
// other's: CTA z adds and writes the tile's columns [z, z + 1) NB / gridDim.z.
// Rows of a row-tile past M are neither loaded (the A box is cut to a_rows)
// nor written, so one token costs one row of traffic.
constexpr int kI8KTile = 128;                        // K elements (= bytes) per stage row
constexpr int kI8StageA = 128 * kI8KTile;            // 16 KB
constexpr int kI8Threads = 192;

template <int NB>
struct Int8Cfg {
  static constexpr int kStageB = NB * kI8KTile;
  static constexpr int kStageBytes = kI8StageA + kStageB;
  static constexpr int kStages = NB == 64 ? 4 : 3;
  static constexpr int kLd = NB + 4;                 // int32 per row of the staged tile
  static constexpr int kTileBytes = 128 * kLd * 4;
  static constexpr int kRing = kStages * kStageBytes > kTileBytes ? kStages * kStageBytes : kTileBytes;
  static constexpr int kBarOffset = kRing;
  static constexpr int kBytes = kBarOffset + 128 + 1024;
};

__device__ __forceinline__ int4 ld_cluster_int4(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

template <int NB, typename OT>
__global__ void __launch_bounds__(kI8Threads) svdq_int8_gemm_kernel(const __grid_constant__ CUtensorMap tm_x,
                                                                    const __grid_constant__ CUtensorMap tm_w,
                                                                    const Int8GemmArgs a) {
  using C = Int8Cfg<NB>;
  extern __shared__ __align__(1024) unsigned char i8_smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(i8_smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);
  uint64_t* empty = full + C::kStages;
  uint64_t* done = empty + C::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles_n = (a.N + NB - 1) / NB;
  const int n0 = (int)(blockIdx.x % tiles_n) * NB, m0 = (int)(blockIdx.x / tiles_n) * 128;
  const int splits = gridDim.z, z = blockIdx.z;
  const int kts = (a.K + kI8KTile - 1) / kI8KTile;
  const int kt0 = (int)((long long)kts * z / splits), kt1 = (int)((long long)kts * (z + 1) / splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    mbar_init(done, 1);
    fence_mbar_init();
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
  }
  if (warp == 5) {
    tmem_alloc(tmem_slot, NB);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();

  bool ok = true;
  if (warp == 4) {
    if (lane == 0) {
      const uint32_t bytes = (uint32_t)(a.a_rows * kI8KTile + C::kStageB);
      int it = 0;
      for (int kt = kt0; kt < kt1; ++kt, ++it) {
        const int s = it % C::kStages;
        if (!mbar_wait(empty + s, ((it / C::kStages) & 1) ^ 1, kDevErrTimeoutEmpty)) break;
        unsigned char* sa = smem + s * C::kStageBytes;
        mbar_arrive_expect_tx(full + s, bytes);
        tma_load_2d(sa, &tm_x, full + s, kt * kI8KTile, m0);
        tma_load_2d(sa + kI8StageA, &tm_w, full + s, kt * kI8KTile, n0);
      }
      if (device_error_set())   // let the copies this thread issued land before the CTA exits
        for (int j = it > C::kStages ? it - C::kStages : 0; j < it; ++j)
          mbar_drain(full + j % C::kStages, (j / C::kStages) & 1);
    }
  } else if (warp == 5) {
    if (lane == 0) {
      const uint32_t idesc = idesc_i8(128, NB);
      int it = 0;
      for (int kt = kt0; kt < kt1; ++kt, ++it) {
        const int s = it % C::kStages;
        if (!mbar_wait(full + s, (it / C::kStages) & 1, kDevErrTimeoutFull)) break;
        tc_fence_after();
        const uint64_t ad = smem_desc(smem_u32(smem + s * C::kStageBytes), 16, 1024, kSwizzle128B);
        const uint64_t bd = smem_desc(smem_u32(smem + s * C::kStageBytes + kI8StageA), 16, 1024, kSwizzle128B);
#pragma unroll
        for (int j = 0; j < kI8KTile / 32; ++j)   // 32 K elements (32 bytes) per MMA
          mma_i8(tmem, ad + 2u * j, bd + 2u * j, idesc, (it | j) != 0 ? 1u : 0u);
        tc_commit(empty + s);
      }
      tc_commit(done);
    }
  }
  __syncwarp();
  // every MMA has read its stages: the ring is free for the tile
  if (warp < 4) {
    ok = mbar_wait(done, 0, kDevErrTimeoutAccum) && !device_error_set();
    ok = __all_sync(0xFFFFFFFFu, ok);
    tc_fence_after();
    const int row = 32 * warp + lane;
    if (ok && 32 * warp < a.M - m0) {
      int* tile = reinterpret_cast<int*>(smem) + row * C::kLd;
#pragma unroll
      for (int c = 0; c < NB; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * warp) << 16) + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          *reinterpret_cast<uint4*>(tile + c + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
    }
    tc_fence_before();
  }
  if (splits > 1) cluster_sync();
  else __syncthreads();
  if (!device_error_set()) {
    const int rows = min(128, a.M - m0), cols = NB / splits;
    const int c_begin = z * cols;
    OT* y = static_cast<OT*>(a.y) + (long long)m0 * a.ldy + n0;
    const bool vec = (a.ldy & 3) == 0;
    const uint32_t base = smem_u32(smem);
    for (int j = threadIdx.x; j < rows * (cols / 4); j += kI8Threads) {
      const int r = j / (cols / 4), c = c_begin + 4 * (j % (cols / 4));
      if (n0 + c >= a.N) continue;
      int4 v = *reinterpret_cast<const int4*>(smem + ((size_t)r * C::kLd + c) * 4);
      for (int p = 1; p < splits; ++p) {
        const int4 u = ld_cluster_int4(mapa_shared(base + (uint32_t)(r * C::kLd + c) * 4, (uint32_t)((z + p) % splits)));
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
      }
      const float sx = a.sx[m0 + r];
      const int t[4] = {v.x, v.y, v.z, v.w};
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = min(n0 + c + i, a.N - 1);
        f[i] = fmaf((float)t[i] * a.sw[n], sx, a.bias ? a.bias[n] : 0.f);
      }
      OT* p = y + (long long)r * a.ldy + c;
      if (vec && n0 + c + 4 <= a.N) {
        if constexpr (sizeof(OT) == 4) *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
        else *reinterpret_cast<uint2*>(p) = make_uint2(pack2(f[0], f[1], OT()), pack2(f[2], f[3], OT()));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n0 + c + i < a.N) p[i] = from_float<OT>(f[i]);
      }
    }
  }
  tc_fence_before();
  if (splits > 1) cluster_sync();   // no CTA leaves while a peer may read its tile
  else __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, NB);
  }
}

// ---------------------------------------------------------------- CTA-pair kernel
// Large products: one tcgen05 MMA (cta_group::2) spans the two SMs of a cluster
// of 2 and computes a 256 x 256 tile; each CTA stages its own 128 rows of X and
// its own 128 rows of W (64 bytes of operands per 1024 multiply-adds and CTA,
// half of what two single CTAs would fetch). Persistent: cluster c takes tiles
// c, c + clusters, ...; two accumulators (all 512 columns of tensor memory)
// alternate, so a tile's epilogue runs under the next tile's MMAs.
// Roles per CTA (320 threads):
//   warps 0-7  epilogue: warp (q, h) takes accumulator lanes 32q.. and columns
//              128h..: scales, bias, rounding, 128B-swizzled boxes, TMA stores
//   warp 8     producer: TMA loads of this CTA's rows, counted on the even
//              CTA's stage barrier (64 KB for both)
//   warp 9     the even CTA's lane 0 issues the MMAs; a multicast commit frees
//              each stage, and hands over each accumulator, in both CTAs
// Tiles go in bands of kP8Band tile rows, column by column: the clusters that
// run at one time then share few rows of X and of W, and L2 serves the rest.
constexpr int kP8Stages = 5;
constexpr int kP8StageBytes = 2 * 128 * kI8KTile;            // 32 KB: 128 rows of X, 128 rows of W
constexpr int kP8Threads = 320;
constexpr int kP8EpiWarps = 8;
constexpr int kP8Band = 8;
constexpr int kP8BoxBytes = 4096;                            // 32 rows x 128 bytes
constexpr int kP8BoxOffset = kP8Stages * kP8StageBytes;
constexpr int kP8ColOffset = kP8BoxOffset + kP8EpiWarps * kP8BoxBytes;   // (sw, bias) of each warp's 128 columns
constexpr int kP8BarOffset = kP8ColOffset + kP8EpiWarps * 128 * 8;
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

// tm_y views Y as bytes, in boxes of 32 rows x 128; tma_y = 0 where Y's address or
// row stride does not allow it (then the staged boxes are written by plain stores).
template <typename OT>
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
  const uint32_t crank = cluster_ctarank();
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
  const int tiles_m = (a.M + 255) / 256, tiles_n = (a.N + 255) / 256;
  const int ntiles = tiles_m * tiles_n;
  const int kts = (a.K + kI8KTile - 1) / kI8KTile;

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

  if (warp == 8) {
    if (lane == 0) {
      const uint32_t full_even = mapa_shared(smem_u32(full), 0);
      uint32_t it = 0;
      bool ok = true;
      for (int tile = cluster; tile < ntiles && ok; tile += nclusters) {
        const Int8Tile t = int8_pair_tile(tile, tiles_m, tiles_n);
        for (int kt = 0; kt < kts; ++kt, ++it) {
          const uint32_t s = it % kP8Stages;
          if (!mbar_wait(empty + s, ((it / kP8Stages) & 1u) ^ 1u, kDevErrTimeoutEmpty)) {
            ok = false;
            break;
          }
          unsigned char* sa = smem + s * kP8StageBytes;
          if (crank == 0) mbar_arrive_expect_tx(full + s, 2 * kP8StageBytes);
          tma_load_2d_pair(sa, &tm_x, full_even + 8 * s, kt * kI8KTile, t.m0 + 128 * (int)crank);
          tma_load_2d_pair(sa + kP8StageBytes / 2, &tm_w, full_even + 8 * s, kt * kI8KTile, t.n0 + 128 * (int)crank);
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
      const uint64_t dB0 = smem_desc(smem_u32(smem) + kP8StageBytes / 2, 16, 1024, kSwizzle128B);
      uint32_t it = 0, tcount = 0;
      bool ok = true;
      for (int tile = cluster; tile < ntiles && ok; tile += nclusters, ++tcount) {
        const uint32_t buf = tcount & 1u;
        if (!mbar_wait(acc_empty + buf, ((tcount >> 1) & 1u) ^ 1u, kDevErrTimeoutAccum)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kt = 0; kt < kts; ++kt, ++it) {
          const uint32_t s = it % kP8Stages;
          if (!mbar_wait(full + s, (it / kP8Stages) & 1u, kDevErrTimeoutFull)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t off = (uint64_t)(s * ((uint32_t)kP8StageBytes >> 4));
#pragma unroll
          for (int j = 0; j < kI8KTile / 32; ++j)
            mma_i8_pair(tmem + 256 * buf, dA0 + off + 2u * j, dB0 + off + 2u * j, idesc, (kt | j) != 0 ? 1u : 0u);
          tc_commit_pair(empty + s, 0x3);
        }
        if (ok) tc_commit_pair(acc_full + buf, 0x3);
      }
      if (!ok) {
        tc_commit_pair(mma_drain, 0x1);
        mbar_drain(mma_drain, 0);
      }
    }
  } else {
    const int q = warp & 3, h = warp >> 2;
    unsigned char* box = smem + kP8BoxOffset + warp * kP8BoxBytes;
    float2* colv = reinterpret_cast<float2*>(smem + kP8ColOffset) + warp * 128;
    const uint32_t acc_empty_even = mapa_shared(smem_u32(acc_empty), 0);
    constexpr int kBoxCols = 128 / (int)sizeof(OT);
    uint32_t tcount = 0;
    for (int tile = cluster; tile < ntiles; tile += nclusters, ++tcount) {
      const Int8Tile t = int8_pair_tile(tile, tiles_m, tiles_n);
      const uint32_t buf = tcount & 1u;
      const int m0 = t.m0 + 128 * (int)crank + 32 * q, n0 = t.n0 + 128 * h;
      const float sx = m0 + lane < a.M ? a.sx[m0 + lane] : 0.f;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + 32 * i + lane;
        colv[32 * i + lane] = n < a.N ? make_float2(a.sw[n], a.bias ? a.bias[n] : 0.f) : make_float2(0.f, 0.f);
      }
      __syncwarp();
      bool ok = mbar_wait(acc_full + buf, (tcount >> 1) & 1u, kDevErrTimeoutAccum) && !device_error_set();
      ok = __all_sync(0xFFFFFFFFu, ok);
      tc_fence_after();
      if (!ok) break;
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + 256 * buf + (uint32_t)(h * 128);
      const bool live = m0 < a.M;
#pragma unroll
      for (int b = 0; b < 128 / kBoxCols; ++b) {
        if (tma_y && lane == 0) bulk_wait_read<0>();   // the previous store from this box has read it
        __syncwarp();
#pragma unroll
        for (int c = 0; c < kBoxCols; c += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + b * kBoxCols + c, v);
          tmem_ld_wait();
          if (b * kBoxCols + c + 32 == 128) {   // the accumulator is drained
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(acc_empty_even + 8 * buf);
          }
          float f[32];
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float4 sb = *reinterpret_cast<const float4*>(colv + b * kBoxCols + c + i);
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
          for (int r = 0; r < rows; ++r)
#pragma unroll
            for (int c = 0; c < kBoxCols; c += 32) {
              const int e = c + lane, byte = e * (int)sizeof(OT);
              const OT value = *reinterpret_cast<const OT*>(box + r * 128 + (((byte >> 4) ^ (r & 7)) << 4) + (byte & 15));
              if (col0 + e < a.N) static_cast<OT*>(a.y)[(long long)(m0 + r) * a.ldy + col0 + e] = value;
            }
        }
      }
    }
    if (lane == 0) bulk_wait<0>();
  }
  tc_fence_before();
  cluster_sync();   // no CTA leaves while its peer may still signal its barriers
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace svdq
