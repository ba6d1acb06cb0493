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
  int a_rows;          // single-CTA kernel: rows of the A box (8..128)
  int stages;          // single-CTA kernel: stages of its ring
};

// ---------------------------------------------------------------- few tokens
// Y for at most 8 tokens: every weight is read once and used M times, so the
// product is bound by HBM and the integer dot-product instruction (dp4a: four
// products per lane) keeps up. A warp holds a 512-byte slice of kGvChannels
// rows of W (16 bytes a lane, all loads in flight at once) and the same slice
// of each token; a block's warps take `warps_k` slices of the same channels in
// turn, or several channel groups where K is short. Sums are integers, so any
// order gives the same bits.
constexpr int kGvThreads = 256;
constexpr int kGvChannels = 8;

template <int MT, typename OT>
__global__ void __launch_bounds__(kGvThreads) int8_few_tokens_kernel(const int8_t* __restrict__ qx,
                                                                     const int8_t* __restrict__ qw,
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
  bool waited = false;
  for (int k = wk * 512 + lane * 16; k < a.K; k += warps_k * 512) {
    uint4 r[kGvChannels];
#pragma unroll
    for (int c = 0; c < kGvChannels; ++c)
      r[c] = n0 + c < a.N ? load_once(w + (long long)c * a.K + k) : make_uint4(0, 0, 0, 0);
    if (!waited) {   // the weights are no earlier kernel's output: their first loads go ahead of the wait
      grid_dependency_wait();
      waited = true;
    }
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
  if (!waited) grid_dependency_wait();
  grid_launch_dependents();
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
// One 128 x NB output tile per CTA and K slice; a cluster of gridDim.z CTAs
// splits K when there are too few tiles for the GPU. Warp 0 loads (TMA, 128
// bytes of K per stage), warp 1 issues the MMAs, then all eight warps take the
// accumulator out of tensor memory (warp w: lanes 32 (w % 4).., half of the
// columns) into shared memory (the ring's, idle by then). The CTAs of a cluster
// read each other's tiles there: CTA z adds and writes the columns
// [z, z + 1) NB / gridDim.z. A lane keeps its columns and their scales from row
// to row. Rows past M are neither loaded (the A box is cut to a_rows) nor
// written, so few tokens cost little traffic.
constexpr int kI8KTile = 128;                        // K elements (= bytes) per stage row
constexpr int kI8StageA = 128 * kI8KTile;            // 16 KB
constexpr int kI8Threads = 256;

// The ring follows the barriers in shared memory; it has `few` stages where two
// CTAs share an SM and `many` where each has one to itself (what is in flight
// bounds a CTA's rate: 96 KB of it).
template <int NB>
struct Int8Cfg {
  static constexpr int kStageB = NB * kI8KTile;
  static constexpr int kStageBytes = kI8StageA + kStageB;
  static constexpr int kFew = NB == 64 ? 4 : 3, kMany = NB == 64 ? 8 : 6;
  static constexpr int kLd = NB + 4;                 // int32 per row of the staged tile
  static constexpr int kTileBytes = 128 * kLd * 4;
  static_assert(kFew * kStageBytes >= kTileBytes, "the tile is staged in the ring");
  static constexpr int bytes(int stages) { return 1024 + 1024 + stages * kStageBytes; }
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
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + C::kMany;
  uint64_t* done = empty + C::kMany;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  smem += 1024;
  const int stages = a.stages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tiles_n = (a.N + NB - 1) / NB;
  const int n0 = (int)(blockIdx.x % tiles_n) * NB, m0 = (int)(blockIdx.x / tiles_n) * 128;
  const int splits = gridDim.z, z = blockIdx.z;
  const int kts = (a.K + kI8KTile - 1) / kI8KTile;
  const int kt0 = (int)((long long)kts * z / splits), kt1 = (int)((long long)kts * (z + 1) / splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    mbar_init(done, 1);
    fence_mbar_init();
    prefetch_tmap(&tm_x);
    prefetch_tmap(&tm_w);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, NB);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  grid_launch_dependents();

  if (warp == 0 && lane == 0) {
    const uint32_t bytes = (uint32_t)(a.a_rows * kI8KTile + C::kStageB);
    int s = 0, kt = kt0;
    uint32_t ph = 1;
    for (; kt < kt1; ++kt) {
      if (!mbar_wait(empty + s, ph, kDevErrTimeoutEmpty)) break;
      unsigned char* sa = smem + s * C::kStageBytes;
      mbar_arrive_expect_tx(full + s, bytes);
      tma_load_2d(sa, &tm_x, full + s, kt * kI8KTile, m0);
      tma_load_2d(sa + kI8StageA, &tm_w, full + s, kt * kI8KTile, n0);
      if (++s == stages) {
        s = 0;
        ph ^= 1u;
      }
    }
    if (device_error_set()) {   // let the copies this thread issued land before the CTA exits
      const int it = kt - kt0;
      for (int j = it > stages ? it - stages : 0; j < it; ++j) mbar_drain(full + j % stages, (j / stages) & 1);
    }
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = idesc_i8(128, NB);
    int s = 0;
    uint32_t ph = 0;
    for (int kt = kt0; kt < kt1; ++kt) {
      if (!mbar_wait(full + s, ph, kDevErrTimeoutFull)) break;
      tc_fence_after();
      const uint64_t ad = smem_desc(smem_u32(smem + s * C::kStageBytes), 16, 1024, kSwizzle128B);
      const uint64_t bd = smem_desc(smem_u32(smem + s * C::kStageBytes + kI8StageA), 16, 1024, kSwizzle128B);
#pragma unroll
      for (int j = 0; j < kI8KTile / 32; ++j)   // 32 K elements (32 bytes) per MMA
        mma_i8(tmem, ad + 2u * j, bd + 2u * j, idesc, kt > kt0 || j > 0 ? 1u : 0u);
      tc_commit(empty + s);
      if (++s == stages) {
        s = 0;
        ph ^= 1u;
      }
    }
    tc_commit(done);
  }
  __syncwarp();
  // every MMA has read its stages: the ring is free for the tile
  const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(done, 0, kDevErrTimeoutAccum) && !device_error_set());
  tc_fence_after();
  const int q = warp & 3;
  if (ok && 32 * q < a.M - m0) {
    int* tile = reinterpret_cast<int*>(smem) + (32 * q + lane) * C::kLd;
#pragma unroll
    for (int c = (warp >> 2) * (NB / 2); c < ((warp >> 2) + 1) * (NB / 2); c += 32) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(tmem + ((uint32_t)(32 * q) << 16) + c, v);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 32; i += 4)
        *reinterpret_cast<uint4*>(tile + c + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
  }
  tc_fence_before();
  if (splits > 1) cluster_sync();
  else __syncthreads();
  if (ok) {
    // a lane's four columns: neighbours where Y's rows allow wide stores, else
    // a quarter of the columns apart, so that a warp's single stores are dense
    const int rows = min(128, a.M - m0), cols = NB / splits, per_row = cols / 4;
    const bool wide = (a.ldy & 3) == 0;
    const int place = lane % per_row;
    const int c0 = z * cols + (wide ? 4 * place : place), dc = wide ? 1 : per_row;
    float sw[4], bias[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = min(n0 + c0 + i * dc, a.N - 1);
      sw[i] = a.sw[n];
      bias[i] = a.bias ? a.bias[n] : 0.f;
    }
    const int rows_per_warp = 32 / per_row;
    const uint32_t base = smem_u32(smem);
    OT* y = static_cast<OT*>(a.y) + (long long)m0 * a.ldy + n0 + c0;
#pragma unroll 2
    for (int r = warp * rows_per_warp + lane / per_row; r < rows; r += (kI8Threads / 32) * rows_per_warp) {
      const uint32_t at = (uint32_t)(r * C::kLd + c0) * 4;
      int t[4];
      if (wide) {
        int4 v = *reinterpret_cast<const int4*>(smem + at);
        for (int p = 1; p < splits; ++p) {
          const int4 u = ld_cluster_int4(mapa_shared(base + at, (uint32_t)((z + p) % splits)));
          v.x += u.x;
          v.y += u.y;
          v.z += u.z;
          v.w += u.w;
        }
        t[0] = v.x; t[1] = v.y; t[2] = v.z; t[3] = v.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          t[i] = *reinterpret_cast<const int*>(smem + at + 4 * i * dc);
          for (int p = 1; p < splits; ++p) {
            int u;
            asm volatile("ld.shared::cluster.b32 %0, [%1];"
                         : "=r"(u)
                         : "r"(mapa_shared(base + at + 4 * i * dc, (uint32_t)((z + p) % splits)))
                         : "memory");
            t[i] += u;
          }
        }
      }
      const float sx = a.sx[m0 + r];
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
  if (splits > 1) cluster_sync();   // no CTA leaves while a peer may read its tile
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, NB);
  }
}

// ---------------------------------------------------------------- CTA-pair kernel
// Large products: one tcgen05 MMA (cta_group::2) spans the two SMs of a cluster
// of 2 and computes a 256 x NB tile (NB = 256, or 128 where that fills more SMs);
// each CTA stages its own 128 rows of X and its own NB / 2 rows of W (at NB = 256
// half of what two single CTAs would fetch for the same tile). Persistent:
// cluster c takes tiles c, c + clusters, ...; two accumulators alternate, so a
// tile's epilogue runs under the next tile's MMAs.
// Roles per CTA (320 threads):
//   warps 0-7  epilogue: warp (q, h) takes accumulator lanes 32q.. and columns
//              h NB/2..: scales, bias, rounding, 128B-swizzled boxes, TMA stores
//   warp 8     producer: TMA loads of this CTA's rows, counted on the even
//              CTA's stage barrier (both CTAs' bytes)
//   warp 9     the even CTA's lane 0 issues the MMAs; a multicast commit frees
//              each stage, and hands over each accumulator, in both CTAs
// Tiles go in bands of kP8Band tile rows, column by column: the clusters that
// run at one time then share few rows of X and of W, and L2 serves the rest.
constexpr int kP8Threads = 320;
constexpr int kP8EpiWarps = 8;
constexpr int kP8Band = 8;
constexpr int kP8BoxBytes = 4096;                            // 32 rows x 128 bytes

template <int NB>
struct Int8PairCfg {
  static constexpr int kStageBytes = (128 + NB / 2) * kI8KTile;   // 32 | 24 KB
  static constexpr int kStages = NB == 256 ? 5 : 7;
  static constexpr int kCols = NB / 2;                            // accumulator columns per epilogue warp
  static constexpr int kBoxOffset = kStages * kStageBytes;
  static constexpr int kColOffset = kBoxOffset + kP8EpiWarps * kP8BoxBytes;   // (sw, bias) of each warp's columns
  static constexpr int kBarOffset = kColOffset + kP8EpiWarps * kCols * 8;
  static constexpr int kBytes = kBarOffset + 256 + 1024;
};

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

template <int NB>
__device__ __forceinline__ Int8Tile int8_pair_tile(int tile, int tiles_m, int tiles_n) {
  const int band = tile / (kP8Band * tiles_n);
  const int rows = min(kP8Band, tiles_m - band * kP8Band);
  const int i = tile - band * kP8Band * tiles_n;
  return Int8Tile{(band * kP8Band + i % rows) * 256, (i / rows) * NB};
}

// tm_y views Y as bytes, in boxes of 32 rows x 128; tma_y = 0 where Y's address or
// row stride does not allow it (then the staged boxes are written by plain stores).
template <int NB, typename OT>
__global__ void __launch_bounds__(kP8Threads, 1) svdq_int8_gemm_pair_kernel(const __grid_constant__ CUtensorMap tm_x,
                                                                            const __grid_constant__ CUtensorMap tm_w,
                                                                            const __grid_constant__ CUtensorMap tm_y,
                                                                            const Int8GemmArgs a, int tma_y) {
  using C = Int8PairCfg<NB>;
  constexpr int kP8Stages = C::kStages, kP8StageBytes = C::kStageBytes;
  extern __shared__ __align__(1024) unsigned char p8_smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(p8_smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);   // even CTA: both CTAs' loads
  uint64_t* empty = full + kP8Stages;
  uint64_t* acc_full = empty + kP8Stages;    // [2]
  uint64_t* acc_empty = acc_full + 2;        // [2], even CTA: both CTAs' epilogue warps
  uint64_t* mma_drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
  const int tiles_m = (a.M + 255) / 256, tiles_n = (a.N + NB - 1) / NB;
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
    tmem_alloc_pair(tmem_slot, 2 * NB);
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
        const Int8Tile t = int8_pair_tile<NB>(tile, tiles_m, tiles_n);
        for (int kt = 0; kt < kts; ++kt, ++it) {
          const uint32_t s = it % kP8Stages;
          if (!mbar_wait(empty + s, ((it / kP8Stages) & 1u) ^ 1u, kDevErrTimeoutEmpty)) {
            ok = false;
            break;
          }
          unsigned char* sa = smem + s * kP8StageBytes;
          if (crank == 0) mbar_arrive_expect_tx(full + s, 2 * kP8StageBytes);
          tma_load_2d_pair(sa, &tm_x, full_even + 8 * s, kt * kI8KTile, t.m0 + 128 * (int)crank);
          tma_load_2d_pair(sa + kI8StageA, &tm_w, full_even + 8 * s, kt * kI8KTile, t.n0 + NB / 2 * (int)crank);
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
      const uint32_t idesc = idesc_i8(256, NB);
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
            mma_i8_pair(tmem + NB * buf, dA0 + off + 2u * j, dB0 + off + 2u * j, idesc, (kt | j) != 0 ? 1u : 0u);
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
    unsigned char* box = smem + C::kBoxOffset + warp * kP8BoxBytes;
    float2* colv = reinterpret_cast<float2*>(smem + C::kColOffset) + warp * C::kCols;
    const uint32_t acc_empty_even = mapa_shared(smem_u32(acc_empty), 0);
    constexpr int kBoxCols = 128 / (int)sizeof(OT);
    uint32_t tcount = 0;
    for (int tile = cluster; tile < ntiles; tile += nclusters, ++tcount) {
      const Int8Tile t = int8_pair_tile<NB>(tile, tiles_m, tiles_n);
      const uint32_t buf = tcount & 1u;
      const int m0 = t.m0 + 128 * (int)crank + 32 * q, n0 = t.n0 + C::kCols * h;
      const float sx = m0 + lane < a.M ? a.sx[m0 + lane] : 0.f;
      __syncwarp();
#pragma unroll
      for (int i = 0; i < C::kCols / 32; ++i) {
        const int n = n0 + 32 * i + lane;
        colv[32 * i + lane] = n < a.N ? make_float2(a.sw[n], a.bias ? a.bias[n] : 0.f) : make_float2(0.f, 0.f);
      }
      __syncwarp();
      bool ok = mbar_wait(acc_full + buf, (tcount >> 1) & 1u, kDevErrTimeoutAccum) && !device_error_set();
      ok = __all_sync(0xFFFFFFFFu, ok);
      tc_fence_after();
      if (!ok) break;
      const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + NB * buf + (uint32_t)(h * C::kCols);
      const bool live = m0 < a.M;
#pragma unroll
      for (int b = 0; b < C::kCols / kBoxCols; ++b) {
        if (tma_y && lane == 0) bulk_wait_read<0>();   // the previous store from this box has read it
        __syncwarp();
#pragma unroll
        for (int c = 0; c < kBoxCols; c += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + b * kBoxCols + c, v);
          tmem_ld_wait();
          if (b * kBoxCols + c + 32 == C::kCols) {   // the accumulator is drained
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
    tmem_dealloc_pair(tmem, 2 * NB);
  }
}

}  // namespace svdq
