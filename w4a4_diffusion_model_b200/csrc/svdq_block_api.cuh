// Host side of the operators around the 4-bit linear layer: the W8A8 linear
// layer, layer norm (forward, backward, with the 8-bit quantizer) and rotary
// positions. Part of the translation unit svdq_api.cu, whose error, device and
// tensor-map helpers it uses.
#pragma once

namespace {

cudaLaunchConfig_t pdl_config(dim3 grid, dim3 block, size_t smem, cudaStream_t st, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

bool float_type(int t) { return t == SVDQ_BF16 || t == SVDQ_FP16 || t == SVDQ_FP32; }
int type_bytes(int t) { return t == SVDQ_FP32 ? 4 : 2; }

svdq_status check_pointers(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p && !aligned16(p)) return fail(SVDQ_ERR_MISALIGNED, "every pointer must be 16-byte aligned");
  return SVDQ_OK;
}

// A matrix of `rows` rows of `cols` values with row stride ld: rows must not
// overlap, and offsets must stay within 2^62 bytes.
svdq_status check_rows(const char* what, int64_t rows, int64_t cols, int64_t ld) {
  if (rows > 1 && (ld < cols || ld > (1ll << 40)))
    return fail(SVDQ_ERR_INVALID_ARG, "%s: row stride %lld for rows of %lld", what, (long long)ld, (long long)cols);
  return SVDQ_OK;
}

// Two matrices in the same memory have the same row stride.
svdq_status check_in_place(const char* what, const void* out, int64_t ldo, const void* in, int64_t ldi, int64_t rows) {
  if (rows > 1 && out == in && ldo != ldi)
    return fail(SVDQ_ERR_INVALID_ARG, "%s in place: row strides %lld and %lld", what, (long long)ldo, (long long)ldi);
  return SVDQ_OK;
}

template <typename T>
struct Tag {
  using type = T;
};

template <int N>
using Int = std::integral_constant<int, N>;

template <auto K>
struct Kern {
  static constexpr auto value = K;
};

template <typename F>
svdq_status with_type(int dtype, F&& f) {
  switch (dtype) {
    case SVDQ_BF16: return f(Tag<__nv_bfloat16>());
    case SVDQ_FP16: return f(Tag<__half>());
    default: return f(Tag<float>());
  }
}

int round_up(int v, int m) { return (v + m - 1) / m * m; }

// Lanes that hold a row of up to 512 values, 16 each: a power of two.
int team_lanes(int values) {
  int lanes = 1;
  while (lanes < 32 && lanes * 16 < values) lanes *= 2;
  return lanes;
}

// Kernels that stream rows through a ring (svdq_rows.cuh) run 512 threads per SM
// (640 in the backward pass up to 320 a block); the blocks share 192 KB, less
// `other` bytes each, for their stages: at least one and at most kRingMaxStages.
constexpr int kRingBytes = 3 * 65536;   // one stage of two rows of 16384 fp32, and the backward pass's weight

int ring_depth(int threads, size_t stage_bytes, size_t other = 0) {
  const int blocks = std::max(1, (other && threads <= 320 ? 640 : 512) / threads);
  const size_t share = kRingBytes / blocks;
  return (int)std::max<size_t>(1, std::min<size_t>(svdq::kRingMaxStages, (share - std::min(share, other)) / stage_bytes));
}

// Resident blocks per SM of a ring kernel; sets its shared-memory attribute.
template <auto KERN>
int ring_blocks_per_sm(int threads, size_t smem) {
  static std::atomic<int> done[kMaxDevices];
  per_device_once(done, current_device(), [] {
    if (cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes) == cudaSuccess) return 1;
    cudaGetLastError();
    return 0;
  });
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, KERN, threads, smem) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  return std::max(n, 1);
}

// Launches a ring kernel that takes rows in turn, `elems` elements a thread;
// FULL_KERN where the columns fill whole warps.
template <auto KERN, auto FULL_KERN, typename Args>
svdq_status launch_rows(Args a, int64_t rows, int64_t cols, int elems, size_t row_bytes, cudaStream_t st) {
  const auto kern = cols % (32 * elems) == 0 ? FULL_KERN : KERN;
  const int threads = round_up((int)((cols + elems - 1) / elems), 32);
  a.depth = ring_depth(threads, row_bytes);
  const size_t smem = a.depth * row_bytes;
  const int64_t blocks = (int64_t)sm_count() *
                         (kern == FULL_KERN ? ring_blocks_per_sm<FULL_KERN>(threads, smem) : ring_blocks_per_sm<KERN>(threads, smem));
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config((unsigned)std::min<int64_t>(rows, blocks), threads, smem, st, attr);
  SVDQ_CUDA(cudaLaunchKernelEx(&cfg, kern, a));
  return SVDQ_OK;
}

// ---------------------------------------------------------------- 8-bit quantizer
constexpr int64_t kInt8MaxK = 131072;   // 127^2 K < 2^31

svdq_status check_int8_k(int64_t rows, int64_t K) {
  if (rows < 0 || rows > (1ll << 30) || K < 16 || K % 16 || K > kInt8MaxK)
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "int8 matrix of %lld x K=%lld: need K a multiple of 16, 16 <= K <= %lld",
                (long long)rows, (long long)K, (long long)kInt8MaxK);
  return SVDQ_OK;
}

template <typename T, int NV, int MAXT>
svdq_status launch_int8_quantize(const svdq::Int8QuantArgs& a, dim3 grid, dim3 block, cudaStream_t st) {
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(grid, block, 0, st, attr);
  SVDQ_CUDA(cudaLaunchKernelEx(&cfg, svdq::int8_quantize_kernel<T, NV, MAXT>, a));
  return SVDQ_OK;
}

svdq_status int8_quantize(int64_t M, int64_t K, int dtype, const void* X, int64_t ldx, const float* mult, void* Q,
                          float* S, void* stream) {
  g_last_error[0] = 0;
  svdq_status r = check_int8_k(M, K);
  if (r != SVDQ_OK) return r;
  if (!float_type(dtype)) return fail(SVDQ_ERR_INVALID_ARG, "unknown type %d", dtype);
  if (M > 0 && (!X || !Q || !S)) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if ((r = check_pointers({X, mult, Q, S})) != SVDQ_OK) return r;
  if ((r = check_rows("X", M, K, ldx)) != SVDQ_OK) return r;
  if (M > 1 && ldx * type_bytes(dtype) % 16)
    return fail(SVDQ_ERR_MISALIGNED, "row stride %lld is not a multiple of 16 bytes", (long long)ldx);
  if ((r = check_device()) != SVDQ_OK) return r;
  if (M == 0) return SVDQ_OK;
  const svdq::Int8QuantArgs a{X, ldx, mult, static_cast<int8_t*>(Q), S, M, (int)K, 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return with_type(dtype, [&](auto tag) -> svdq_status {
    using T = typename decltype(tag)::type;
    constexpr int NV = 16 / svdq::kVecN<T>;   // 16 values a thread
    const int64_t sms = sm_count();
    if (K <= 512) {   // rows that a warp, or some of its lanes, hold
      const int lanes = team_lanes((int)K), teams = 256 / lanes;
      return launch_int8_quantize<T, NV, 256>(a, (unsigned)std::min<int64_t>((M + teams - 1) / teams, sms * 8),
                                              dim3(lanes, teams), st);
    }
    // Many rows: the ring. Measured, us, ring against one row per block: 9001 x
    // 13824 67 / 105, 4608 x 4096 12 / 19; one row per block has the shorter way
    // from memory to registers where rows do not queue.
    if (K <= 16384 && M > 2 * sms) {
      using namespace svdq;
      auto go = [&](auto elems, auto warps) -> svdq_status {
        constexpr int E = decltype(elems)::value, W = decltype(warps)::value;
        return launch_rows<int8_quantize_rows_kernel<T, E, W, false>, int8_quantize_rows_kernel<T, E, W, true>>(
            a, M, K, E, (size_t)K * sizeof(T), st);
      };
      if (K <= 2048) return go(Int<16>(), Int<4>());
      if (K <= 4096) return go(Int<32>(), Int<4>());
      if (K <= 8192) return go(Int<32>(), Int<8>());
      return go(Int<32>(), Int<16>());
    }
    const unsigned grid = (unsigned)std::min<int64_t>(M, sms * 8);
    if (K <= 4096) return launch_int8_quantize<T, NV, 256>(a, grid, round_up((int)(K + 15) / 16, 32), st);
    if (K <= 16384) return launch_int8_quantize<T, NV, 1024>(a, grid, round_up((int)(K + 15) / 16, 32), st);
    return launch_int8_quantize<T, 0, 1024>(a, grid, 1024, st);
  });
}

// ---------------------------------------------------------------- W8A8 product
cudaLaunchConfig_t int8_single_config(int64_t tiles, int splits, cudaStream_t st, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg =
      pdl_config(dim3((unsigned)tiles, 1, (unsigned)splits), svdq::kI8Threads, svdq::kI8Bytes, st, attr);
  if (splits > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = splits;
    cfg.numAttrs = 2;
  }
  return cfg;
}

// Tiles of the single-CTA kernel that run at once with K split `splits` ways (0:
// the kernel cannot run); also sets its shared-memory attribute.
template <typename OT>
int int8_single_tiles(int splits) {
  static std::atomic<int> cache[5][kMaxDevices];
  return per_device_once(cache[splits / 2], current_device(), [splits] {   // splits 1, 2, 4, 8
    auto kern = svdq::svdq_int8_gemm_kernel<OT>;
    int n = 0;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, svdq::kI8Bytes) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = int8_single_config(1, splits, nullptr, attr);
    if (splits == 1) return sm_count() + 1;
    cfg.attrs = attr + 1;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, (void*)kern, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    return n + 1;
  }) - 1;
}

template <typename OT>
svdq_status launch_int8_single(const svdq::Int8GemmArgs& args, const void* Qx, const void* Qw, int splits,
                               cudaStream_t st) {
  svdq::Int8GemmArgs a = args;
  a.a_rows = a.M >= 128 ? 128 : round_up(a.M, 8);
  CUtensorMap tx, tw;
  svdq_status r;
  if ((r = make_tmap(&tx, Qx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)a.K, (uint64_t)a.M, svdq::kI8KTile,
                     (uint32_t)a.a_rows, CU_TENSOR_MAP_SWIZZLE_128B)) != SVDQ_OK)
    return r;
  if ((r = make_tmap(&tw, Qw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)a.K, (uint64_t)a.N, svdq::kI8KTile,
                     svdq::kI8Cols, CU_TENSOR_MAP_SWIZZLE_128B)) != SVDQ_OK)
    return r;
  const int64_t tiles = (int64_t)((a.N + svdq::kI8Cols - 1) / svdq::kI8Cols) * ((a.M + 127) / 128);
  if (tiles > (1ll << 31) - 1) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "too many tiles");
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = int8_single_config(tiles, splits, st, attr);
  SVDQ_CUDA(cudaLaunchKernelEx(&cfg, svdq::svdq_int8_gemm_kernel<OT>, tx, tw, a));
  return SVDQ_OK;
}

// Launch configuration of the pair kernel: clusters of one pair, or two (SPLIT).
// The attributes are the cluster's size and programmatic stream serialization.
cudaLaunchConfig_t int8_pair_config(int clusters, int ctas, cudaStream_t st, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = pdl_config(ctas * clusters, svdq::kP8Threads, svdq::kP8Bytes, st, attr + 1);
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Clusters of the pair kernel that fit on the device at once (0: none); also
// sets the kernel's shared-memory attribute there.
template <typename OT, bool SPLIT>
int int8_pair_clusters() {
  static std::atomic<int> cache[kMaxDevices];
  return per_device_once(cache, current_device(), [] {
    auto kern = svdq::svdq_int8_gemm_pair_kernel<OT, SPLIT>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, svdq::kP8Bytes) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = int8_pair_config(1, SPLIT ? 4 : 2, nullptr, attr);
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, (void*)kern, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    return n + 1;
  }) - 1;
}

template <typename OT, bool SPLIT>
svdq_status launch_int8_pair(const svdq::Int8GemmArgs& a, const void* Qx, const void* Qw, int clusters,
                             cudaStream_t st) {
  CUtensorMap tx, tw, ty;
  svdq_status r;
  if ((r = make_tmap(&tx, Qx, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)a.K, (uint64_t)a.M, svdq::kI8KTile, 128,
                     CU_TENSOR_MAP_SWIZZLE_128B)) != SVDQ_OK)
    return r;
  if ((r = make_tmap(&tw, Qw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)a.K, (uint64_t)a.N, svdq::kI8KTile, 128,
                     CU_TENSOR_MAP_SWIZZLE_128B)) != SVDQ_OK)
    return r;
  const uint64_t ld = a.M > 1 ? (uint64_t)a.ldy : (uint64_t)a.N;
  // Y by TMA where its rows are whole 16-byte pieces: a store writes the last piece of
  // a row in full, and with it what a wider matrix has behind column N.
  const bool tma_y = ld * sizeof(OT) % 16 == 0 && a.N * sizeof(OT) % 16 == 0;
  memset(&ty, 0, sizeof(ty));
  if (tma_y && (r = make_tmap(&ty, a.y, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)a.N * sizeof(OT), (uint64_t)a.M,
                              128, 32, CU_TENSOR_MAP_SWIZZLE_128B, ld * sizeof(OT))) != SVDQ_OK)
    return r;
  const int64_t tiles = (int64_t)((a.M + 255) / 256) * ((a.N + 255) / 256);
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = int8_pair_config((int)std::min<int64_t>(tiles, clusters), SPLIT ? 4 : 2, st, attr);
  SVDQ_CUDA(cudaLaunchKernelEx(&cfg, svdq::svdq_int8_gemm_pair_kernel<OT, SPLIT>, tx, tw, ty, a, tma_y ? 1 : 0));
  return SVDQ_OK;
}

template <int MT, typename OT>
svdq_status launch_int8_few(const svdq::Int8GemmArgs& a, const void* Qx, const void* Qw, cudaStream_t st) {
  const int warps = svdq::kGvThreads / 32;
  int warps_k = 1;
  while (warps_k < warps && warps_k * 512 < a.K) warps_k *= 2;
  const int channels = svdq::kGvChannels * (warps / warps_k);
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config((a.N + channels - 1) / channels, svdq::kGvThreads, 0, st, attr);
  SVDQ_CUDA(cudaLaunchKernelEx(&cfg, svdq::int8_few_tokens_kernel<MT, OT>, static_cast<const int8_t*>(Qx),
                               static_cast<const int8_t*>(Qw), a, warps_k));
  return SVDQ_OK;
}

// Which kernel serves a product, by estimated microseconds on this GPU. The
// constants are fits to sweeps over M 1..4608, K 1024..13824, N 1024..24576:
//   0.29 us per 128 bytes of K and wave, whatever the tile (see the kernels), or
//   what L2 delivers: 11.7e6 bytes per us over all CTAs (32 KB each of a pair, 48
//   KB of a single one);
//   6.2e6 weight bytes per us where HBM bounds it;
//   a fixed part of 5.7 for CTA pairs, 10.5 with K halved between two pairs, and
//   for single CTAs 5.1 + 0.033 per row of the tile with K whole, 5.0 + 0.055 with
//   K halved, 5.7 + 0.046 with K in quarters, 5.0 + 0.047 in eighths (the cluster's
//   sum).
// Measured, us, pairs against the best single: 16 x 4096 x 4096 15 / 8.8,
// 64 x 4096 x 24576 29 / 23, 128 x 4096 x 4096 15.4 / 13.8, 128 x 4096 x 12288
// 17 / 20, 333 x 1360 x 2304 9.7 / 11.5, 1024 x 4096 x 4096 16 / 22; pairs whole
// against halved: 1396 x 10544 x 1088 35.8 / 26.3, 512 x 4096 x 4096 15.5 / 16.3,
// 1024 x 2048 x 2048 10.6 / 13.5; single CTAs in quarters against eighths: 16 x
// 13824 x 1024 14.3 / 10.5, 178 x 10208 x 380 17.3 / 13.6, 60 x 2048 x 1024 7.7 /
// 7.0 (16 x 4096 x 4096 8.8 / 14: its 16 clusters of eight do not fit at once).
// Single CTAs and halved pairs are considered for one wave only.
template <typename OT>
svdq_status launch_int8_linear(const svdq::Int8GemmArgs& a, const void* Qx, const void* Qw, cudaStream_t st) {
  const int64_t weights = (int64_t)a.N * a.K;
  // Up to 8 tokens: the dot-product kernel. Measured, us, at 4096 x 4096, 4096 x
  // 16384 and 4096 x 24576: one token 4.8, 13.5, 19.5; two 6.0, 14.3, 19.7; four 7.7,
  // 17.6; eight 8.6; the single-CTA kernel (9 tokens, and 5 to 8 from 4096 x 8192 on)
  // 8.0, 17.4, 21.1, which four and eight tokens reach at the sizes below.
  if (a.M <= 2 || (a.M <= 4 && weights <= (1ll << 26)) || (a.M <= 8 && weights <= (1ll << 24))) {
    if (a.M == 1) return launch_int8_few<1, OT>(a, Qx, Qw, st);
    if (a.M == 2) return launch_int8_few<2, OT>(a, Qx, Qw, st);
    if (a.M <= 4) return launch_int8_few<4, OT>(a, Qx, Qw, st);
    return launch_int8_few<8, OT>(a, Qx, Qw, st);
  }
  const double steps = (a.K + svdq::kI8KTile - 1) / svdq::kI8KTile, hbm_us = (double)weights / 6.2e6;
  auto step_us = [](double ctas, double bytes) { return std::max(0.29, ctas * bytes / 11.7e6); };
  const int clusters = int8_pair_clusters<OT, false>();
  const int64_t pairs = (int64_t)((a.M + 255) / 256) * ((a.N + 255) / 256);
  const int64_t tiles = (int64_t)((a.M + 127) / 128) * ((a.N + svdq::kI8Cols - 1) / svdq::kI8Cols);
  if (pairs > (1ll << 30)) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "too many tiles");
  int best = clusters > 0 ? 0 : 1;   // 0: pairs, -1: pairs with K halved, else single CTAs with K split that many ways
  double best_us = 1e30;
  if (clusters > 0)
    best_us = 5.7 + std::max(hbm_us, steps * step_us(2.0 * (double)std::min<int64_t>(pairs, clusters), svdq::kP8StageBytes) *
                                         (double)((pairs + clusters - 1) / clusters));
  if (pairs <= int8_pair_clusters<OT, true>() && steps >= 4) {
    const double us = 10.5 + std::max(hbm_us, steps / 2 * step_us(4.0 * (double)pairs, svdq::kP8StageBytes));
    if (us < best_us) {
      best_us = us;
      best = -1;
    }
  }
  const double rows = (double)std::min(a.M, 128);
  const double fixed[4] = {5.1 + 0.033 * rows, 5.0 + 0.055 * rows, 5.7 + 0.046 * rows, 5.0 + 0.047 * rows};
  for (int i = 0; i < 4; ++i) {
    const int splits = 1 << i;
    if (a.K < 2 * splits * svdq::kI8KTile && splits > 1) break;
    if (tiles > int8_single_tiles<OT>(splits)) break;
    const double us = fixed[i] + std::max(hbm_us, steps / splits * step_us((double)tiles * splits, svdq::kI8StageBytes));
    if (us < best_us) {
      best_us = us;
      best = splits;
    }
  }
  if (best == 0) return launch_int8_pair<OT, false>(a, Qx, Qw, clusters, st);
  if (best == -1) return launch_int8_pair<OT, true>(a, Qx, Qw, (int)pairs, st);
  if (int8_single_tiles<OT>(best) <= 0) return fail(SVDQ_ERR_CUDA, "svdq_int8_gemm_kernel cannot run on this device");
  return launch_int8_single<OT>(a, Qx, Qw, best, st);
}

// ---------------------------------------------------------------- norm
constexpr int64_t kNormMaxC = 16384;

struct NormCall {
  int64_t M, C;
  int dtype, w_dtype;
  int64_t rows_per_group;
  unsigned flags;
};

svdq_status check_norm(const NormCall& n) {
  if (n.M < 0 || n.M > (1ll << 31) - 1 || n.C < 1 || n.C > kNormMaxC)
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "norm of %lld rows of %lld: need 1 <= C <= %lld", (long long)n.M,
                (long long)n.C, (long long)kNormMaxC);
  if (!float_type(n.dtype)) return fail(SVDQ_ERR_INVALID_ARG, "unknown type %d", n.dtype);
  if (n.w_dtype != n.dtype && n.w_dtype != SVDQ_FP32)
    return fail(SVDQ_ERR_INVALID_ARG, "weight and bias have the type of X or fp32");
  if (n.rows_per_group < 0) return fail(SVDQ_ERR_INVALID_ARG, "rows_per_group %lld", (long long)n.rows_per_group);
  if (n.flags & ~(unsigned)SVDQ_NORM_ADD_ONE) return fail(SVDQ_ERR_INVALID_ARG, "unknown flags 0x%x", n.flags);
  return SVDQ_OK;
}

int64_t norm_group_rows(const NormCall& n) {
  return n.rows_per_group == 0 || n.rows_per_group > n.M ? std::max<int64_t>(n.M, 1) : n.rows_per_group;
}
int64_t norm_groups(const NormCall& n) {
  const int64_t rows = norm_group_rows(n);
  return std::max<int64_t>(1, (n.M + rows - 1) / rows);
}

// Whether rows of C values with these strides are whole 16-byte pieces.
bool norm_pieces(const NormCall& n, std::initializer_list<int64_t> strides) {
  const int64_t piece = 16 / type_bytes(n.dtype);
  bool vec = n.C % piece == 0;
  if (n.M > 1)
    for (int64_t ld : strides) vec = vec && ld % piece == 0;
  return vec;
}

// Calls f<T, WT, VEC>.
template <typename F>
svdq_status norm_dispatch(const NormCall& n, bool vec, F&& f) {
  return with_type(n.dtype, [&](auto tag) -> svdq_status {
    auto go = [&](auto wtag) -> svdq_status {
      if (vec) return f(tag, wtag, std::true_type());
      return f(tag, wtag, std::false_type());
    };
    if (n.w_dtype == n.dtype) return go(tag);
    return go(Tag<float>());
  });
}

// Threads per row, and f<pieces per thread, limit of the block's threads>: 16
// values a thread in 16-byte pieces (some lanes of a warp up to 512 values); single
// values, 4 to 16 a thread (up to kNormValues only for the form that ends in codes:
// layernorm_values_kernel has the others).
template <typename T, bool VEC, bool QUANT, typename F>
svdq_status norm_width(int C, F&& f) {
  if constexpr (VEC) {
    constexpr int NV = 16 / svdq::kVecN<T>;
    const int threads = C <= 512 ? team_lanes(C) : round_up((C + 15) / 16, 32);
    return threads <= 256 ? f(threads, Int<NV>(), Int<256>()) : f(threads, Int<NV>(), Int<1024>());
  } else {
    if constexpr (QUANT)
      if (C <= 2048) return f(round_up((C + 3) / 4, 32), Int<4>(), Int<512>());
    if (C <= 8192) return f(round_up((C + 7) / 8, 32), Int<8>(), Int<1024>());
    return f(round_up((C + 15) / 16, 32), Int<16>(), Int<1024>());
  }
}

// Rows of single values up to kNormValues: threads of a row, 4 or 8 values each,
// threads of a block (whole rows side by side), and f<values a thread, threads>.
constexpr int64_t kNormValues = 4096;
int value_lanes(int64_t C) { return C <= 128 ? 32 : round_up((int)(C + 7) / 8, 32); }
int value_limit(int64_t C) { return C <= 2048 ? 256 : 512; }
template <typename F>
svdq_status value_width(int64_t C, F&& f) {
  if (C <= 128) return f(Int<4>(), Int<256>());
  if (C <= 2048) return f(Int<8>(), Int<256>());
  return f(Int<8>(), Int<512>());
}

template <bool QUANT>
svdq_status launch_layernorm(const NormCall& n, svdq::NormArgs a, cudaStream_t st) {
  return norm_dispatch(n, norm_pieces(n, {a.ldx, QUANT ? (int64_t)0 : (int64_t)a.ldy}), [&](auto tag, auto wtag, auto vec) -> svdq_status {
    using T = typename decltype(tag)::type;
    using WT = typename decltype(wtag)::type;
    constexpr bool VEC = decltype(vec)::value;
    if constexpr (VEC) {
      // many rows: the ring (9216 x 4096 26 us, one row per block 54)
      if (n.C > 512 && n.M > 2 * sm_count()) {
        using namespace svdq;
        const size_t row = (size_t)n.C * sizeof(T);
        auto go = [&](auto elems, auto warps) -> svdq_status {
          constexpr int E = decltype(elems)::value, W = decltype(warps)::value;
          return launch_rows<layernorm_rows_kernel<T, WT, E, W, QUANT, false>,
                             layernorm_rows_kernel<T, WT, E, W, QUANT, true>>(a, n.M, n.C, E, row, st);
        };
        if (n.C <= 2048) return go(Int<16>(), Int<4>());
        if (n.C <= 4096) return go(Int<32>(), Int<4>());
        if (n.C <= 8192) return go(Int<32>(), Int<8>());
        return go(Int<32>(), Int<16>());
      }
    }
    if constexpr (!VEC && !QUANT) {
      if (n.C <= kNormValues)
        return value_width(n.C, [&](auto nv, auto maxt) -> svdq_status {
          constexpr int MAXT = decltype(maxt)::value;
          const int64_t groups = norm_groups(n), rows = norm_group_rows(n);
          const int lanes = value_lanes(n.C), teams = (int)std::min<int64_t>(MAXT / lanes, rows);
          const int64_t per_sm = (MAXT > 256 ? MAXT : 3 * MAXT) / (lanes * teams);   // as many as are resident
          a.chunks = (int)std::min<int64_t>(std::max<int64_t>(1, per_sm * sm_count() / groups), (rows + teams - 1) / teams);
          cudaLaunchAttribute attr[1];
          cudaLaunchConfig_t cfg = pdl_config((unsigned)(groups * a.chunks), dim3(lanes, teams), 0, st, attr);
          SVDQ_CUDA(cudaLaunchKernelEx(&cfg, svdq::layernorm_values_kernel<T, WT, decltype(nv)::value, MAXT>, a));
          return SVDQ_OK;
        });
    }
    return norm_width<T, VEC, QUANT>((int)n.C, [&](int threads, auto nv, auto maxt) -> svdq_status {
      constexpr int NV = decltype(nv)::value, MAXT = decltype(maxt)::value;
      const dim3 block(threads, threads <= 32 ? 256 / threads : 1);
      const unsigned grid = (unsigned)std::min<int64_t>((n.M + block.y - 1) / block.y, (int64_t)sm_count() * 16);
      cudaLaunchAttribute attr[1];
      cudaLaunchConfig_t cfg = pdl_config(grid, block, 0, st, attr);
      SVDQ_CUDA(cudaLaunchKernelEx(&cfg, svdq::layernorm_kernel<T, WT, NV, MAXT, VEC, QUANT>, a));
      return SVDQ_OK;
    });
  });
}

// What serves a backward pass: decided here alone, from the type, the width, the
// rows and whether these are whole 16-byte pieces, for the workspace query, the
// check of the workspace and the launch alike.
enum class NormForm {
  kFew,      // layernorm_backward_few_kernel: one launch, no workspace
  kRing,     // layernorm_backward_rows_kernel
  kLanes,    // layernorm_backward_kernel: a row in some lanes of a warp
  kValues,   // layernorm_backward_values_kernel: off 16-byte boundaries
};

struct NormPlan {
  NormForm form;
  int64_t chunks;     // row chunks per group
  size_t workspace;   // bytes of the chunks' partial sums
};

// kFew for few rows, and for rows too wide for single values in registers: it reads
// them twice, instead of two launches and partial sums. Measured, us, few against
// ring (bf16): 32 x 1152 2.7 / 5.6, 226 x 4096 6.2 / 8.1, 226 x 8192 9.3 / 11.8
// (fp32 13.2 / 12.7), 512 x 2048 6.6 / 6.3, 1024 x 1152 9.6 / 8.2; against single
// values: 32 x 1151 3.4 / 7.4, 226 x 1151 fp32 4.7 / 7.7, 400 x 691 6.8 / 7.8,
// 400 x 51 6.2 / 5.2 (one launch and no workspace are 5 us less on the host),
// 2048 x 3001 38 / 23, 4096 x 1151 68 / 18; 16 values a thread, of 1024, without the
// next row's loads: 8192 x 8763 333 / 622.
// Row chunks of the others: over all groups as many blocks per SM as are resident
// at once or, in the ring, blocks of about 640 threads in all (16 channels a
// thread; at the narrower widths the registers hold 512 of these at a time). More groups than that: each block takes a group's rows alone, and no
// partial sums are kept. (Single values: 4 blocks per SM 4133 x 338 14.9 against
// 11.8 us, 14324 x 571 36.0 against 34.6.)
NormPlan norm_backward_plan(const NormCall& n, bool pieces) {
  const int64_t few = n.M <= 256 ? 1ll << 21 : n.M <= 400 ? 1ll << 20 : 0;
  if (n.M * n.C <= few || (!pieces && n.C > kNormValues)) return NormPlan{NormForm::kFew, 1, 0};
  const int64_t groups = norm_groups(n);
  NormForm form = NormForm::kLanes;
  int64_t per_sm = 2;
  if (!pieces) {
    const int lanes = value_lanes(n.C), limit = value_limit(n.C);
    form = NormForm::kValues;
    per_sm = 512 / (limit / lanes * lanes);
  } else if (n.C > 512) {
    form = NormForm::kRing;
    per_sm = std::max<int64_t>(1, 640 / round_up((int)(n.C + 15) / 16, 32));
  }
  const int64_t per = std::max<int64_t>(1, per_sm * sm_count() / groups);
  const int64_t chunks = std::min<int64_t>(per, std::max<int64_t>(1, (norm_group_rows(n) + 3) / 4));
  return NormPlan{form, chunks, chunks == 1 ? 0 : (size_t)(2 * chunks * groups * n.C) * 4u};
}

// The largest workspace over the types and strides that X, dY and dX may have.
size_t norm_workspace_bytes(NormCall n) {
  size_t most = 0;
  for (int dtype : {SVDQ_BF16, SVDQ_FP32}) {   // fp16 is dealt with as bf16
    n.dtype = n.w_dtype = dtype;
    for (bool pieces : {false, norm_pieces(n, {})}) most = std::max(most, norm_backward_plan(n, pieces).workspace);
  }
  return most;
}

// Whether two matrices of a norm share memory.
bool overlap(const void* p, int64_t ldp, const void* q, int64_t ldq, const NormCall& n) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  const uintptr_t es = type_bytes(n.dtype);
  return a < b + ((n.M - 1) * ldq + n.C) * es && b < a + ((n.M - 1) * ldp + n.C) * es;
}

// ---------------------------------------------------------------- rotary positions
template <typename T>
svdq_status launch_rope(svdq::RopeArgs a, bool halves, cudaStream_t st) {
  constexpr int V = svdq::kVecN<T>;
  bool vec = (a.D - a.R) % V == 0 && (halves ? a.R / 2 : a.R) % V == 0 && a.D % V == 0;
  if (a.T > 1) vec = vec && a.xt % V == 0 && a.yt % V == 0;
  if (a.heads > 1) vec = vec && a.xh % V == 0 && a.yh % V == 0;
  // Two waves of resident blocks (4 per SM) at the least: few tokens share their
  // heads among several blocks, many go together, as far as the angle table
  // holds them. 4608 x 48 heads: 22.7, 22.5 and 23.5 us with 4, 8 and 16 per SM.
  const int64_t resident = 8ll * sm_count(), T64 = a.T;
  const int shares = (int)std::min<int64_t>(a.heads, std::max<int64_t>(1, resident / T64));
  a.heads_per_block = (a.heads + shares - 1) / shares;
  a.tokens_per_block = (int)std::max<int64_t>(
      1, std::min<int64_t>((T64 + resident - 1) / resident, (int64_t)svdq::kRopeTable / (a.R / 2)));
  const dim3 grid((unsigned)((T64 + a.tokens_per_block - 1) / a.tokens_per_block),
                  (unsigned)((a.heads + a.heads_per_block - 1) / a.heads_per_block));
  const int items = a.heads_per_block * (vec ? (a.R / (halves ? 2 * V : V) + (a.D - a.R) / V) : a.D - a.R / 2);
  const int threads = std::min(svdq::kRopeThreads, round_up(std::max(items, a.R / 2), 32));
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(grid, threads, 0, st, attr);
  if (halves) {
    if (vec) SVDQ_CUDA(cudaLaunchKernelEx(&cfg, svdq::rope_kernel<T, true, true>, a));
    else SVDQ_CUDA(cudaLaunchKernelEx(&cfg, svdq::rope_kernel<T, true, false>, a));
  } else {
    if (vec) SVDQ_CUDA(cudaLaunchKernelEx(&cfg, svdq::rope_kernel<T, false, true>, a));
    else SVDQ_CUDA(cudaLaunchKernelEx(&cfg, svdq::rope_kernel<T, false, false>, a));
  }
  return SVDQ_OK;
}

// Whether [T][heads][D] with these strides holds every element once.
bool disjoint(int64_t T, int64_t heads, int64_t D, int64_t st, int64_t sh) {
  if (T <= 1) return heads <= 1 || sh >= D;
  if (heads <= 1) return st >= D;
  return (sh >= D && st >= (heads - 1) * sh + D) || (st >= D && sh >= (T - 1) * st + D);
}

}  // namespace

extern "C" {

svdq_status svdq_int8_quantize_act(int64_t M, int64_t K, int x_dtype, const void* X, int64_t ldx,
                                   const float* inv_lambda, void* Qx, float* Sx, void* stream) {
  return int8_quantize(M, K, x_dtype, X, ldx, inv_lambda, Qx, Sx, stream);
}

svdq_status svdq_int8_quantize_weight(int64_t N, int64_t K, int w_dtype, const void* W_lin, int64_t ldw,
                                      const float* lambda, void* Qw, float* Sw, void* stream) {
  return int8_quantize(N, K, w_dtype, W_lin, ldw, lambda, Qw, Sw, stream);
}

svdq_status svdq_int8_linear(int64_t M, int64_t K, int64_t N, const void* Qx, const float* Sx, const void* Qw,
                             const float* Sw, const float* bias, int y_dtype, void* Y, int64_t ldy, void* stream) {
  g_last_error[0] = 0;
  svdq_status r = check_int8_k(M, K);
  if (r != SVDQ_OK) return r;
  if (N < 1 || N > (1ll << 24)) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "int8 linear with N=%lld", (long long)N);
  if (!float_type(y_dtype)) return fail(SVDQ_ERR_INVALID_ARG, "unknown type %d", y_dtype);
  if (!Qw || !Sw || (M > 0 && (!Qx || !Sx || !Y))) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if ((r = check_pointers({Qx, Sx, Qw, Sw, bias, Y})) != SVDQ_OK) return r;
  if ((r = check_rows("Y", M, N, ldy)) != SVDQ_OK) return r;
  if ((r = check_device()) != SVDQ_OK) return r;
  if (M == 0) return SVDQ_OK;
  const svdq::Int8GemmArgs a{Sx, Sw, bias, Y, ldy, (int)M, (int)N, (int)K, 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return with_type(y_dtype, [&](auto tag) -> svdq_status {
    using T = typename decltype(tag)::type;
    return launch_int8_linear<T>(a, Qx, Qw, st);
  });
}

svdq_status svdq_layernorm(int64_t M, int64_t C, int dtype, int w_dtype, const void* X, int64_t ldx,
                           const void* weight, const void* bias, int64_t rows_per_group, float eps,
                           unsigned int flags, void* Y, int64_t ldy, float* mean, float* rstd, void* stream) {
  g_last_error[0] = 0;
  const NormCall n{M, C, dtype, w_dtype, rows_per_group, flags};
  svdq_status r = check_norm(n);
  if (r != SVDQ_OK) return r;
  if (!(eps >= 0.f)) return fail(SVDQ_ERR_INVALID_ARG, "eps must be >= 0");
  if (M > 0 && (!X || !Y)) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if ((r = check_pointers({X, weight, bias, Y, mean, rstd})) != SVDQ_OK) return r;
  if ((r = check_rows("X", M, C, ldx)) != SVDQ_OK || (r = check_rows("Y", M, C, ldy)) != SVDQ_OK ||
      (r = check_in_place("Y", Y, ldy, X, ldx, M)) != SVDQ_OK)
    return r;
  if ((r = check_device()) != SVDQ_OK) return r;
  if (M == 0) return SVDQ_OK;
  svdq::NormArgs a = {};
  a.x = X; a.ldx = ldx; a.w = weight; a.b = bias; a.mean = mean; a.rstd = rstd;
  a.M = M; a.rows_per_group = norm_group_rows(n); a.C = (int)C; a.eps = eps;
  a.add = flags & SVDQ_NORM_ADD_ONE ? 1.f : 0.f;
  a.y = Y; a.ldy = ldy;
  return launch_layernorm<false>(n, a, static_cast<cudaStream_t>(stream));
}

svdq_status svdq_int8_layernorm_quantize(int64_t M, int64_t C, int dtype, int w_dtype, const void* X, int64_t ldx,
                                         const void* weight, const void* bias, int64_t rows_per_group, float eps,
                                         unsigned int flags, const float* inv_lambda, void* Qx, float* Sx,
                                         void* stream) {
  g_last_error[0] = 0;
  const NormCall n{M, C, dtype, w_dtype, rows_per_group, flags};
  svdq_status r = check_norm(n);
  if (r != SVDQ_OK) return r;
  if (C % 16) return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "C=%lld must be a multiple of 16", (long long)C);
  if (!(eps >= 0.f)) return fail(SVDQ_ERR_INVALID_ARG, "eps must be >= 0");
  if (M > 0 && (!X || !Qx || !Sx)) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if ((r = check_pointers({X, weight, bias, inv_lambda, Qx, Sx})) != SVDQ_OK) return r;
  if ((r = check_rows("X", M, C, ldx)) != SVDQ_OK) return r;
  if ((r = check_device()) != SVDQ_OK) return r;
  if (M == 0) return SVDQ_OK;
  svdq::NormArgs a = {};
  a.x = X; a.ldx = ldx; a.w = weight; a.b = bias;
  a.M = M; a.rows_per_group = norm_group_rows(n); a.C = (int)C; a.eps = eps;
  a.add = flags & SVDQ_NORM_ADD_ONE ? 1.f : 0.f;
  a.inv_lambda = inv_lambda; a.q = static_cast<int8_t*>(Qx); a.s = Sx;
  return launch_layernorm<true>(n, a, static_cast<cudaStream_t>(stream));
}

svdq_status svdq_layernorm_backward_workspace(int64_t M, int64_t C, int64_t rows_per_group, size_t* bytes) {
  g_last_error[0] = 0;
  const NormCall n{M, C, SVDQ_FP32, SVDQ_FP32, rows_per_group, 0};
  svdq_status r = check_norm(n);
  if (r != SVDQ_OK) return r;
  if (!bytes) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  *bytes = norm_workspace_bytes(n);
  return SVDQ_OK;
}

svdq_status svdq_layernorm_backward(int64_t M, int64_t C, int dtype, int w_dtype, const void* dY, int64_t lddy,
                                    const void* X, int64_t ldx, const void* weight, const float* mean,
                                    const float* rstd, int64_t rows_per_group, unsigned int flags, void* dX,
                                    int64_t lddx, float* dweight, float* dbias, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  g_last_error[0] = 0;
  const NormCall n{M, C, dtype, w_dtype, rows_per_group, flags};
  svdq_status r = check_norm(n);
  if (r != SVDQ_OK) return r;
  if (M > 0 && (!dY || !X || !mean || !rstd || !dX)) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if ((r = check_pointers({dY, X, weight, mean, rstd, dX, dweight, dbias, workspace})) != SVDQ_OK) return r;
  if ((r = check_rows("dY", M, C, lddy)) != SVDQ_OK || (r = check_rows("X", M, C, ldx)) != SVDQ_OK ||
      (r = check_rows("dX", M, C, lddx)) != SVDQ_OK || (r = check_in_place("dX", dX, lddx, dY, lddy, M)) != SVDQ_OK ||
      (r = check_in_place("dX", dX, lddx, X, ldx, M)) != SVDQ_OK)
    return r;
  const bool sums = dweight || dbias;
  const bool pieces = norm_pieces(n, {lddy, ldx, lddx});
  const NormPlan plan = norm_backward_plan(n, pieces);
  const size_t need = sums ? plan.workspace : 0;
  if (need && (!workspace || workspace_bytes < need))
    return fail(SVDQ_ERR_BUFFER_TOO_SMALL, "workspace of %zu bytes, need %zu", workspace ? workspace_bytes : 0, need);
  if ((r = check_device()) != SVDQ_OK) return r;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (M == 0) {   // the sums over no rows
    if (dweight) SVDQ_CUDA(cudaMemsetAsync(dweight, 0, (size_t)C * 4, st));
    if (dbias) SVDQ_CUDA(cudaMemsetAsync(dbias, 0, (size_t)C * 4, st));
    return SVDQ_OK;
  }
  svdq::NormArgs a = {};
  a.x = X; a.ldx = ldx; a.w = weight; a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
  a.M = M; a.rows_per_group = norm_group_rows(n); a.C = (int)C;
  a.add = flags & SVDQ_NORM_ADD_ONE ? 1.f : 0.f;
  a.dy = dY; a.lddy = lddy; a.dx = dX; a.lddx = lddx; a.dw = dweight; a.db = dbias;
  a.chunks = (int)plan.chunks;
  a.part = need ? static_cast<float*>(workspace) : nullptr;
  const int64_t groups = norm_groups(n);
  // The few-rows form, in one launch; dX in the memory of an input: the sums come
  // first, in a launch of their own.
  auto few = [&](auto tag, auto wtag, auto vec) -> svdq_status {
    auto kern = svdq::layernorm_backward_few_kernel<typename decltype(tag)::type, typename decltype(wtag)::type,
                                                    decltype(vec)::value>;
    const bool in_place = sums && (overlap(dX, lddx, dY, lddy, n) || overlap(dX, lddx, X, ldx, n));
    const int rows = (int)(C <= 1024 ? (M + svdq::kNormFewThreads / 32 - 1) / (svdq::kNormFewThreads / 32) : M);
    a.strip_blocks = sums ? (int)(groups * ((C + 31) / 32)) : 0;
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = pdl_config(in_place ? a.strip_blocks : a.strip_blocks + rows, svdq::kNormFewThreads, 0, st, attr);
    SVDQ_CUDA(cudaLaunchKernelEx(&cfg, kern, a));
    if (in_place) {
      a.first_block = a.strip_blocks;
      cfg.gridDim = dim3(rows);
      SVDQ_CUDA(cudaLaunchKernelEx(&cfg, kern, a));
    }
    return SVDQ_OK;
  };
  r = norm_dispatch(n, pieces, [&](auto tag, auto wtag, auto vec) -> svdq_status {
    using T = typename decltype(tag)::type;
    using WT = typename decltype(wtag)::type;
    constexpr bool VEC = decltype(vec)::value;
    if (plan.form == NormForm::kFew) return few(tag, wtag, vec);
    if constexpr (VEC) {
      if (plan.form == NormForm::kRing) {
        using namespace svdq;
        const size_t rows = 2 * (size_t)n.C * sizeof(T);
        auto go = [&](auto elems, auto warps, auto blocks, auto hold, auto full) -> svdq_status {
          constexpr int E = decltype(elems)::value;
          constexpr auto kern = layernorm_backward_rows_kernel<T, WT, E, decltype(warps)::value, decltype(blocks)::value,
                                                               decltype(hold)::value, decltype(full)::value>;
          const int threads = round_up(((int)n.C + E - 1) / E, 32);
          a.depth = ring_depth(threads, rows, (size_t)n.C * 4);
          const size_t smem = a.depth * rows + (size_t)n.C * 4;
          ring_blocks_per_sm<kern>(threads, smem);   // sets the attribute
          cudaLaunchAttribute attr[1];
          cudaLaunchConfig_t cfg = pdl_config((unsigned)(groups * a.chunks), threads, smem, st, attr);
          SVDQ_CUDA(cudaLaunchKernelEx(&cfg, kern, a));
          return SVDQ_OK;
        };
        auto size = [&](auto elems, auto warps, auto blocks, auto hold) -> svdq_status {
          if (n.C % (32 * decltype(elems)::value) == 0) return go(elems, warps, blocks, hold, std::true_type());
          return go(elems, warps, blocks, hold, std::false_type());
        };
        if (n.C <= 4096) return size(Int<16>(), Int<8>(), Int<2>(), std::true_type());
        if (n.C <= 5120) return size(Int<16>(), Int<10>(), Int<2>(), std::true_type());
        if (n.C <= 8192) return size(Int<16>(), Int<16>(), Int<1>(), std::true_type());
        return size(Int<32>(), Int<16>(), Int<1>(), std::false_type());
      }
    }
    cudaLaunchAttribute attr[1];
    auto go = [&](auto kern, int threads, int limit) -> svdq_status {
      const dim3 block(threads, limit / threads);
      const size_t smem = (size_t)block.y * n.C * 4;   // at most 16 KB: the teams' sums
      cudaLaunchConfig_t cfg = pdl_config((unsigned)(groups * a.chunks), block, smem, st, attr);
      SVDQ_CUDA(cudaLaunchKernelEx(&cfg, kern, a));
      return SVDQ_OK;
    };
    if constexpr (VEC) {   // kLanes: 16 values each
      return go(svdq::layernorm_backward_kernel<T, WT, 16 / svdq::kVecN<T>, 256>, team_lanes((int)n.C), 256);
    } else {               // kValues: warps, 4 or 8 a thread
      return value_width(n.C, [&](auto nv, auto maxt) {
        constexpr int MAXT = decltype(maxt)::value;
        return go(svdq::layernorm_backward_values_kernel<T, WT, decltype(nv)::value, MAXT>, value_lanes(n.C), MAXT);
      });
    }
  });
  if (r != SVDQ_OK || !a.part) return r;
  const int64_t cols = groups * C;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)((cols + 31) / 32), 2), 32 * svdq::kPartWarps, 0, st, attr);
  SVDQ_CUDA(cudaLaunchKernelEx(&cfg, svdq::layernorm_partials_kernel, static_cast<const float*>(a.part), dweight,
                               dbias, (long long)cols, a.chunks));
  return SVDQ_OK;
}

svdq_status svdq_rope(int64_t T, int32_t heads, int32_t D, int dtype, const void* X, int64_t x_token_stride,
                      int64_t x_head_stride, void* Y, int64_t y_token_stride, int64_t y_head_stride,
                      const void* positions, int pos_dtype, int64_t pos_rows, int32_t axes, const int32_t* axis_dims,
                      const double* freqs, unsigned int flags, void* stream) {
  g_last_error[0] = 0;
  if (T < 0 || T > (1ll << 31) - 1 || heads < 0 || heads > 65535 || D < 2 || D > svdq::kRopeMaxD || D % 2)
    return fail(SVDQ_ERR_UNSUPPORTED_SHAPE, "rope T=%lld heads=%d D=%d: need an even D in [2, %d]", (long long)T,
                (int)heads, (int)D, svdq::kRopeMaxD);
  if (!float_type(dtype)) return fail(SVDQ_ERR_INVALID_ARG, "unknown type %d", dtype);
  if (pos_dtype != SVDQ_INT32 && pos_dtype != SVDQ_FP32) return fail(SVDQ_ERR_INVALID_ARG, "positions are int32 or fp32");
  if (flags & ~(unsigned)(SVDQ_ROPE_HALVES | SVDQ_ROPE_INVERSE)) return fail(SVDQ_ERR_INVALID_ARG, "unknown flags 0x%x", flags);
  if (axes < 1 || axes > svdq::kRopeMaxAxes || !axis_dims)
    return fail(SVDQ_ERR_INVALID_ARG, "axes=%d: need 1 to %d of them", (int)axes, svdq::kRopeMaxAxes);
  svdq::RopeArgs a = {};
  int64_t R = 0;
  for (int i = 0; i < axes; ++i) {
    if (axis_dims[i] < 2 || axis_dims[i] % 2 || axis_dims[i] > D)
      return fail(SVDQ_ERR_INVALID_ARG, "axis %d has %d elements: need an even number of at least 2", i, (int)axis_dims[i]);
    R += axis_dims[i];
    a.axis_end[i] = (int)(R / 2);
  }
  for (int i = axes; i < svdq::kRopeMaxAxes; ++i) a.axis_end[i] = svdq::kRopeMaxD;
  if (R > D) return fail(SVDQ_ERR_INVALID_ARG, "the axes have %lld elements, a head has %d", (long long)R, (int)D);
  const bool any = T > 0 && heads > 0;
  if (any && (!X || !Y || !positions || !freqs)) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  svdq_status r;
  if ((r = check_pointers({X, Y, positions, freqs})) != SVDQ_OK) return r;
  if (any && (pos_rows < 1 || T % pos_rows))
    return fail(SVDQ_ERR_INVALID_ARG, "%lld tokens with %lld rows of positions", (long long)T, (long long)pos_rows);
  for (int64_t s : {x_token_stride, x_head_stride, y_token_stride, y_head_stride})
    if (any && (s < 0 || s > (1ll << 40))) return fail(SVDQ_ERR_INVALID_ARG, "stride %lld", (long long)s);
  if (any && !disjoint(T, heads, D, y_token_stride, y_head_stride))
    return fail(SVDQ_ERR_INVALID_ARG, "the heads of Y overlap");
  if (any && X == Y && ((T > 1 && x_token_stride != y_token_stride) || (heads > 1 && x_head_stride != y_head_stride)))
    return fail(SVDQ_ERR_INVALID_ARG, "in place, X and Y have the same strides");
  if ((r = check_device()) != SVDQ_OK) return r;
  if (!any) return SVDQ_OK;
  a.x = X; a.y = Y; a.xt = x_token_stride; a.xh = x_head_stride; a.yt = y_token_stride; a.yh = y_head_stride;
  a.pos = positions; a.freq = freqs; a.T = (int)T; a.pos_rows = (int)pos_rows; a.heads = heads; a.D = D; a.R = (int)R;
  a.axes = axes; a.pos_fp32 = pos_dtype == SVDQ_FP32; a.inverse = (flags & SVDQ_ROPE_INVERSE) != 0;
  return with_type(dtype, [&](auto tag) -> svdq_status {
    using E = typename decltype(tag)::type;
    return launch_rope<E>(a, (flags & SVDQ_ROPE_HALVES) != 0, static_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
