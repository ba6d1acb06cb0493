// Streams rows through shared memory for kernels whose block works on one row
// at a time: a ring of stages, each one row (or one row of each of several
// matrices), filled ahead by bulk copies. What a block has in flight is then
// set by the ring and not by how many blocks its registers leave room for.
//
// A stage needs no "empty" barrier: every row passes a barrier of the block
// (its reduction) after all threads have read the stage into registers, and
// the thread that issues the copies refills the stage behind that barrier.
#pragma once

#include "svdq_int4.cuh"   // add2_rn, fma2_rn
#include "svdq_ptx.cuh"
#include "svdq_quant.cuh"  // mul2_rn
#include "svdq_vec.cuh"

namespace svdq {

constexpr int kRingMaxStages = 8;

// MATS matrices with the same row size: row_bytes, the row addresses and the
// strides are multiples of 16.
template <int MATS>
struct RowRing {
  unsigned char* stages;          // [depth][MATS][row_bytes]
  uint64_t* full;                 // [depth]
  const unsigned char* base[MATS];
  long long ld[MATS];             // row strides in bytes
  uint32_t row_bytes;
  int depth;

  // Thread 0, before a __syncthreads().
  __device__ void init() {
    for (int s = 0; s < depth; ++s) mbar_init(full + s, 1);
    fence_mbar_init();
  }
  // Thread 0: start the copies of row m into `stage`.
  __device__ void fetch(int stage, long long m) {
    mbar_arrive_expect_tx(full + stage, MATS * row_bytes);
#pragma unroll
    for (int i = 0; i < MATS; ++i)
      bulk_load(stages + ((size_t)stage * MATS + i) * row_bytes, base[i] + m * ld[i], row_bytes, full + stage);
  }
  // Every thread: wait for the stage's row. A wait that gives up has recorded
  // the device error; the caller goes on (with what the stage holds), so that
  // the block's barriers stay matched, and every later wait returns at once.
  __device__ void wait(int stage, uint32_t parity) { mbar_wait(full + stage, parity, kDevErrTimeoutFull); }
  // Thread 0, at the end: after a wait that gave up, a time that no copy in flight
  // can outlast, before the block's shared memory goes.
  __device__ void leave() {
    if (!device_error_set()) return;
    const unsigned long long t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
  }
};

// A 16-byte piece as pairs of fp32, and back.
template <typename T>
__device__ __forceinline__ void unpack_pairs(const uint4& r, float2 (&f)[kVecN<T> / 2]) {
  float t[kVecN<T>];
  unpack_vec<T>(r, t);
#pragma unroll
  for (int i = 0; i < kVecN<T> / 2; ++i) f[i] = make_float2(t[2 * i], t[2 * i + 1]);
}

template <typename T>
__device__ __forceinline__ uint4 pack_pairs(const float2 (&f)[kVecN<T> / 2]) {
  float t[kVecN<T>];
#pragma unroll
  for (int i = 0; i < kVecN<T> / 2; ++i) {
    t[2 * i] = f[i].x;
    t[2 * i + 1] = f[i].y;
  }
  return pack_vec<T>(t);
}

template <typename WT, int N>
__device__ __forceinline__ void load_pairs(const WT* p, float2 (&f)[N / 2]) {
  float t[N];
  load_params<WT, N>(p, t);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) f[i] = make_float2(t[2 * i], t[2 * i + 1]);
}

__device__ __forceinline__ float2 pair(float v) { return make_float2(v, v); }

// Sums of a and b over a warp in five shuffles: the half-warps take one each.
// Lanes 0-15 end with the sum of a, lanes 16-31 with the sum of b.
__device__ __forceinline__ float warp_sum_halves(float a, float b, int lane) {
  const bool hi = (lane & 16) != 0;
  float v = hi ? b : a;
  v += __shfl_xor_sync(0xFFFFFFFFu, hi ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// The largest |v| of a warp, NaN if any is.
__device__ __forceinline__ float warp_amax_nan(float v) {
  float r;
  asm volatile("redux.sync.max.abs.NaN.f32 %0, %1, 0xFFFFFFFF;" : "=f"(r) : "f"(v));
  return r;
}

// max(|a|, |b|, |c|), NaN if any is.
__device__ __forceinline__ float amax3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

}  // namespace svdq
