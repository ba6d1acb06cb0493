// Streams rows through shared memory for kernels whose block works on one row
// at a time: a ring of stages, each one row (or one row of each of several
// matrices), filled ahead by bulk copies. What a block has in flight is then
// set by the ring and not by how many blocks its registers leave room for.
//
// A stage needs no "empty" barrier: every row passes a barrier of the block
// (its reduction) after all threads have read the stage into registers, and
// the thread that issues the copies refills the stage behind that barrier.
#pragma once

#include "svdq_ptx.cuh"
#include "svdq_vec.cuh"

namespace svdq {

constexpr int kRingMaxStages = 8;

// MATS matrices with the same row size; `bytes` of a row is a multiple of 16,
// and so are the row addresses.
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
  __device__ const unsigned char* row(int stage, int mat) const {
    return stages + ((size_t)stage * MATS + mat) * row_bytes;
  }
};

// Elements a thread holds of a row in these kernels, and the pieces they are.
constexpr int kRowElems = 16;
template <typename T>
inline constexpr int kRowPieces = kRowElems / kVecN<T>;

}  // namespace svdq
