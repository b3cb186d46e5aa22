// pipeline.cuh — what the warps of the tensor-core attention kernels share:
// warp-wide bounded waits, ring positions, and block ids read 32 at a time.
#pragma once

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr uint32_t kFull = 0xffffffffu;

// Wait with every lane of the warp; the result is the same for all lanes.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(kFull, mbar_wait(bar, parity));
}

// Running position in an N-slot ring: slot and phase parity.
template <int N>
struct Ring {
  int idx = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next() {
    if (++idx == N) {
      idx = 0;
      ph ^= 1u;
    }
  }
};

// Block ids of a table row, 32 at a time across the lanes of a warp.
struct BlockIds {
  int chunk = -1;
  int mine = 0;
  // Block id of table entry blk; every lane of the warp calls this together.
  __device__ __forceinline__ int get(const int32_t* table, int limit, int blk, int lane,
                                     int64_t num_blocks, unsigned* err) {
    if ((blk >> 5) != chunk) {
      chunk = blk >> 5;
      const int bi = chunk * 32 + lane;
      mine = bi < limit ? __ldg(table + bi) : 0;
    }
    int id = __shfl_sync(kFull, mine, blk & 31);
    if (id < 0 || id >= num_blocks) {
      if (lane == 0) record_error(err, kErrIndex);
      id = 0;   // never form an out-of-range address
    }
    return id;
  }
};

}  // namespace pkv
