// State rows of a batch of requests: which row of the pool request b may update.
#pragma once

#include "moe_internal.h"

namespace moe {

// Row of the pool for request b, or -1 to skip it: a padding row (-1), a row out of range, or
// one that an earlier request of the batch has already named (two blocks would race on its
// state); the last two are reported.  Called by whole blocks, every thread with the same b.
__device__ __forceinline__ int claimed_slot(int b, const int* slot, int n_slots,
                                            int* dev_status) {
  if (!slot) return b;
  const int row = slot[b];
  if (row == -1) return -1;
  int bad = row < 0 || row >= n_slots;
  if (!bad)
    for (int i = threadIdx.x; i < b; i += blockDim.x) bad |= slot[i] == row;
  bad = __syncthreads_or(bad);
  if (!bad) return row;
  if (threadIdx.x == 0 && dev_status) atomicCAS(dev_status, 0, MOE_ERR_BAD_INDEX);
  return -1;
}

}  // namespace moe
