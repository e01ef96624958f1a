// State rows of a batch of requests: which row of the pool request b may update.
#pragma once

#include "moe_internal.h"

namespace moe {

// Whether an earlier request of the batch has already named request b's row: two blocks would race
// on its state.  That is reported.  Called by whole blocks, every thread with the same b.
__device__ __forceinline__ bool named_before(int b, int row, const int* slot, int* dev_status) {
  int bad = 0;
  for (int i = threadIdx.x; i < b; i += blockDim.x) bad |= slot[i] == row;
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0 && dev_status) atomicCAS(dev_status, 0, MOE_ERR_BAD_INDEX);
  return bad;
}

}  // namespace moe
