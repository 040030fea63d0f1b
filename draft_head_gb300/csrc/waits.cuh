// Waits of the target-side kernels beside those of common.cuh.
#pragma once

#include "common.cuh"

namespace domino {

// Before the memory that an asynchronous operation reads or writes is given up: waits for one that is in flight and needs
// nobody else to end. Its limit is its own, as the caller's may be shorter than a copy.
__device__ __forceinline__ void mbar_land(uint64_t* bar, uint32_t parity, Ctl* ctl) {
  mbar_wait(bar, parity, nullptr, ctl, 2000000000ull);
}

}  // namespace domino
