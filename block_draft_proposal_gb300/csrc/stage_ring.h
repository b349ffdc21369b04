// Blocks through a ring of shared-memory stages: block k uses stage k % stages for the
// (k / stages)-th time.  Plain C++, so that a host program can check the arithmetic.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define DFLASH2_RING __host__ __device__ __forceinline__
#else
#define DFLASH2_RING inline
#endif

namespace dflash2 {

// The parity of a stage's barrier while block k's use of it is not complete.
DFLASH2_RING uint32_t ring_parity(uint32_t k, uint32_t stages) { return (k / stages) & 1u; }

// A producer of blocks first, first + step, ... (below `end`, as all the ring's blocks are):
// the first of its blocks whose stage no later block takes.  It and those after it are
// the uses that no producer has waited for when its loop ends.
DFLASH2_RING uint32_t ring_last_uses(uint32_t first, uint32_t step, uint32_t end, uint32_t stages) {
    const uint32_t from = end > stages ? end - stages : 0;
    return from <= first ? first : first + (from - first + step - 1) / step * step;
}

}  // namespace dflash2
