// ring.h -- the order of a ring's slots, free of device code: a copy per slot, an
// mbarrier phase per copy.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define MSS_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MSS_HOST_DEVICE inline
#endif

namespace mss {

// After a wait that gave up: wait(k, slot, parity) for the `count` copies in
// flight, k from 0 on in the order they were issued.  The first is the one whose
// wait ran out, in `slot` under `parity`: it may still arrive, and no block may
// leave or use the ring's memory for something else before.
template <typename Wait>
MSS_HOST_DEVICE void drain_ring(int slot, uint32_t parity, int stages, int count, Wait&& wait) {
    for (int k = 0; k < count; ++k) {
        wait(k, slot, parity);
        if (++slot == stages) slot = 0, parity ^= 1;
    }
}

}  // namespace mss
