// state_bytes.h -- how much of a run the reordering of states moves; plain arithmetic, for the device and the host.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define SPEC_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SPEC_HOST_DEVICE inline
#endif

namespace specstate {

// The bytes of the first `length` of a run's T positions.  The product is below the run where it is taken: a state
// without positions is one position of any size, and "all" is a length of 2^31 - 1.
SPEC_HOST_DEVICE int64_t moved_bytes(int64_t run, int64_t unit, int32_t T, int32_t length) {
    return length >= T ? run : static_cast<int64_t>(length) * unit;
}

}  // namespace specstate
