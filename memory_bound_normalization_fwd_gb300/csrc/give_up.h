// How the threads of a row team agree to give up. Plain C++: the kernels keep it
// in shared memory, a host test explores its interleavings.
//
// A thread whose bounded wait for a row runs out marks that row; behind the
// row's team barrier every thread reads the mark and leaves the loop, or goes on.
// With one barrier per row a fast thread may already be waiting for row r + 1 when
// a slow one reads the mark of row r, so a row's mark must not be seen at the row
// before it: the slow thread would leave while the fast one waits for it at the
// barrier of row r + 1. Two flags, taken by turns, are enough: no thread is two
// rows ahead of another, as the barrier of row r + 1 lies between.
#pragma once

#if defined(__CUDACC__)
#define RMSN_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define RMSN_HOST_DEVICE inline
#endif

namespace rmsn {

struct GiveUp {
    volatile unsigned int late[2];

    RMSN_HOST_DEVICE void clear() { late[0] = late[1] = 0; }
    // Before row's barrier, or behind the barrier of the row before it.
    RMSN_HOST_DEVICE void mark(int row) { late[row & 1] = 1; }
    // Between row's barrier and the next row's: the same for every thread.
    RMSN_HOST_DEVICE bool at(int row) const { return late[row & 1] != 0; }
};

}  // namespace rmsn
