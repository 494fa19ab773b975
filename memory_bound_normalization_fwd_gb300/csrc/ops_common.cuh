// Device helpers shared by the block, rope and cache kernels.
#pragma once

#include "common.cuh"

namespace rmsn {

// Sums of K values over the block, in a fixed order: warp butterfly, then the
// warps' sums in order. `part` holds 2 * K * 32 floats; `parity` alternates
// between calls, so one barrier per call is enough.
template <int K>
__device__ __forceinline__ void block_sums(float (&v)[K], float* part, int& parity) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
    }
    const int warps = blockDim.x >> 5;
    if (warps == 1) return;
    float* slot = part + parity * K * 32;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) slot[k * 32 + (threadIdx.x >> 5)] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        float t = 0.f;
        for (int q = 0; q < warps; ++q) t += slot[k * 32 + q];
        v[k] = t;
    }
    parity ^= 1;
}

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
    return Elem<DT>::load(static_cast<const typename Elem<DT>::T*>(p)[i]);
}

template <int DT>
__device__ __forceinline__ void store1(void* p, int64_t i, float f) {
    static_cast<typename Elem<DT>::T*>(p)[i] = Elem<DT>::store(f);
}

}  // namespace rmsn
