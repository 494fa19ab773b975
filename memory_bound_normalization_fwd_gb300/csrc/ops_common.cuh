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

// Columns t, t + T, ... of a row of N elements starting at element `base`, zero past
// the row's end. Every load is made (the last column again past the end), so that
// none waits for another.
template <int DT, int V>
__device__ __forceinline__ void load_columns(const void* p, int64_t base, int t, int T, int N, float (&out)[V]) {
    const typename Elem<DT>::T* q = static_cast<const typename Elem<DT>::T*>(p) + base;
    typename Elem<DT>::T raw[V];
#pragma unroll
    for (int v = 0; v < V; ++v) raw[v] = q[min(v * T + t, N - 1)];
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = v * T + t < N ? Elem<DT>::load(raw[v]) : 0.f;
}

// Pairs of fp32 values for the packed instructions of sm_100 and later
// (mul/add/fma.rn.f32x2: each half rounded as the scalar instruction would be),
// half the instructions of scalar code.
using f2 = uint64_t;

__device__ __forceinline__ f2 f2_make(float a, float b) {
    f2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ f2 f2_dup(float a) { return f2_make(a, a); }
__device__ __forceinline__ float2 f2_get(f2 d) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
    return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ float f2_sum(f2 a) {
    const float2 v = f2_get(a);
    return v.x + v.y;
}

// A 16-byte vector as pairs, and back (one rounding to the dtype).
template <int DT>
__device__ __forceinline__ void unpack2(const uint4& v, f2* o) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (DT == kFP32) {
        o[0] = f2_make(__uint_as_float(w[0]), __uint_as_float(w[1]));
        o[1] = f2_make(__uint_as_float(w[2]), __uint_as_float(w[3]));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = Codec<DT>::unpack2(w[k]);
            o[k] = f2_make(f.x, f.y);
        }
    }
}
template <int DT>
__device__ __forceinline__ uint4 pack2(const f2* o) {
    if constexpr (DT == kFP32) {
        const float2 a = f2_get(o[0]), b = f2_get(o[1]);
        return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x),
                          __float_as_uint(b.y));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 a = f2_get(o[k]);
            w[k] = Codec<DT>::pack2(a.x, a.y);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}
// offset + w of a vector of weights, as pairs.
template <int DT>
__device__ __forceinline__ void weights2(const uint4& v, float offset, f2* o) {
    unpack2<DT>(v, o);
#pragma unroll
    for (int k = 0; k < VecElems<DT>::value / 2; ++k) o[k] = f2_add(o[k], f2_dup(offset));
}

}  // namespace rmsn
