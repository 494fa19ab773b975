// The quantised cache: k and v written into its slots in 8 or 4 bits with one
// power-of-two scale for 32 values, and read back by page table (the
// operations are stated in include/rmsnorm.h).
//
// A power of two as the scale makes both directions exact but for the one
// rounding to the format: x / scale is x * 2^-k in fp32, and code * scale is a
// value of every activation type within its range. So the codes are a function
// of the values alone, whatever the order of the arithmetic.
#include "rmsnorm.h"

#include "ops.h"
#include "ops_common.cuh"
#include "row_ring_host.h"

#include <algorithm>

#include <cuda_fp4.h>
#include <cuda_fp8.h>

namespace rmsn {

// Bit 0: an index was out of range since the last read. One word per device.
__device__ unsigned int g_cache_status;

namespace {

constexpr int kGroup = 32;

// The scale byte of a group whose largest magnitude has these bits (fp32):
// for the largest value L = (1 + f) 2^e of the format, the smallest k with
// amax <= L 2^k is amax's exponent - e, plus one where its fraction exceeds f.
template <int F>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    constexpr uint32_t top = F == RMSNORM_CACHE_E4M3 ? 0x600000u : 0x400000u;
    constexpr int e = F == RMSNORM_CACHE_E4M3 ? 8 : 2;
    if (amax >= 0x7f800000u) return 255u;
    const int k = static_cast<int>(amax >> 23) - e + ((amax & 0x7fffffu) > top ? 1 : 0);
    return k < 0 ? 0u : static_cast<uint32_t>(k);
}

// 1 / scale. A byte is at most 254 - 8 for finite values, so this is normal;
// a group with scale byte 255 takes 0 (its codes are not looked at).
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
    return byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float scale_of(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7fc00000u)
                        : __uint_as_float(byte ? byte << 23 : 0x400000u);
}

__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t to_e2m1x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp4x2(make_float2(lo, hi), __NV_E2M1, cudaRoundNearest);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
    return __half22float2(
        static_cast<__half2>(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3)));
}
__device__ __forceinline__ float2 from_e2m1x2(uint32_t c) {
    return __half22float2(
        static_cast<__half2>(__nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(c), __NV_E2M1)));
}

// Index of (slot, head) among the cache's heads.
__device__ __forceinline__ int64_t cache_head(const CacheP& p, int64_t slot, int h) {
    if (!p.heads_first) return slot * p.heads + h;
    const int64_t page = slot / p.page_size;
    return (page * p.heads + h) * p.page_size + (slot - page * p.page_size);
}

// The sequence whose rows hold row i: the last b with cu_rows[b] <= i.
__device__ __forceinline__ int64_t sequence_of(const CacheP& p, int64_t i) {
    int64_t lo = 0, hi = p.sequences - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (p.cu_rows[mid] <= i) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The slot of row i: -1 for a row behind the last sequence, -2 for one whose
// page is not there.
__device__ __forceinline__ int64_t read_slot(const CacheP& p, int64_t i) {
    if (p.sequences <= 0 || i >= p.cu_rows[p.sequences]) return -1;
    const int64_t b = sequence_of(p, i);
    const int64_t pos = i - p.cu_rows[b] + (p.starts ? p.starts[b] : 0);
    if (pos < 0) return -2;
    const int64_t col = pos / p.page_size;
    if (col >= p.table_width) return -2;
    const int64_t slot = p.table[b * p.table_width + col] * p.page_size + (pos - col * p.page_size);
    return slot < 0 || slot >= p.slots ? -2 : slot;
}

// Element-wise kernels: any head size, alignment and stride; a thread takes one
// group of one head of one token.
template <int DT, int F>
__global__ void __launch_bounds__(256) cache_write_generic_kernel(const CacheP p) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t units = p.T * p.heads * p.groups;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; u < units; u += step) {
        const int64_t t = u / (p.heads * p.groups);
        const int rest = static_cast<int>(u - t * (p.heads * p.groups));
        const int h = rest / p.groups, g = rest - h * p.groups;
        const int64_t slot = p.slot[t];
        if (slot < 0) continue;
        if (slot >= p.slots) {
            if (rest == 0) atomicOr(&g_cache_status, 1u);
            continue;
        }
        const int64_t head = cache_head(p, slot, h);
        const int j0 = g * kGroup, n = p.D - j0 < kGroup ? p.D - j0 : kGroup;
        for (int k = 0; k < 2; ++k) {
            if (!p.codes[k]) continue;
            const int64_t x0 = t * p.t[k].st + h * p.t[k].sh + j0;
            uint32_t amax = 0;
            for (int j = 0; j < n; ++j) {
                const uint32_t m = __float_as_uint(load1<DT>(p.t[k].p, x0 + j)) & 0x7fffffffu;
                amax = m > amax ? m : amax;
            }
            const uint32_t byte = scale_byte<F>(amax);
            const float inv = inverse_scale(byte);
            p.scales[k][head * p.groups + g] = static_cast<uint8_t>(byte);
            for (int j = 0; j < n; j += 2) {
                float lo = load1<DT>(p.t[k].p, x0 + j) * inv;
                float hi = j + 1 < n ? load1<DT>(p.t[k].p, x0 + j + 1) * inv : 0.f;
                if (byte == 255u) lo = hi = 0.f;
                if (F == RMSNORM_CACHE_E4M3) {
                    const uint32_t c = to_e4m3x2(lo, hi);
                    uint8_t* out = p.codes[k] + head * p.code_bytes + j0 + j;
                    out[0] = static_cast<uint8_t>(c);
                    if (j + 1 < n) out[1] = static_cast<uint8_t>(c >> 8);
                } else {
                    p.codes[k][head * p.code_bytes + (j0 + j) / 2] =
                        static_cast<uint8_t>(to_e2m1x2(lo, hi));
                }
            }
        }
    }
}

template <int DT, int F>
__global__ void __launch_bounds__(256) cache_read_generic_kernel(const CacheP p) {
    pdl_wait();
    pdl_launch_dependents();
    const int64_t units = p.rows * p.heads * p.groups;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    for (int64_t u = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; u < units; u += step) {
        const int64_t i = u / (p.heads * p.groups);
        const int rest = static_cast<int>(u - i * (p.heads * p.groups));
        const int h = rest / p.groups, g = rest - h * p.groups;
        const int64_t slot = read_slot(p, i);
        if (slot == -1) continue;
        if (slot < 0 && rest == 0) atomicOr(&g_cache_status, 1u);
        const int64_t head = slot < 0 ? 0 : cache_head(p, slot, h);
        const int j0 = g * kGroup, n = p.D - j0 < kGroup ? p.D - j0 : kGroup;
        for (int k = 0; k < 2; ++k) {
            if (!p.t[k].p) continue;
            const int64_t y0 = i * p.t[k].st + h * p.t[k].sh + j0;
            const float scale = slot < 0 ? 0.f : scale_of(p.scales[k][head * p.groups + g]);
            for (int j = 0; j < n; ++j) {
                float v = 0.f;
                if (slot >= 0) {
                    if (F == RMSNORM_CACHE_E4M3) {
                        v = from_e4m3x2(p.codes[k][head * p.code_bytes + j0 + j]).x;
                    } else {
                        const uint32_t c = p.codes[k][head * p.code_bytes + (j0 + j) / 2];
                        v = from_e2m1x2(j & 1 ? c >> 4 : c & 15u).x;
                    }
                }
                store1<DT>(p.t[k].p, y0 + j, v * scale);
            }
        }
    }
}

// Vector kernels: groups of 32 values as 16-byte vectors. A thread takes 16
// values: half a group, whose other half is the neighbouring lane's, and one
// 16-byte (E4M3) or 8-byte (E2M1) piece of codes. Consecutive threads take
// consecutive halves of k's token, then of v's. Bound by HBM: each value read
// and each code written once, or the other way round.

// The largest magnitude of 16 values, as fp32 bits.
__device__ __forceinline__ uint32_t amax16(const float* f) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const uint32_t b = __float_as_uint(f[i]) & 0x7fffffffu;
        m = b > m ? b : m;
    }
    return m;
}

// `halves`: 16-value pieces of a token's heads of one tensor; units = T * tensors * halves.
template <int DT, int F>
__global__ void __launch_bounds__(256) cache_write_kernel(const CacheP p, int tensors, int halves, int head_halves) {
    constexpr int E = VecElems<DT>::value, NV = 16 / E;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t units = p.T * tensors * halves;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    // whole warps stay together: the two halves of a group are neighbouring lanes
    for (int64_t u0 = static_cast<int64_t>(blockIdx.x) * blockDim.x; u0 < units; u0 += step) {
        const int64_t u = u0 + threadIdx.x;
        const int64_t tk = u / halves;
        const int i = static_cast<int>(u - tk * halves);
        const int64_t t = tensors == 2 ? tk >> 1 : tk;
        const int k = tensors == 2 ? static_cast<int>(tk & 1) : 0;
        const int h = i / head_halves, part = i - h * head_halves;
        const int64_t slot = u < units ? __ldg(p.slot + t) : -1;
        const bool in = slot >= 0 && slot < p.slots;
        if (slot >= p.slots && i == 0 && k == 0) atomicOr(&g_cache_status, 1u);
        float f[16];
#pragma unroll
        for (int q = 0; q < 16; ++q) f[q] = 0.f;
        if (in) {
            const uint4* x = static_cast<const uint4*>(p.t[k].p) + t * p.t[k].st + h * p.t[k].sh + part * NV;
            uint4 v[NV];
#pragma unroll
            for (int q = 0; q < NV; ++q) v[q] = ld_stream(x + q);
#pragma unroll
            for (int q = 0; q < NV; ++q) unpack_vec<DT>(v[q], f + q * E);
        }
        uint32_t amax = amax16(f);
        const uint32_t other = __shfl_xor_sync(0xffffffffu, amax, 1);
        amax = other > amax ? other : amax;
        const uint32_t byte = scale_byte<F>(amax);
        const float inv = inverse_scale(byte);
        if (!in) continue;
        const int64_t head = cache_head(p, slot, h);
        if ((part & 1) == 0) p.scales[k][head * p.groups + (part >> 1)] = static_cast<uint8_t>(byte);
#pragma unroll
        for (int q = 0; q < 16; ++q) f[q] = byte == 255u ? 0.f : f[q] * inv;
        if (F == RMSNORM_CACHE_E4M3) {
            uint32_t c[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                c[q] = to_e4m3x2(f[4 * q], f[4 * q + 1]) | to_e4m3x2(f[4 * q + 2], f[4 * q + 3]) << 16;
            *reinterpret_cast<uint4*>(p.codes[k] + head * p.code_bytes + part * 16) =
                make_uint4(c[0], c[1], c[2], c[3]);
        } else {
            uint32_t c[2];
#pragma unroll
            for (int q = 0; q < 2; ++q)
                c[q] = to_e2m1x2(f[8 * q], f[8 * q + 1]) | to_e2m1x2(f[8 * q + 2], f[8 * q + 3]) << 8 |
                       to_e2m1x2(f[8 * q + 4], f[8 * q + 5]) << 16 | to_e2m1x2(f[8 * q + 6], f[8 * q + 7]) << 24;
            *reinterpret_cast<uint2*>(p.codes[k] + head * p.code_bytes + part * 8) = make_uint2(c[0], c[1]);
        }
    }
}

// A CTA takes rows of the outputs in tiles: a row's slot is looked up once, by one
// thread, and shared; then the threads take the tile's 16-value pieces.
constexpr int kReadRows = 64;  // most rows of a tile

template <int DT, int F>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheP p, int tensors, int first, int halves,
                                                         int head_halves, int tile_rows) {
    constexpr int E = VecElems<DT>::value, NV = 16 / E;
    __shared__ int64_t slots[kReadRows];
    pdl_wait();
    pdl_launch_dependents();
    const int64_t tiles = (p.rows + tile_rows - 1) / tile_rows;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t row0 = tile * tile_rows;
        const int n = static_cast<int>(min(static_cast<int64_t>(tile_rows), p.rows - row0));
        __syncthreads();  // the slots of the tile before are read
        if (threadIdx.x < n) {
            const int64_t slot = read_slot(p, row0 + threadIdx.x);
            if (slot == -2) atomicOr(&g_cache_status, 1u);
            slots[threadIdx.x] = slot;
        }
        __syncthreads();
        const int units = n * tensors * halves;
#pragma unroll 2
        for (int u = threadIdx.x; u < units; u += 256) {
            const int rk = u / halves, i = u - rk * halves;
            const int row = tensors == 2 ? rk >> 1 : rk;
            const int k = tensors == 2 ? rk & 1 : first;
            const int64_t slot = slots[row];
            if (slot == -1) continue;
            const int h = i / head_halves, part = i - h * head_halves;
            uint4* y = static_cast<uint4*>(p.t[k].p) + (row0 + row) * p.t[k].st + h * p.t[k].sh + part * NV;
            float f[16];
            if (slot < 0) {
#pragma unroll
                for (int q = 0; q < 16; ++q) f[q] = 0.f;
            } else {
                const int64_t head = cache_head(p, slot, h);
                const float scale = scale_of(__ldg(p.scales[k] + head * p.groups + (part >> 1)));
                if (F == RMSNORM_CACHE_E4M3) {
                    const uint4 c = ld_stream(
                        reinterpret_cast<const uint4*>(p.codes[k] + head * p.code_bytes + part * 16));
                    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 a = from_e4m3x2(w[q] & 0xffffu), b = from_e4m3x2(w[q] >> 16);
                        f[4 * q] = a.x * scale;
                        f[4 * q + 1] = a.y * scale;
                        f[4 * q + 2] = b.x * scale;
                        f[4 * q + 3] = b.y * scale;
                    }
                } else {
                    const uint2 c = __ldcs(reinterpret_cast<const uint2*>(p.codes[k] + head * p.code_bytes + part * 8));
                    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float2 a = from_e2m1x2((w[q >> 2] >> (8 * (q & 3))) & 0xffu);
                        f[2 * q] = a.x * scale;
                        f[2 * q + 1] = a.y * scale;
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < NV; ++q) st_stream(y + q, pack_vec<DT>(f + q * E));
        }
    }
}

// Whole groups, vectors and pieces everywhere.
bool vectors(bool write, const CacheP& p) {
    const int E = vec_elems(p.dtype);
    if (p.D % kGroup != 0) return false;
    const int64_t rows = write ? p.T : p.rows;
    const uintptr_t to = p.format == RMSNORM_CACHE_E4M3 ? 15 : 7;
    for (int k = 0; k < 2; ++k) {
        if (!p.t[k].p) continue;
        if (!aligned16(p.t[k].p) || (rows > 1 && p.t[k].st % E) || (p.heads > 1 && p.t[k].sh % E) ||
            (reinterpret_cast<uintptr_t>(p.codes[k]) & to))
            return false;
    }
    return static_cast<int64_t>(p.heads) * p.D / 16 * 2 * kReadRows < (int64_t(1) << 31);
}

template <int DT, int F>
cudaError_t run_vector(bool write, CacheP p, const OpCfg& c) {
    const int E = VecElems<DT>::value;
    const int head_halves = p.D / 16, halves = p.heads * head_halves;
    for (int k = 0; k < 2; ++k) {
        p.t[k].st /= E;
        p.t[k].sh /= E;
    }
    const int tensors = (p.t[0].p ? 1 : 0) + (p.t[1].p ? 1 : 0);
    if (write) {
        const int64_t G = persistent_grid(p.T * tensors * halves, 256, c.dev.sm_count, 8, c.max_ctas);
        return op_launch(c, cache_write_kernel<DT, F>, G, 256, 0, p, tensors, halves, head_halves);
    }
    // About eight pieces per thread and tile, fewer where rows are few.
    int64_t tile = std::max<int64_t>(1, 8 * 256 / (tensors * halves));
    tile = std::min<int64_t>(tile, std::max<int64_t>(1, p.rows / (2 * c.dev.sm_count)));
    tile = std::min<int64_t>(tile, kReadRows);
    const int64_t G = persistent_grid((p.rows + tile - 1) / tile, 1, c.dev.sm_count, 8, c.max_ctas);
    return op_launch(c, cache_read_kernel<DT, F>, G, 256, 0, p, tensors, p.t[0].p ? 0 : 1, halves, head_halves,
                     static_cast<int>(tile));
}

template <int DT, int F>
cudaError_t run(bool write, const CacheP& p, const OpCfg& c) {
    if (c.variant != RMSNORM_VARIANT_GENERIC && vectors(write, p)) return run_vector<DT, F>(write, p, c);
    if (c.variant == RMSNORM_VARIANT_CTA) return cudaErrorNotSupported;
    const int64_t units = (write ? p.T : p.rows) * p.heads * p.groups;
    const int64_t G = persistent_grid(units, 256, c.dev.sm_count, 8, c.max_ctas);
    return op_launch(c, write ? cache_write_generic_kernel<DT, F> : cache_read_generic_kernel<DT, F>,
                     G, 256, 0, p);
}

template <int F>
cudaError_t pick(bool write, const CacheP& p, const OpCfg& c) {
    switch (p.dtype) {
        case kBF16: return run<kBF16, F>(write, p, c);
        case kFP16: return run<kFP16, F>(write, p, c);
        default: return run<kFP32, F>(write, p, c);
    }
}

}  // namespace

cudaError_t cache_write_run(const CacheP& p, const OpCfg& c) {
    return p.format == RMSNORM_CACHE_E4M3 ? pick<RMSNORM_CACHE_E4M3>(true, p, c)
                                          : pick<RMSNORM_CACHE_E2M1>(true, p, c);
}

cudaError_t cache_read_run(const CacheP& p, const OpCfg& c) {
    return p.format == RMSNORM_CACHE_E4M3 ? pick<RMSNORM_CACHE_E4M3>(false, p, c)
                                          : pick<RMSNORM_CACHE_E2M1>(false, p, c);
}

cudaError_t cache_status_read_and_clear(unsigned int* value) {
    return symbol_read_and_clear(g_cache_status, value);
}

}  // namespace rmsn
