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
static std::atomic<bool> g_launched{false};  // a kernel that writes it

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

// The sequence whose rows hold row i: the last b with cu[b] <= i. cu is cu_rows
// or a copy of it.
__device__ __forceinline__ int64_t sequence_of(const CacheP& p, const int32_t* cu, int64_t i) {
    int64_t lo = 0, hi = p.sequences - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= i) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The slot of row i: -1 for a row behind the last sequence, -2 for one whose
// page is not there.
__device__ __forceinline__ int64_t read_slot(const CacheP& p, const int32_t* cu, int64_t i) {
    if (p.sequences <= 0 || i >= cu[p.sequences]) return -1;
    const int64_t b = sequence_of(p, cu, i);
    const int64_t pos = i - cu[b] + (p.starts ? p.starts[b] : 0);
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
        const int64_t per = static_cast<int64_t>(p.heads) * p.groups;
        const int64_t t = u / per, rest = u - t * per;
        const int h = static_cast<int>(rest / p.groups), g = static_cast<int>(rest - static_cast<int64_t>(h) * p.groups);
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
        const int64_t per = static_cast<int64_t>(p.heads) * p.groups;
        const int64_t i = u / per, rest = u - i * per;
        const int h = static_cast<int>(rest / p.groups), g = static_cast<int>(rest - static_cast<int64_t>(h) * p.groups);
        const int64_t slot = read_slot(p, p.cu_rows, i);
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

// Vector kernels. A piece is 16 values: half a group, whose other half is the
// neighbouring lane's, and one 16-byte (E4M3) or 8-byte (E2M1) run of codes. A CTA
// takes tokens in tiles; a token's slot is looked up once, by one thread, a tile
// ahead, and shared; then consecutive threads take consecutive pieces of k's and
// v's heads. Where a token's pieces divide the CTA's
// threads, a thread's head and place in it never change. Bound by HBM: each value
// read and each code written once, or the other way round; so the arithmetic is on
// pairs (f32x2), 16-bit magnitudes are compared two at a time, and there is no
// division in the loops (with those it was bound by instructions: a write of 32768
// tokens 45 us, a read of 134k rows 200 us; now 34 and 146). Pieces in flight per
// thread, GB300, us: write of 32768 tokens at 1 / 2 / 4: 34.3 / 33.8 / 35.7; read of
// 134k rows 146 / 159 / 161.
constexpr int kTileTokens = 64;   // most tokens of a tile
constexpr int kWriteBatch = 2;    // pieces of a thread in flight
constexpr int kSharedRows = 2048; // sequences whose first rows fit into shared memory

// How a tile's pieces go round the CTA's threads.
struct Pieces {
    int tensors, first;       // 1 or 2, and which one where it is one
    int halves, head_halves;  // pieces of a token's heads of one tensor, of a head
    int tile;                 // tokens per tile
    int64_t tiles;
};

// A thread's way through a tile: token, tensor, head and part, going up by the CTA's
// 256 threads.
struct PieceWay {
    int per, dt, dp;   // pieces of a token; 256 over that, and the remainder
    int t0, p0;
    int t, p;          // token of the tile, piece of the token
    int k, h, part;
    __device__ __forceinline__ void set(const Pieces& g) {
        const int q = p / g.halves, i = p - q * g.halves;
        k = g.tensors == 2 ? q : g.first;
        h = i / g.head_halves;
        part = i - h * g.head_halves;
    }
    __device__ __forceinline__ explicit PieceWay(const Pieces& g) {
        per = g.tensors * g.halves;
        dt = 256 / per;
        dp = 256 - dt * per;
        t0 = threadIdx.x / per;
        p0 = threadIdx.x - t0 * per;
        t = t0;
        p = p0;
        set(g);
    }
    __device__ __forceinline__ void restart(const Pieces& g) {
        t = t0;
        if (dp != 0) {
            p = p0;
            set(g);
        }
    }
    __device__ __forceinline__ void go(const Pieces& g) {
        t += dt;
        if (dp != 0) {
            p += dp;
            if (p >= per) {
                p -= per;
                ++t;
            }
            set(g);
        }
    }
};

// Index of a slot's head 0 among the cache's heads; head h is h * stride further.
__device__ __forceinline__ int64_t first_head(const CacheP& p, int64_t slot) {
    if (!p.heads_first) return slot * p.heads;
    const int64_t page = slot / p.page_size;
    return page * p.heads * p.page_size + (slot - page * p.page_size);
}

// The largest magnitude of a lane's 16 values as fp32 bits. 16-bit values are
// compared by their bits, two at a time.
template <int DT>
__device__ __forceinline__ uint32_t amax16(const uint4* v) {
    if constexpr (DT == kFP32) {
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            m = max(m, max(v[q].x & 0x7fffffffu, v[q].y & 0x7fffffffu));
            m = max(m, max(v[q].z & 0x7fffffffu, v[q].w & 0x7fffffffu));
        }
        return m;
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            m = __vmaxu2(m, __vmaxu2(v[q].x & 0x7fff7fffu, v[q].y & 0x7fff7fffu));
            m = __vmaxu2(m, __vmaxu2(v[q].z & 0x7fff7fffu, v[q].w & 0x7fff7fffu));
        }
        const uint32_t top = max(m & 0xffffu, m >> 16);
        return __float_as_uint(Codec<DT>::unpack1(static_cast<uint16_t>(top)));
    }
}

template <int DT, int F>
__global__ void __launch_bounds__(256) cache_write_kernel(const CacheP p, const Pieces g) {
    constexpr int E = VecElems<DT>::value, NV = 16 / E;
    __shared__ int64_t heads_of[2][kTileTokens];  // -1: no slot
    const int64_t head_stride = p.heads_first ? p.page_size : 1;
    PieceWay way(g);
    pdl_wait();
    pdl_launch_dependents();
    auto lookup = [&](int64_t tile) -> int64_t {
        const int64_t t = tile * g.tile + threadIdx.x;
        if (threadIdx.x >= g.tile || t >= p.T) return -1;
        const int64_t slot = __ldg(p.slot + t);
        if (slot < 0) return -1;
        if (slot >= p.slots) {
            atomicOr(&g_cache_status, 1u);
            return -1;
        }
        return first_head(p, slot);
    };
    int64_t found = lookup(blockIdx.x);
    int buffer = 0;
    for (int64_t tile = blockIdx.x; tile < g.tiles; tile += gridDim.x, buffer ^= 1) {
        if (threadIdx.x < g.tile) heads_of[buffer][threadIdx.x] = found;
        __syncthreads();  // the other buffer is free behind the next tile's barrier
        found = lookup(tile + gridDim.x);
        const int64_t t0 = tile * g.tile;
        const int n = static_cast<int>(min(static_cast<int64_t>(g.tile), p.T - t0));
        const int units = n * way.per;
        way.restart(g);
        for (int u = 0; u < units; u += 256 * kWriteBatch) {
            uint4 v[kWriteBatch][NV];
            int64_t head[kWriteBatch];
            int k[kWriteBatch], part[kWriteBatch];
#pragma unroll
            for (int b = 0; b < kWriteBatch; ++b) {
                head[b] = way.t < n ? heads_of[buffer][way.t] : -1;
                k[b] = way.k;
                part[b] = way.part;
                if (head[b] >= 0) {
                    head[b] += way.h * head_stride;
                    const uint4* x = static_cast<const uint4*>(p.t[way.k].p) + (t0 + way.t) * p.t[way.k].st +
                                     way.h * p.t[way.k].sh + way.part * NV;
#pragma unroll
                    for (int q = 0; q < NV; ++q) v[b][q] = ld_stream(x + q);
                } else {
#pragma unroll
                    for (int q = 0; q < NV; ++q) v[b][q] = make_uint4(0u, 0u, 0u, 0u);
                }
                way.go(g);
            }
#pragma unroll
            for (int b = 0; b < kWriteBatch; ++b) {
                uint32_t amax = amax16<DT>(v[b]);
                amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                if (head[b] < 0) continue;
                const uint32_t byte = scale_byte<F>(amax);
                const f2 inv = f2_dup(inverse_scale(byte));
                f2 f[8];
#pragma unroll
                for (int q = 0; q < NV; ++q) unpack2<DT>(v[b][q], f + q * (E / 2));
                uint32_t c[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float2 y = f2_get(f2_mul(f[q], inv));
                    c[q] = F == RMSNORM_CACHE_E4M3 ? to_e4m3x2(y.x, y.y) : to_e2m1x2(y.x, y.y);
                }
                uint8_t* codes = p.codes[k[b]] + head[b] * p.code_bytes;
                const bool bad = byte == 255u;
                if (F == RMSNORM_CACHE_E4M3) {
                    const uint32_t w0 = c[0] | c[1] << 16, w1 = c[2] | c[3] << 16;
                    const uint32_t w2 = c[4] | c[5] << 16, w3 = c[6] | c[7] << 16;
                    *reinterpret_cast<uint4*>(codes + part[b] * 16) =
                        make_uint4(bad ? 0u : w0, bad ? 0u : w1, bad ? 0u : w2, bad ? 0u : w3);
                } else {
                    const uint32_t w0 = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
                    const uint32_t w1 = c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24;
                    *reinterpret_cast<uint2*>(codes + part[b] * 8) = make_uint2(bad ? 0u : w0, bad ? 0u : w1);
                }
                if ((part[b] & 1) == 0)
                    p.scales[k[b]][head[b] * p.groups + (part[b] >> 1)] = static_cast<uint8_t>(byte);
            }
        }
    }
}

template <int DT, int F>
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheP p, const Pieces g) {
    constexpr int E = VecElems<DT>::value, NV = 16 / E;
    __shared__ int64_t heads_of[2][kTileTokens];  // -1: not a row, -2: zeros
    __shared__ int32_t first_rows[kSharedRows + 1];
    const int64_t head_stride = p.heads_first ? p.page_size : 1;
    PieceWay way(g);
    pdl_wait();
    pdl_launch_dependents();
    const bool shared_rows = p.sequences <= kSharedRows;
    if (shared_rows) {
        for (int i = threadIdx.x; i <= p.sequences; i += 256) first_rows[i] = p.cu_rows[i];
        __syncthreads();
    }
    const int32_t* cu = shared_rows ? first_rows : p.cu_rows;
    auto lookup = [&](int64_t tile) -> int64_t {
        const int64_t i = tile * g.tile + threadIdx.x;
        if (threadIdx.x >= g.tile || i >= p.rows) return -1;
        const int64_t slot = read_slot(p, cu, i);
        if (slot == -2) atomicOr(&g_cache_status, 1u);
        return slot < 0 ? slot : first_head(p, slot);
    };
    int64_t found = lookup(blockIdx.x);
    int buffer = 0;
    for (int64_t tile = blockIdx.x; tile < g.tiles; tile += gridDim.x, buffer ^= 1) {
        if (threadIdx.x < g.tile) heads_of[buffer][threadIdx.x] = found;
        __syncthreads();  // the other buffer is free behind the next tile's barrier
        found = tile + gridDim.x < g.tiles ? lookup(tile + gridDim.x) : -1;
        const int64_t row0 = tile * g.tile;
        const int n = static_cast<int>(min(static_cast<int64_t>(g.tile), p.rows - row0));
        const int units = n * way.per;
        way.restart(g);
        for (int u = 0; u < units; u += 256, way.go(g)) {
            const int64_t base = way.t < n ? heads_of[buffer][way.t] : -1;
            if (base == -1) continue;
            uint4 c = make_uint4(0u, 0u, 0u, 0u);
            uint32_t byte = 0;
            if (base >= 0) {
                const int64_t head = base + way.h * head_stride;
                const uint8_t* codes = p.codes[way.k] + head * p.code_bytes;
                if (F == RMSNORM_CACHE_E4M3) {
                    c = ld_stream(reinterpret_cast<const uint4*>(codes + way.part * 16));
                } else {
                    const uint2 w = __ldcs(reinterpret_cast<const uint2*>(codes + way.part * 8));
                    c.x = w.x;
                    c.y = w.y;
                }
                byte = __ldg(p.scales[way.k] + head * p.groups + (way.part >> 1));
            }
            const f2 scale = f2_dup(scale_of(byte));
            const uint32_t w[4] = {c.x, c.y, c.z, c.w};
            f2 f[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const float2 a = F == RMSNORM_CACHE_E4M3 ? from_e4m3x2((w[q >> 1] >> (16 * (q & 1))) & 0xffffu)
                                                         : from_e2m1x2((w[q >> 2] >> (8 * (q & 3))) & 0xffu);
                f[q] = f2_mul(f2_make(a.x, a.y), scale);
            }
            uint4* y = static_cast<uint4*>(p.t[way.k].p) + (row0 + way.t) * p.t[way.k].st + way.h * p.t[way.k].sh +
                       way.part * NV;
#pragma unroll
            for (int q = 0; q < NV; ++q) st_stream(y + q, pack2<DT>(f + q * (E / 2)));
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
    return static_cast<int64_t>(p.heads) * p.D / 16 * 2 * kTileTokens < (int64_t(1) << 30);
}

template <int DT, int F>
cudaError_t run_vector(bool write, CacheP p, const OpCfg& c) {
    const int E = VecElems<DT>::value;
    for (int k = 0; k < 2; ++k) {
        p.t[k].st /= E;
        p.t[k].sh /= E;
    }
    Pieces g;
    g.tensors = (p.t[0].p ? 1 : 0) + (p.t[1].p ? 1 : 0);
    g.first = p.t[0].p ? 0 : 1;
    g.head_halves = p.D / 16;
    g.halves = p.heads * g.head_halves;
    auto fn = write ? cache_write_kernel<DT, F> : cache_read_kernel<DT, F>;
    const int occ = std::max(1, occupancy(reinterpret_cast<const void*>(fn), 256, 0));
    const int64_t rows = write ? p.T : p.rows;
    const int per = g.tensors * g.halves;
    // Four pieces per thread and tile, two of 16 code bytes in a read (GB300, us,
    // 134k rows at 2 / 4 / 8 pieces: E4M3 145 / 160 / 164, E2M1 145 / 130 / 126);
    // fewer where tokens are few.
    const int pieces = !write && F == RMSNORM_CACHE_E4M3 ? 2 : 4;
    int64_t tile = std::max<int64_t>(1, pieces * 256 / per);
    tile = std::min<int64_t>(tile, std::max<int64_t>(1, rows / c.dev.sm_count));
    g.tile = static_cast<int>(std::min<int64_t>(tile, kTileTokens));
    g.tiles = (rows + g.tile - 1) / g.tile;
    const int64_t G = persistent_grid(g.tiles, 1, c.dev.sm_count, occ, c.max_ctas);
    return op_launch(c, fn, G, 256, 0, p, g);
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
    g_launched.store(true);
    return p.format == RMSNORM_CACHE_E4M3 ? pick<RMSNORM_CACHE_E4M3>(true, p, c)
                                          : pick<RMSNORM_CACHE_E2M1>(true, p, c);
}

cudaError_t cache_read_run(const CacheP& p, const OpCfg& c) {
    g_launched.store(true);
    return p.format == RMSNORM_CACHE_E4M3 ? pick<RMSNORM_CACHE_E4M3>(false, p, c)
                                          : pick<RMSNORM_CACHE_E2M1>(false, p, c);
}

cudaError_t cache_status_read_and_clear(unsigned int* value) {
    return symbol_read_and_clear(g_cache_status, g_launched, value);
}

}  // namespace rmsn
