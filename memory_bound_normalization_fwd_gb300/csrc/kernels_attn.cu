// Attention over the quantised cache: the element-wise kernel for any head size, and the
// choice of a kernel (the operation is stated in include/rmsnorm.h).
#include "rmsnorm.h"

#include "attn_common.cuh"
#include "row_ring_host.h"

#include <algorithm>

namespace rmsn {

// Bit 0: a token's page was not there since the last read. One word per device.
__device__ unsigned int g_attn_status;
static std::atomic<bool> g_launched{false};  // a kernel that writes it

namespace {

// Element-wise: a CTA of four warps a row of a head. Lane l holds the values l, l + 32, ...
// (one of each group); the warps take every fourth token, with a running maximum and
// sum each, and are joined at the end. 16 * 32 values: head_dim up to 512.
template <int DT, int F>
__global__ void __launch_bounds__(128) attn_generic_kernel(const AttnP p) {
    constexpr int V = 16;
    __shared__ float part[4][V * 32 + 2];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    const int64_t units = p.rows * p.heads_q;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t row = u / p.heads_q;
        const int h = static_cast<int>(u - row * p.heads_q), hk = h / p.G;
        // the last sequence that begins at or before the row
        int64_t b = row;
        if (p.cu) {
            int64_t lo = 0, hi = p.sequences - 1;
            while (lo < hi) {
                const int64_t mid = (lo + hi + 1) >> 1;
                if (p.cu[mid] <= row) lo = mid;
                else hi = mid - 1;
            }
            b = lo;
        }
        const Sequence s = sequence(p, b);
        if (row < s.row0 || row >= s.row0 + s.n) continue;  // behind the last sequence
        const Seen see = seen(p, s, row - s.row0);
        float q[V], o[V], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int d = j * 32 + lane;
            q[j] = d < p.D ? load1<DT>(p.q.p, row * p.q.st + h * p.q.sh + d) : 0.f;
            o[j] = 0.f;
        }
        auto value = [&](int which, int64_t head, int j) {
            const int d = j * 32 + lane;
            if (d >= p.D) return 0.f;
            const uint8_t* c = p.codes[which] + head * p.code_bytes;
            const float f = scale_of(__ldg(p.scales[which] + head * p.groups + j));
            uint32_t pair;
            if (F == RMSNORM_CACHE_E4M3) {
                pair = __half_as_ushort(static_cast<__half>(
                    __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(c[d]), __NV_E4M3)));
            } else {
                const uint32_t byte = c[d >> 1];
                pair = __half_as_ushort(static_cast<__half>(__nv_cvt_fp4_to_halfraw(
                    static_cast<__nv_fp4_storage_t>(d & 1 ? byte >> 4 : byte & 15u), __NV_E2M1)));
            }
            return __half2float(__ushort_as_half(static_cast<unsigned short>(pair))) * f;
        };
        for (int64_t t = see.low + w; t < see.high && t < s.len; t += 4) {
            int64_t head = token_at(p, b, t);
            if (head < 0) {
                if (lane == 0) atomicOr(p.status, 1u);
                continue;
            }
            head += hk * head_step(p);
            float x = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < p.groups) x = fmaf(q[j], value(0, head, j), x);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
            x *= p.scale;
            if (x > m) {
                const float c = expf(m - x);
                m = x;
                l *= c;
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] *= c;
            }
            // a score that is NaN, or infinite like the maximum, stays one
            const float e = x == -INFINITY ? 0.f : expf(x - m);
            l += e;
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (j < p.groups) o[j] = fmaf(e, value(1, head, j), o[j]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) part[w][j * 32 + lane] = o[j];
        if (lane == 0) {
            part[w][V * 32] = m;
            part[w][V * 32 + 1] = l;
        }
        __syncthreads();
        // A warp without tokens counts nothing; one whose sum is a NaN makes all of them NaN.
        float top = -INFINITY, sum = 0.f, f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) top = fmaxf(top, part[k][V * 32]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float lk = part[k][V * 32 + 1];
            f[k] = lk == 0.f ? 0.f : lk != lk ? lk : expf(part[k][V * 32] - top);
            sum += f[k] * lk;
        }
        for (int d = threadIdx.x; d < p.D; d += 128) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) v += f[k] * part[k][d];
            store1<DT>(p.out.p, row * p.out.st + h * p.out.sh + d, sum == 0.f ? 0.f : v / sum);
        }
        if (p.lse && threadIdx.x == 0) p.lse[row * p.heads_q + h] = sum == 0.f ? -INFINITY : top + logf(sum);
        __syncthreads();  // part is free again
    }
}

template <int F>
cudaError_t run_generic(const AttnP& p, const OpCfg& c) {
    const int64_t G = persistent_grid(p.rows * p.heads_q, 1, c.dev.sm_count, 12, c.max_ctas);
    switch (p.dtype) {
        case kBF16: return op_launch(c, attn_generic_kernel<kBF16, F>, G, 128, 0, p);
        case kFP16: return op_launch(c, attn_generic_kernel<kFP16, F>, G, 128, 0, p);
        default: return op_launch(c, attn_generic_kernel<kFP32, F>, G, 128, 0, p);
    }
}

// The status word's address on the current device, for kernels of other files.
cudaError_t status_word(unsigned int** word) {
    constexpr int kDevices = 64;
    static std::atomic<unsigned int*> known[kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kDevices && (*word = known[dev].load()) != nullptr) return cudaSuccess;
    void* at = nullptr;
    e = cudaGetSymbolAddress(&at, g_attn_status);
    if (e != cudaSuccess) return e;
    *word = static_cast<unsigned int*>(at);
    if (dev < kDevices) known[dev].store(*word);
    return cudaSuccess;
}

}  // namespace

int64_t attn_ws_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int) { return 0; }

cudaError_t attn_run(const AttnP& given, const OpCfg& c) {
    AttnP p = given;
    const cudaError_t e = status_word(&p.status);
    if (e != cudaSuccess) return e;
    g_launched.store(true);
    if (c.variant == RMSNORM_VARIANT_CTA) return cudaErrorNotSupported;
    return p.format == RMSNORM_CACHE_E4M3 ? run_generic<RMSNORM_CACHE_E4M3>(p, c)
                                          : run_generic<RMSNORM_CACHE_E2M1>(p, c);
}

cudaError_t attn_status_read_and_clear(unsigned int* value) {
    return symbol_read_and_clear(g_attn_status, g_launched, value);
}

}  // namespace rmsn
