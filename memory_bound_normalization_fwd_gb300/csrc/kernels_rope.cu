// Rotary positions on the heads of q and k after each head's RMSNorm, and the
// backward of the two (the operation is stated in include/rmsnorm.h).
//
// Angles. A frequency is held as the fraction of a turn per position times
// 2^64, so position * step modulo 2^64 is the phase, exact for any position:
// its top 32 bits as a signed number are the angle in half turns times 2^31,
// and sincospif of that needs no range reduction. The phase is off by 2^-32
// turns and its fp32 value by 2^-25 half turns.
#include "rmsnorm.h"

#include "ops.h"
#include "ops_common.cuh"

#include <algorithm>

namespace rmsn {
namespace {

// cos and sin (times magnitude) of pair i at a position.
__device__ __forceinline__ float2 turn(int64_t position, uint64_t step, float magnitude) {
    const uint64_t phase = static_cast<uint64_t>(position) * step;
    const float x = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(x, &s, &c);
    return make_float2(c * magnitude, s * magnitude);
}

__device__ __forceinline__ int64_t position_of(const RopeP& p, int64_t b, int64_t s) {
    return p.positions ? p.positions[b * p.positions_stride + s] : s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Element-wise kernels: any head size, alignment and stride; one warp per head
// of a token (head index over q's and then k's heads). A lane owns the pairs
// lane, lane + 32, ... and the values behind rotary_dim in the same way, reads
// both values of a pair before it writes them, and no lane reads another's, so
// the outputs may lie on the inputs.
struct Unit {
    int seg;
    int64_t b, s, h, token;
};

__device__ __forceinline__ Unit unit_of(const RopeP& p, int64_t u) {
    const int H = p.seg[0].heads + p.seg[1].heads;
    Unit o;
    o.token = u / H;
    o.h = u - o.token * H;
    o.seg = o.h >= p.seg[0].heads;
    if (o.seg) o.h -= p.seg[0].heads;
    o.b = o.token / p.seq;
    o.s = o.token - o.b * p.seq;
    return o;
}

__device__ __forceinline__ int64_t at(const HeadsP& h, const Unit& u) {
    return u.b * h.sb + u.s * h.st + u.h * h.sh;
}

template <int DT>
__global__ void __launch_bounds__(256) rope_fwd_generic_kernel(const RopeP p) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
    const int64_t units = p.batch * p.seq * (p.seg[0].heads + p.seg[1].heads);
    const int half = p.R / 2;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < units; i += warps) {
        const Unit u = unit_of(p, i);
        const RopeSeg& g = p.seg[u.seg];
        const int64_t x0 = at(g.in, u), y0 = at(g.out, u);
        float r = 1.f;
        if (g.w) {
            float ss = 0.f;
            for (int j = lane; j < p.D; j += 32) {
                const float f = load1<DT>(g.in.p, x0 + j);
                ss = fmaf(f, f, ss);
            }
            r = row_rstd(warp_sum(ss), static_cast<float>(p.D), p.eps);
            if (lane == 0 && g.rstd) g.rstd[u.token * g.heads + u.h] = r;
        }
        auto x = [&](int j) {
            const float f = load1<DT>(g.in.p, x0 + j);
            return g.w ? f * r * (p.offset + load1<DT>(g.w, j)) : f;
        };
        const int64_t pos = position_of(p, u.b, u.s);
        __syncwarp();  // every lane's reads for the sum before the first write
        for (int j = lane; j < half; j += 32) {
            const float2 cs = turn(pos, p.steps[j], p.magnitude);
            const int a = p.interleaved ? 2 * j : j, b = p.interleaved ? 2 * j + 1 : j + half;
            const float xa = x(a), xb = x(b);
            store1<DT>(g.out.p, y0 + a, fmaf(xa, cs.x, -xb * cs.y));
            store1<DT>(g.out.p, y0 + b, fmaf(xb, cs.x, xa * cs.y));
        }
        for (int j = p.R + lane; j < p.D; j += 32) store1<DT>(g.out.p, y0 + j, x(j));
    }
}

// Backward: the gradient turned back, then the norm's backward. A warp keeps
// the weights' gradient sums of the heads it sees in its own two partial rows.
template <int DT>
__global__ void __launch_bounds__(256) rope_bwd_generic_kernel(const RopeP p) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
    const int64_t me = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t units = p.batch * p.seq * (p.seg[0].heads + p.seg[1].heads);
    const int half = p.R / 2;
    pdl_wait();
    for (int k = 0; k < 2; ++k) {
        if (!p.seg[k].w) continue;
        float* acc = p.ws + (k * warps + me) * p.D;
        for (int j = lane; j < half; j += 32) acc[j] = acc[half + j] = 0.f;
        for (int j = p.R + lane; j < p.D; j += 32) acc[j] = 0.f;
    }
    for (int64_t i = me; i < units; i += warps) {
        const Unit u = unit_of(p, i);
        const RopeSeg& g = p.seg[u.seg];
        const int64_t d0 = at(g.in, u), o0 = at(g.out, u), x0 = at(g.x, u);
        const int64_t pos = position_of(p, u.b, u.s);
        // The gradient of the normed head at pair j (as its two values) and
        // behind rotary_dim.
        auto back = [&](int j) {
            const float2 cs = turn(pos, p.steps[j], p.magnitude);
            const int a = p.interleaved ? 2 * j : j, b = p.interleaved ? 2 * j + 1 : j + half;
            const float da = load1<DT>(g.in.p, d0 + a), db = load1<DT>(g.in.p, d0 + b);
            return make_float2(fmaf(da, cs.x, db * cs.y), fmaf(db, cs.x, -da * cs.y));
        };
        float r = 1.f, f = 0.f;
        if (g.w) {
            r = g.rstd[u.token * g.heads + u.h];
            float c = 0.f;
            for (int j = lane; j < half; j += 32) {
                const int a = p.interleaved ? 2 * j : j, b = p.interleaved ? 2 * j + 1 : j + half;
                const float2 d = back(j);
                c = fmaf(d.x * (p.offset + load1<DT>(g.w, a)), load1<DT>(g.x.p, x0 + a), c);
                c = fmaf(d.y * (p.offset + load1<DT>(g.w, b)), load1<DT>(g.x.p, x0 + b), c);
            }
            for (int j = p.R + lane; j < p.D; j += 32)
                c = fmaf(load1<DT>(g.in.p, d0 + j) * (p.offset + load1<DT>(g.w, j)),
                         load1<DT>(g.x.p, x0 + j), c);
            f = r * r * (warp_sum(c) / static_cast<float>(p.D));
        }
        float* acc = p.ws + (u.seg * warps + me) * p.D;
        auto put = [&](int j, int slot, float d) {
            if (g.w) {
                const float x = load1<DT>(g.x.p, x0 + j);
                acc[slot] = fmaf(d, x * r, acc[slot]);
                d = r * fmaf(d, p.offset + load1<DT>(g.w, j), -x * f);
            }
            store1<DT>(g.out.p, o0 + j, d);
        };
        for (int j = lane; j < half; j += 32) {
            const float2 d = back(j);
            // sums are kept at j and half + j (this lane's), whatever the layout
            put(p.interleaved ? 2 * j : j, j, d.x);
            put(p.interleaved ? 2 * j + 1 : j + half, half + j, d.y);
        }
        for (int j = p.R + lane; j < p.D; j += 32) put(j, j, load1<DT>(g.in.p, d0 + j));
    }
    pdl_launch_dependents();
}

// dw_q and dw_k: sums of the partial rows in order. blockIdx.y is the tensor.
// Partial rows hold the first value of pair i at i, the second at half + i.
__global__ void __launch_bounds__(256) rope_dw_kernel(const RopeP p, int64_t rows) {
    __shared__ float part[8][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, half = p.R / 2;
    const int slot = static_cast<int>(blockIdx.x) * 32 + lane;
    pdl_wait();
    if (!p.seg[blockIdx.y].w) return;
    float t = 0.f;
    if (slot < p.D) {
        const float* q = p.ws + static_cast<int64_t>(blockIdx.y) * rows * p.D + slot;
        for (int64_t i = w; i < rows; i += 8) t += q[i * p.D];
    }
    part[w][lane] = t;
    __syncthreads();
    if (w == 0 && slot < p.D) {
        t = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += part[k][lane];
        const int j = !p.interleaved || slot >= p.R ? slot
                      : slot < half ? 2 * slot : 2 * (slot - half) + 1;
        p.seg[blockIdx.y].dw[j] = t;
    }
}

constexpr int kGenericCtasPerSM = 8;

int64_t generic_grid(const RopeP& p, const OpCfg& c) {
    const int64_t units = p.batch * p.seq * (p.seg[0].heads + p.seg[1].heads);
    return persistent_grid(units, 8, c.dev.sm_count, kGenericCtasPerSM, c.max_ctas);
}

template <int DT>
cudaError_t fwd(const RopeP& p, const OpCfg& c) {
    return op_launch(c, rope_fwd_generic_kernel<DT>, generic_grid(p, c), 256, 0, p);
}

template <int DT>
cudaError_t bwd(const RopeP& p, const OpCfg& c) {
    const int64_t G = generic_grid(p, c);
    cudaError_t e = op_launch(c, rope_bwd_generic_kernel<DT>, G, 256, 0, p);
    if (e != cudaSuccess || (!p.seg[0].w && !p.seg[1].w)) return e;
    Launch l;
    l.grid = (p.D + 31) / 32;
    l.threads = 256;
    LaunchCfg cfg(l, c.stream, c.pdl);
    cfg.cfg.gridDim.y = 2;
    return cudaLaunchKernelEx(&cfg.cfg, rope_dw_kernel, p, G * 8);
}

}  // namespace

int64_t rope_bwd_partial_rows(int sm_count) {
    return 2LL * sm_count * kGenericCtasPerSM * 8;
}

cudaError_t rope_fwd_run(const RopeP& p, const OpCfg& c) {
    switch (p.dtype) {
        case kBF16: return fwd<kBF16>(p, c);
        case kFP16: return fwd<kFP16>(p, c);
        default: return fwd<kFP32>(p, c);
    }
}

cudaError_t rope_bwd_run(const RopeP& p, const OpCfg& c) {
    switch (p.dtype) {
        case kBF16: return bwd<kBF16>(p, c);
        case kFP16: return bwd<kFP16>(p, c);
        default: return bwd<kFP32>(p, c);
    }
}

}  // namespace rmsn
