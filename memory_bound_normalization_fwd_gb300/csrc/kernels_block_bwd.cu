// Backward of the block operator (the formulas are in include/rmsnorm.h).
//
// One reduction per row: with u = dy (offset + w_pre), k2 = rstd_pre,
// a = alpha gate (offset + w_post),
//
//   c2 = sum u s,   A = sum a h (ds + k2 u),   B = sum a h s
//   t  = ds + k2 u - e s            e = k2^3 c2 / N
//   sum a h t = A - e B             (what the norm after the block subtracts)
//
// so both norms' row sums come from one pass. Sums over rows: P = sum of
// t h rstd_post over the rows of one gate row gives that row's dgate
// (alpha (offset + w_post) P) and its part of dw_post (alpha gate P), so one
// column sum serves both.
//
// Rows are split over the CTAs in contiguous ranges. A gate row whose rows all
// lie in one CTA's range is finished there; the others leave a partial row
// per CTA (a CTA's range starts and ends in at most two such gate rows).
// A second launch sums the partial rows in CTA order.
#include "rmsnorm.h"

#include "ops.h"
#include "ops_common.cuh"

#include <algorithm>

namespace rmsn {
namespace {

__host__ __device__ inline int64_t range_begin(int64_t b, int64_t grid, int64_t M) {
    return b * (M / grid) + (b < M % grid ? b : M % grid);
}
// The CTA whose range holds a row.
__host__ __device__ inline int64_t range_owner(int64_t row, int64_t grid, int64_t M) {
    const int64_t q = M / grid, big = M % grid;
    return row < big * (q + 1) ? row / (q + 1) : big + (row - big * (q + 1)) / q;
}

// Workspace: four areas of `grid` partial rows of `pitch` floats: dw_post,
// dw_pre, gate sums that begin with the CTA's range, gate sums that begin
// inside it.
__device__ inline float* partial(float* ws, int area, int64_t cta, int64_t grid, int64_t pitch) {
    return ws + (area * grid + cta) * pitch;
}

// Element-wise kernel: any N, alignment and stride; a thread owns the columns
// tid, tid + T, ... and keeps their sums in the CTA's partial rows.
template <int DT>
__global__ void __launch_bounds__(512) block_bwd_generic_kernel(const BlockBwdP p) {
    __shared__ float part[2 * 3 * 32];
    int parity = 0;
    const int tid = threadIdx.x, T = blockDim.x;
    const int64_t G = gridDim.x, b = blockIdx.x, pitch = block_bwd_pitch(p.N);
    const int64_t r0 = range_begin(b, G, p.M), r1 = range_begin(b + 1, G, p.M);
    float* acc_post = partial(p.ws, 0, b, G, pitch);
    float* acc_pre = partial(p.ws, 1, b, G, pitch);
    const bool per_element = p.gate && p.gate_rows == 1;
    const bool grouped = p.gate && !per_element;
    pdl_wait();
    for (int64_t j = tid; j < p.N; j += T) {
        if (p.w_post) acc_post[j] = 0.f;
        if (p.w_pre) acc_pre[j] = 0.f;
    }
    float* acc_gate = nullptr;
    for (int64_t row = r0; row < r1; ++row) {
        const int64_t h0 = row * p.ldh, s0 = row * p.lds, dy0 = row * p.lddy, ds0 = row * p.ldds;
        const int64_t grow = p.gate ? row / p.gate_rows : 0;
        const int64_t g0 = grow * p.ldg;
        if (grouped && (row == r0 || row % p.gate_rows == 0)) {
            acc_gate = partial(p.ws, row == r0 ? 2 : 3, b, G, pitch);
            for (int64_t j = tid; j < p.N; j += T) acc_gate[j] = 0.f;
        }
        const float k1 = p.w_post ? p.rstd_post[row] : 1.f;
        const float k2 = p.w_pre ? p.rstd_pre[row] : 0.f;
        auto scale = [&](int64_t j) {  // a
            float a = p.alpha;
            if (p.gate) a *= load1<DT>(p.gate, g0 + j);
            if (p.w_post) a *= p.offset + load1<DT>(p.w_post, j);
            return a;
        };
        float v[3] = {0.f, 0.f, 0.f};
        for (int64_t j = tid; j < p.N; j += T) {
            const float s = p.w_pre ? load1<DT>(p.s, s0 + j) : 0.f;
            const float u = p.w_pre ? load1<DT>(p.dy, dy0 + j) * (p.offset + load1<DT>(p.w_pre, j)) : 0.f;
            const float d = p.ds ? load1<DT>(p.ds, ds0 + j) : 0.f;
            v[0] = fmaf(u, s, v[0]);
            if (p.w_post) {
                const float ah = scale(j) * load1<DT>(p.h, h0 + j);
                v[1] = fmaf(ah, fmaf(k2, u, d), v[1]);
                v[2] = fmaf(ah, s, v[2]);
            }
        }
        block_sums<3>(v, part, parity);
        const float e = k2 * k2 * k2 * (v[0] / p.n);
        const float f = k1 * k1 * (fmaf(-e, v[2], v[1]) / p.n);
        for (int64_t j = tid; j < p.N; j += T) {
            float t = p.ds ? load1<DT>(p.ds, ds0 + j) : 0.f;
            const float a = scale(j);
            const float h = load1<DT>(p.h, h0 + j);
            if (p.w_pre) {
                const float s = load1<DT>(p.s, s0 + j), dy = load1<DT>(p.dy, dy0 + j);
                t = fmaf(k2, dy * (p.offset + load1<DT>(p.w_pre, j)), t);
                t = fmaf(-e, s, t);
                acc_pre[j] = fmaf(dy, s * k2, acc_pre[j]);
            }
            const float th = t * (h * k1);
            store1<DT>(p.dr, row * p.lddr + j, p.beta * t);
            store1<DT>(p.dh, row * p.lddh + j, p.w_post ? k1 * fmaf(a, t, -h * f) : a * t);
            if (per_element) {
                const float gw = p.alpha * th;
                store1<DT>(p.dgate, row * p.lddg + j,
                           p.w_post ? gw * (p.offset + load1<DT>(p.w_post, j)) : gw);
                if (p.w_post) acc_post[j] = fmaf(gw, load1<DT>(p.gate, g0 + j), acc_post[j]);
            } else if (grouped) {
                acc_gate[j] += th;
            } else if (p.w_post) {
                acc_post[j] = fmaf(p.alpha, th, acc_post[j]);
            }
        }
        if (grouped && (row + 1 == r1 || (row + 1) % p.gate_rows == 0)) {
            const int64_t first = grow * p.gate_rows;
            const int64_t last = first + p.gate_rows < p.M ? first + p.gate_rows : p.M;
            const bool whole = first >= r0 && last <= r1;
            for (int64_t j = tid; j < p.N; j += T) {
                const float q = p.alpha * acc_gate[j];
                if (p.w_post) acc_post[j] = fmaf(q, load1<DT>(p.gate, g0 + j), acc_post[j]);
                if (whole)
                    store1<DT>(p.dgate, grow * p.lddg + j,
                               p.w_post ? q * (p.offset + load1<DT>(p.w_post, j)) : q);
            }
        }
    }
    pdl_launch_dependents();
}

// Sums of the partial rows in CTA order: dw_post, dw_pre, and the gate rows
// that more than one CTA worked on. blockIdx.y is the row summed: 0 dw_post,
// 1 dw_pre, then one per gate row.
template <int DT>
__global__ void __launch_bounds__(256) block_bwd_finish_kernel(const BlockBwdP p, int64_t G) {
    const int64_t pitch = block_bwd_pitch(p.N);
    const int64_t j = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    pdl_wait();
    if (j >= p.N) return;
    for (int64_t item = blockIdx.y;; item += gridDim.y) {
        if (item < 2) {
            float* out = item == 0 ? p.dw_post : p.dw_pre;
            if (!out) continue;
            float t = 0.f;
            for (int64_t b = 0; b < G; ++b)
                t += partial(p.ws, static_cast<int>(item), b, G, pitch)[j];
            out[j] = t;
            continue;
        }
        const int64_t grow = item - 2;
        if (!p.gate || p.gate_rows == 1 || grow * p.gate_rows >= p.M) return;
        const int64_t first = grow * p.gate_rows;
        const int64_t last = first + p.gate_rows < p.M ? first + p.gate_rows : p.M;
        const int64_t b0 = range_owner(first, G, p.M), b1 = range_owner(last - 1, G, p.M);
        if (b0 == b1) continue;
        float t = 0.f;
        for (int64_t b = b0; b <= b1; ++b) {
            const int area = b == b0 && range_begin(b, G, p.M) < first ? 3 : 2;
            t += partial(p.ws, area, b, G, pitch)[j];
        }
        t *= p.alpha;
        if (p.w_post) t *= p.offset + load1<DT>(p.w_post, j);
        store1<DT>(p.dgate, grow * p.lddg + j, t);
    }
}

template <int DT>
cudaError_t run(const BlockBwdP& p, const OpCfg& c) {
    int T = 32;
    while (T < 512 && static_cast<int64_t>(T) * 4 < p.N) T <<= 1;
    auto fn = block_bwd_generic_kernel<DT>;
    const int occ = occupancy(reinterpret_cast<const void*>(fn), T, 0);
    const int64_t cap = block_bwd_max_grid(p.M, p.N, c.dev.sm_count);
    const int64_t G = std::min<int64_t>(
        cap, persistent_grid(p.M, 1, c.dev.sm_count, occ, c.max_ctas));
    cudaError_t e = op_launch(c, fn, G, T, 0, p);
    const int64_t grows = p.gate && p.gate_rows > 1 ? (p.M + p.gate_rows - 1) / p.gate_rows : 0;
    if (e != cudaSuccess || (!p.dw_post && !p.dw_pre && grows == 0)) return e;
    Launch l;
    l.grid = static_cast<int>((p.N + 255) / 256);
    l.threads = 256;
    LaunchCfg cfg(l, c.stream, c.pdl);
    cfg.cfg.gridDim.y = static_cast<unsigned>(std::min<int64_t>(2 + grows, 1024));
    return cudaLaunchKernelEx(&cfg.cfg, block_bwd_finish_kernel<DT>, p, G);
}

}  // namespace

int block_bwd_max_grid(int64_t M, int64_t N, int sm_count) {
    // Up to eight CTAs per SM; for very long rows fewer, so that the partial
    // rows stay within about 256 MB.
    const int64_t rows = (int64_t(1) << 28) / (kBlockBwdRows * 4 * block_bwd_pitch(N));
    const int64_t g = std::min<int64_t>(M, std::min<int64_t>(8LL * sm_count, std::max<int64_t>(rows, 1)));
    return static_cast<int>(std::max<int64_t>(g, 1));
}

cudaError_t block_bwd_run(const BlockBwdP& p, const OpCfg& c) {
    switch (p.dtype) {
        case kBF16: return run<kBF16>(p, c);
        case kFP16: return run<kFP16>(p, c);
        default: return run<kFP32>(p, c);
    }
}

}  // namespace rmsn
