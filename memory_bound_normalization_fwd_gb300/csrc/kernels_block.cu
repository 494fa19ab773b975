// The norm after a block, its gate, the scaled residual and the norm before
// the next block (the operation is stated in include/rmsnorm.h).
//
// Both norms need a whole row's sum before the row can go on, and the second
// sum is over what the first norm makes: two row reductions in sequence, with
// 2 reads and 2 writes of a row around them. The bound is HBM: 4 M N elements.
#include "rmsnorm.h"

#include "ops.h"
#include "ops_common.cuh"

namespace rmsn {
namespace {

// Element-wise kernel: any N, alignment and stride. One CTA per row, three
// passes over the row's columns (sum of h^2; sum of s^2 over s recomputed from
// h and r; s again, stored, and y), the later ones from L1/L2. A thread reads
// a column of h and r and then writes it, and no other pass follows, so s and
// y may lie on h and r.
template <int DT>
__global__ void __launch_bounds__(512) block_fwd_generic_kernel(const BlockP p) {
    __shared__ float part[2 * 32];
    int parity = 0;
    const int tid = threadIdx.x, T = blockDim.x;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        const int64_t h0 = row * p.ldh, r0 = row * p.ldr;
        const int64_t g0 = p.gate ? row / p.gate_rows * p.ldg : 0;
        float a = 1.f;
        if (p.w_post) {
            float ss[1] = {0.f};
            for (int64_t j = tid; j < p.N; j += T) {
                const float f = load1<DT>(p.h, h0 + j);
                ss[0] = fmaf(f, f, ss[0]);
            }
            block_sums<1>(ss, part, parity);
            a = row_rstd(ss[0], p.n, p.eps);
            if (tid == 0 && p.rstd_post) p.rstd_post[row] = a;
        }
        auto residual = [&](int64_t j) {
            float n = load1<DT>(p.h, h0 + j);
            if (p.w_post) n = n * a * (p.offset + load1<DT>(p.w_post, j));
            if (p.gate) n *= load1<DT>(p.gate, g0 + j);
            return fmaf(p.beta, load1<DT>(p.r, r0 + j), p.alpha * n);
        };
        float b = 0.f;
        if (p.w_pre) {
            float ss[1] = {0.f};
            for (int64_t j = tid; j < p.N; j += T) {
                const float f = residual(j);
                ss[0] = fmaf(f, f, ss[0]);
            }
            block_sums<1>(ss, part, parity);
            b = row_rstd(ss[0], p.n, p.eps);
            if (tid == 0 && p.rstd_pre) p.rstd_pre[row] = b;
        }
        for (int64_t j = tid; j < p.N; j += T) {
            const float f = residual(j);
            store1<DT>(p.s, row * p.lds + j, f);
            if (p.w_pre)
                store1<DT>(p.y, row * p.ldy + j, f * b * (p.offset + load1<DT>(p.w_pre, j)));
        }
    }
}

template <int DT>
cudaError_t run(const BlockP& p, const OpCfg& c) {
    int T = 32;
    while (T < 512 && static_cast<int64_t>(T) * 4 < p.N) T <<= 1;
    auto fn = block_fwd_generic_kernel<DT>;
    const int occ = occupancy(reinterpret_cast<const void*>(fn), T, 0);
    return op_launch(c, fn, persistent_grid(p.M, 1, c.dev.sm_count, occ, c.max_ctas), T, 0, p);
}

}  // namespace

cudaError_t block_fwd_run(const BlockP& p, const OpCfg& c) {
    switch (p.dtype) {
        case kBF16: return run<kBF16>(p, c);
        case kFP16: return run<kFP16>(p, c);
        default: return run<kFP32>(p, c);
    }
}

}  // namespace rmsn
