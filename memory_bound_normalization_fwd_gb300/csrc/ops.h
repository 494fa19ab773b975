// Internal interface between the front end of the block, rope and cache
// operators (api_ops.cu) and their kernels. Everything here is validated.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace rmsn {

// Launch knobs of these operators (from rmsnorm_options_t) and the device.
struct OpCfg {
    int variant = 0;  // RMSNORM_VARIANT_AUTO, _CTA (vector kernels) or _GENERIC (element-wise)
    int max_ctas = 0;
    bool pdl = true;
    int64_t wait_limit_ns = 0;  // bound of a wait in the kernels that stage rows; 0: one second
    DeviceInfo dev;
    cudaStream_t stream = nullptr;
};

// Launches `fn` with programmatic stream serialisation unless turned off.
template <typename... P, typename... A>
cudaError_t op_launch(const OpCfg& c, void (*fn)(P...), int64_t grid, int threads, int smem,
                      A... args) {
    Launch l;
    l.grid = static_cast<int>(grid);
    l.threads = threads;
    l.smem = smem;
    LaunchCfg cfg(l, c.stream, c.pdl);
    return cudaLaunchKernelEx(&cfg.cfg, fn, static_cast<P>(args)...);
}

// ---- block --------------------------------------------------------------------

struct BlockP {
    const void* h;
    const void* r;
    const void* w_post;  // null: no norm after the block
    const void* gate;    // null: no gate
    const void* w_pre;   // null: no norm before the next block
    void* s;
    void* y;
    float* rstd_post;
    float* rstd_pre;
    int64_t M, N, gate_rows;
    int64_t ldh, ldr, ldg, lds, ldy;
    float n, eps, offset, alpha, beta;
    int dtype;
};

struct BlockBwdP {
    const void* h;
    const void* s;
    const void* w_post;
    const void* gate;
    const void* w_pre;
    const float* rstd_post;
    const float* rstd_pre;
    const void* dy;  // null exactly when w_pre is
    const void* ds;  // may be null when dy is not
    void* dh;
    void* dr;
    void* dgate;
    float* dw_post;
    float* dw_pre;
    int64_t M, N, gate_rows;
    int64_t ldh, lds, ldg, lddy, ldds, lddh, lddr, lddg;
    float n, offset, alpha, beta;
    int dtype;
    float* ws;  // partial rows, see block_bwd_ws
};

cudaError_t block_fwd_run(const BlockP& p, const OpCfg& c);
cudaError_t block_bwd_run(const BlockBwdP& p, const OpCfg& c);
cudaError_t block_status_read_and_clear(unsigned int* value);
cudaError_t block_bwd_status_read_and_clear(unsigned int* value);

// The backward's grid never exceeds this (partial rows are counted by it).
int block_bwd_max_grid(int64_t M, int64_t N, int sm_count);
// Floats per partial row: N rounded up to whole 16-byte vectors.
__host__ __device__ inline int64_t block_bwd_pitch(int64_t N) { return (N + 3) / 4 * 4; }
// Partial rows per CTA: dw_post, dw_pre, and the gate sums of the first and the
// last gate row that a CTA's rows touch.
constexpr int kBlockBwdRows = 4;

// ---- rope ---------------------------------------------------------------------

struct HeadsP {
    void* p;
    int64_t sb, st, sh;  // strides of batch, token, head in elements
};

// One of q and k: what a launch needs for its heads.
struct RopeSeg {
    HeadsP in;    // forward: x; backward: the gradient of the output
    HeadsP out;   // forward: the output; backward: the gradient of x
    HeadsP x;     // backward with weights: x
    const void* w;
    float* rstd;
    float* dw;    // backward with weights
    int heads;
};

struct RopeP {
    RopeSeg seg[2];
    const int64_t* positions;
    int64_t positions_stride;
    const uint64_t* steps;
    int64_t batch, seq;
    int D, R;
    int interleaved;
    float eps, offset, magnitude;
    int dtype;
    float* ws;  // backward: partial rows of D floats
};

cudaError_t rope_fwd_run(const RopeP& p, const OpCfg& c);
cudaError_t rope_bwd_run(const RopeP& p, const OpCfg& c);
// Partial rows of D floats that the backward may write, per device.
int64_t rope_bwd_partial_rows(int sm_count);

// ---- cache --------------------------------------------------------------------

struct CacheP {
    int format;
    int64_t slots;
    int64_t page_size;
    int heads, D;
    int code_bytes;   // of a head
    int groups;       // of a head
    int heads_first;
    uint8_t* codes[2];   // k, v (null: not in this call)
    uint8_t* scales[2];
    HeadsP t[2];         // the tensors written from or read into
    int dtype;
    // write
    const int64_t* slot;
    int64_t T;
    // read
    const int32_t* table;
    int64_t table_width;
    const int32_t* cu_rows;
    const int32_t* starts;
    int64_t sequences, rows;
};

cudaError_t cache_write_run(const CacheP& p, const OpCfg& c);
cudaError_t cache_read_run(const CacheP& p, const OpCfg& c);
cudaError_t cache_status_read_and_clear(unsigned int* value);

// Front end helpers shared with api.cu.
cudaError_t device_info(DeviceInfo* out);

}  // namespace rmsn
