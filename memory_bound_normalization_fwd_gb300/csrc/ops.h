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
    int axes;             // 1, or 2..4: axis a's positions lie at positions + a * axis_stride
    int in_turn;
    int cut[3];           // sections: first pair of the axes 1..3 (past them: R / 2);
                          // in turn: pairs of the axes 1..3
    int64_t axis_stride;
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

// ---- pages of the cache ---------------------------------------------------------

// What a page of the four arrays (k and v codes, k and v scales; null: not there) is
// made of: `runs` runs of `page_size` tokens of `token[a]` bytes (one run of all heads, or with
// heads first a run a head).
struct PageBytes {
    uint8_t* p[4];
    int64_t page[4];   // bytes of a page
    int64_t token[4];  // bytes of a token in a run
    int runs;
    int page_size;
    bool vectors;      // every page a multiple of 16 bytes at such an address
};

constexpr int64_t kMaxPages = int64_t(1) << 25;  // that fork and compact take

struct PagesP {
    PageBytes bytes;
    int64_t pages, sequences, width;
    int32_t* refs;
    int32_t* table;
    int32_t* lengths;
    int64_t n;
    // copy: src, dst; fork: parents, children; free: rows
    const int32_t* a;
    const int32_t* b;
    // compact
    int32_t* refs_out;
    int32_t* table_out;
    int32_t* live;
    void* ws;
};

cudaError_t pages_copy_run(const PagesP& p, const OpCfg& c);
cudaError_t pages_fork_run(const PagesP& p, const OpCfg& c);
cudaError_t pages_free_run(const PagesP& p, const OpCfg& c);
cudaError_t pages_compact_run(const PagesP& p, const OpCfg& c);
cudaError_t pages_status_read_and_clear(unsigned int* value);
int64_t pages_ws_bytes(int64_t pages, int64_t sequences, int64_t n);

// ---- attention over the cache -----------------------------------------------------

struct AttnP {
    int format;
    int64_t slots;
    int page_size, heads, D, code_bytes, groups, heads_first;
    const uint8_t* codes[2];
    const uint8_t* scales[2];
    HeadsP q, out;
    int dtype;
    int heads_q, G;  // query heads, and those of a cache head
    int causal;
    int64_t window;
    int64_t sequences, rows, width;
    const int32_t* table;
    const int32_t* lengths;
    const int32_t* cu;  // null: a row a sequence
    float* lse;
    float scale;
    void* ws;
    unsigned int* status;  // the device's word for pages that are not there
    unsigned int* late;    // and for waits that ran out
};

cudaError_t attn_run(const AttnP& p, const OpCfg& c);
cudaError_t attn_status_read_and_clear(unsigned int* value);
cudaError_t attn_late_read_and_clear(unsigned int* value);
int64_t attn_ws_bytes(int64_t heads, int64_t G, int64_t D, int64_t sequences, int64_t rows, int sm_count);

// Front end helpers shared with api.cu.
cudaError_t device_info(DeviceInfo* out);

}  // namespace rmsn
