// What the attention kernels share: which tokens a row sees, where a token lies, and
// how the work is dealt out.
#pragma once

#include "ops.h"
#include "ops_common.cuh"

#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

namespace rmsn {

// Sequence b of a call: its rows and tokens, kept within the call's arrays whatever the
// device arrays hold.
struct Sequence {
    int64_t row0;
    int64_t n, len;  // queries, tokens
    int64_t held;    // tokens that the row of the table has room for
};

__device__ __forceinline__ int64_t first_row(const AttnP& p, int64_t b) {
    if (!p.cu) return b;
    const int64_t c = __ldg(p.cu + b);
    return c < 0 ? 0 : c > p.rows ? p.rows : c;
}

__device__ __forceinline__ Sequence sequence(const AttnP& p, int64_t b) {
    Sequence s;
    s.row0 = first_row(p, b);
    const int64_t end = first_row(p, b + 1);
    s.n = end > s.row0 ? end - s.row0 : 0;
    const int64_t len = __ldg(p.lengths + b), most = p.width * p.page_size;
    s.len = len < 0 ? 0 : len;
    s.held = s.len < most ? s.len : most;
    return s;
}

// Tokens [low, high) that query i of a sequence sees.
struct Seen {
    int64_t low, high;
};

__device__ __forceinline__ Seen seen(const AttnP& p, const Sequence& s, int64_t i) {
    const int64_t pos = s.len - s.n + i;
    Seen r;
    r.high = p.causal && pos + 1 < s.held ? pos + 1 : s.held;
    r.low = p.window && pos + 1 > p.window ? pos + 1 - p.window : 0;
    if (r.high < 0) r.high = 0;
    return r;
}

// The index of (token t, cache head 0) among the cache's heads; -1 where its page is not
// there. Head h is h * head_step(p) further.
__device__ __forceinline__ int64_t token_at(const AttnP& p, int64_t b, int64_t t) {
    const uint32_t size = static_cast<uint32_t>(p.page_size);
    const uint32_t col = static_cast<uint32_t>(t) / size, off = static_cast<uint32_t>(t) - col * size;
    const int64_t page = __ldg(p.table + b * p.width + col);
    if (page < 0 || page * p.page_size >= p.slots) return -1;
    return p.heads_first ? page * p.heads * p.page_size + off : (page * p.page_size + off) * p.heads;
}
__device__ __forceinline__ int64_t head_step(const AttnP& p) { return p.heads_first ? p.page_size : 1; }

// 2^(byte - 127), NaN for 255.
__device__ __forceinline__ float scale_of(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte ? byte << 23 : 0x400000u);
}

}  // namespace rmsn
