// Argument checks on the host that the C entry points of the operators share:
// arrays and their overlaps, options, heads tensors, the cache.
#pragma once

#include "rmsnorm.h"

#include "ops.h"

#include <algorithm>
#include <cmath>

namespace rmsn {

constexpr int64_t kSpanLimit = int64_t(1) << 48;  // bytes any array may span

inline bool dtype_ok(int dtype) {
    return dtype == RMSNORM_DTYPE_BF16 || dtype == RMSNORM_DTYPE_FP16 || dtype == RMSNORM_DTYPE_FP32;
}

// A strided array: up to three dimensions of (count, stride in bytes) around
// `inner` contiguous bytes. For overlap checks.
struct View {
    uintptr_t base = 0;
    int64_t inner = 0;
    int n = 0;
    int64_t count[3] = {0, 0, 0}, stride[3] = {0, 0, 0};

    View() {}
    View(const void* p, int64_t bytes) : base(reinterpret_cast<uintptr_t>(p)), inner(bytes) {}
    View& dim(int64_t c, int64_t s) {
        if (c > 1) {
            count[n] = c;
            stride[n++] = s;
        }
        return *this;
    }
    bool empty() const { return base == 0 || inner == 0; }
    // Bytes from the first to the last, over the dimensions with a stride below `m`.
    int64_t extent(int64_t m) const {
        int64_t e = inner;
        for (int i = 0; i < n; ++i)
            if (stride[i] < m) e += (count[i] - 1) * stride[i];
        return e;
    }
    int64_t span() const { return extent(INT64_MAX); }
    // Every stride of `m` bytes and above is a multiple of m.
    bool periodic(int64_t m) const {
        for (int i = 0; i < n; ++i)
            if (stride[i] >= m && stride[i] % m != 0) return false;
        return extent(m) <= m;
    }
    // No element of the array lies on another.
    bool distinct() const {
        for (int i = 0; i < n; ++i) {
            int64_t e = inner;
            for (int k = 0; k < n; ++k)
                if (stride[k] < stride[i] || (stride[k] == stride[i] && k < i))
                    e += (count[k] - 1) * stride[k];
            if (stride[i] < e) return false;
        }
        return true;
    }
    bool same(const View& o) const {
        if (base != o.base || inner != o.inner || n != o.n) return false;
        for (int i = 0; i < n; ++i)
            if (count[i] != o.count[i] || stride[i] != o.stride[i]) return false;
        return true;
    }
};

// Whether two arrays may share a byte: their spans meet, and no stride that
// divides both of them into periods keeps them in different parts of a period
// (as for q and k as slices of one projection's rows).
inline bool meet(const View& a, const View& b) {
    if (a.empty() || b.empty()) return false;
    if (a.base >= b.base + static_cast<uintptr_t>(b.span()) ||
        b.base >= a.base + static_cast<uintptr_t>(a.span()))
        return false;
    for (int v = 0; v < 2; ++v) {
        const View& w = v == 0 ? a : b;
        for (int i = 0; i < w.n; ++i) {
            const int64_t m = w.stride[i];
            if (m <= 0 || !a.periodic(m) || !b.periodic(m)) continue;
            const int64_t d = static_cast<int64_t>(
                b.base >= a.base ? (b.base - a.base) % static_cast<uintptr_t>(m)
                                 : (m - static_cast<int64_t>((a.base - b.base) % static_cast<uintptr_t>(m))) % m);
            if (d >= a.extent(m) && d + b.extent(m) <= m) return false;
        }
    }
    return true;
}

inline int read_op_options(const rmsnorm_options_t* opts, OpCfg* c) {
    int variant;
    Knobs k;
    const int rc = read_knobs(opts, &variant, &k);
    if (rc != RMSNORM_OK) return rc;
    if (variant != RMSNORM_VARIANT_AUTO && variant != RMSNORM_VARIANT_CTA &&
        variant != RMSNORM_VARIANT_GENERIC)
        return fail(RMSNORM_ERR_UNSUPPORTED, "the operators have the variants AUTO, CTA and GENERIC only");
    c->variant = variant;
    c->max_ctas = k.max_ctas;
    c->pdl = (k.flags & RMSNORM_FLAG_NO_PDL) == 0;
    c->wait_limit_ns = k.wait_limit_ns < 60000000000LL ? k.wait_limit_ns : 60000000000LL;
    return RMSNORM_OK;
}

inline int finish_cfg(OpCfg* c, void* stream) {
    c->stream = static_cast<cudaStream_t>(stream);
    const cudaError_t e = device_info(&c->dev);
    if (e != cudaSuccess) return fail(RMSNORM_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
    return RMSNORM_OK;
}

// Plans and launches, and reports. The plans' caches allocate host memory: no
// exception leaves the C entry points.
template <typename F>
inline int launched(F run) {
    cudaError_t e;
    try {
        e = run();
    } catch (...) {
        e = cudaErrorMemoryAllocation;
    }
    if (e == cudaErrorNotSupported)
        return fail(RMSNORM_ERR_UNSUPPORTED, "the vector kernels cannot take these sizes, strides or alignments");
    if (e != cudaSuccess) return fail(RMSNORM_ERR_CUDA, "launch: %s", cudaGetErrorString(e));
    return RMSNORM_OK;
}

inline int clear_floats(float* p, int64_t n, void* stream) {
    if (!p) return RMSNORM_OK;
    const cudaError_t e = cudaMemsetAsync(p, 0, static_cast<size_t>(n) * 4, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(RMSNORM_ERR_CUDA, "memset: %s", cudaGetErrorString(e));
    return RMSNORM_OK;
}

inline bool misaligned(const void* p, int64_t to) {
    return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(to - 1)) != 0;
}

// An argument: its array, its name, and a mark. An output may lie exactly on an
// input of the same mark (not 0): those that one thread reads before it writes.
struct Named {
    View v;
    const char* name;
    int mark;
};

inline int check_overlaps(const Named* outs, int nout, const Named* ins, int nin) {
    for (int i = 0; i < nout; ++i) {
        if (outs[i].v.empty()) continue;
        if (!outs[i].v.distinct())
            return fail(RMSNORM_ERR_OVERLAP, "%s overlaps itself (strides)", outs[i].name);
        for (int k = 0; k < i; ++k)
            if (meet(outs[i].v, outs[k].v))
                return fail(RMSNORM_ERR_OVERLAP, "%s overlaps %s", outs[i].name, outs[k].name);
        for (int k = 0; k < nin; ++k) {
            if (!meet(outs[i].v, ins[k].v)) continue;
            const bool pair = outs[i].mark != 0 && outs[i].mark == ins[k].mark;
            if (pair && outs[i].v.same(ins[k].v)) continue;
            return fail(RMSNORM_ERR_OVERLAP, "%s overlaps %s%s", outs[i].name, ins[k].name,
                        pair ? " without being equal to it" : "");
        }
    }
    return RMSNORM_OK;
}

// Strides of a heads tensor: not negative, and the span within 2^48 bytes.
inline int check_heads(const char* name, const rmsnorm_heads_t& h, int64_t batch, int64_t seq, int64_t heads,
                int64_t D, int64_t eb) {
    if (h.ptr == nullptr) return fail(RMSNORM_ERR_NULL, "%s is NULL", name);
    const int64_t count[3] = {batch, seq, heads};
    const int64_t stride[3] = {h.batch_stride, h.token_stride, h.head_stride};
    int64_t span = D;
    for (int i = 0; i < 3; ++i) {
        if (count[i] <= 1) continue;
        if (stride[i] < 0) return fail(RMSNORM_ERR_SHAPE, "%s has a negative stride", name);
        if (stride[i] > kSpanLimit / eb / (count[i] - 1))
            return fail(RMSNORM_ERR_SHAPE, "%s would span more than 2^48 bytes", name);
        span += (count[i] - 1) * stride[i];
    }
    if (span > kSpanLimit / eb) return fail(RMSNORM_ERR_SHAPE, "%s would span more than 2^48 bytes", name);
    if (misaligned(h.ptr, eb))
        return fail(RMSNORM_ERR_ALIGN, "%s must be aligned to the element size (%d bytes)", name,
                    static_cast<int>(eb));
    return RMSNORM_OK;
}

inline View heads_view(const rmsnorm_heads_t& h, int64_t batch, int64_t seq, int64_t heads, int64_t D, int64_t eb) {
    return View(h.ptr, D * eb)
        .dim(batch, h.batch_stride * eb)
        .dim(seq, h.token_stride * eb)
        .dim(heads, h.head_stride * eb);
}

inline HeadsP heads_p(const rmsnorm_heads_t& h) { return {h.ptr, h.batch_stride, h.token_stride, h.head_stride}; }

inline int cache_shapes(const rmsnorm_cache_t* c, int dtype, CacheP* p) {
    if (c == nullptr) return fail(RMSNORM_ERR_NULL, "cache is NULL");
    if (c->struct_size != static_cast<int32_t>(sizeof(*c)))
        return fail(RMSNORM_ERR_OPTIONS, "cache.struct_size is %d, expected %d", c->struct_size,
                    static_cast<int>(sizeof(*c)));
    if (c->format != RMSNORM_CACHE_E4M3 && c->format != RMSNORM_CACHE_E2M1)
        return fail(RMSNORM_ERR_DTYPE, "format %d is not a rmsnorm_cache_format_t", c->format);
    if (!dtype_ok(dtype)) return fail(RMSNORM_ERR_DTYPE, "dtype %d is not a rmsnorm_dtype_t", dtype);
    if (c->pages < 1 || c->page_size < 1 || c->heads < 1 || c->heads > (1 << 20) || c->head_dim < 1 ||
        c->head_dim > 65536 || (c->heads_first != 0 && c->heads_first != 1))
        return fail(RMSNORM_ERR_SHAPE, "the cache needs pages, page_size and heads >= 1, head_dim in "
                    "1..65536 and heads_first 0 or 1");
    *p = CacheP{};
    p->format = c->format;
    p->page_size = c->page_size;
    p->heads = c->heads;
    p->D = c->head_dim;
    p->code_bytes = c->format == RMSNORM_CACHE_E4M3 ? c->head_dim : (c->head_dim + 1) / 2;
    p->groups = (c->head_dim + 31) / 32;
    p->heads_first = c->heads_first;
    p->dtype = dtype;
    const int64_t per_page = static_cast<int64_t>(c->heads) * p->code_bytes;
    if (c->pages > kSpanLimit / c->page_size / per_page)
        return fail(RMSNORM_ERR_SHAPE, "the cache would span more than 2^48 bytes");
    p->slots = c->pages * c->page_size;
    if (!c->k_codes || !c->k_scales || (c->v_codes != nullptr) != (c->v_scales != nullptr))
        return fail(RMSNORM_ERR_NULL, "k_codes and k_scales must be given, v_codes and v_scales together");
    return RMSNORM_OK;
}

inline Named cache_array(const rmsnorm_cache_t* c, const CacheP& p, int which) {
    const int64_t heads = p.slots * p.heads;
    switch (which) {
        case 0: return {View(c->k_codes, heads * p.code_bytes), "k_codes", 0};
        case 1: return {View(c->k_scales, heads * p.groups), "k_scales", 0};
        case 2: return {View(c->v_codes, heads * p.code_bytes), "v_codes", 0};
        default: return {View(c->v_scales, heads * p.groups), "v_scales", 0};
    }
}

}  // namespace rmsn
