// C ABI front end of the block, rope and cache operators: argument validation
// on the host before any CUDA call, then the launch. The operations are
// stated in include/rmsnorm.h.
#include "rmsnorm.h"

#include "ops.h"

#include <algorithm>
#include <cmath>

namespace rmsn {
namespace {

constexpr int64_t kSpanLimit = int64_t(1) << 48;  // bytes any array may span

bool dtype_ok(int dtype) {
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
bool meet(const View& a, const View& b) {
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

int read_op_options(const rmsnorm_options_t* opts, OpCfg* c) {
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

int finish_cfg(OpCfg* c, void* stream) {
    c->stream = static_cast<cudaStream_t>(stream);
    const cudaError_t e = device_info(&c->dev);
    if (e != cudaSuccess) return fail(RMSNORM_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
    return RMSNORM_OK;
}

// Plans and launches, and reports. The plans' caches allocate host memory: no
// exception leaves the C entry points.
template <typename F>
int launched(F run) {
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

int clear_floats(float* p, int64_t n, void* stream) {
    if (!p) return RMSNORM_OK;
    const cudaError_t e = cudaMemsetAsync(p, 0, static_cast<size_t>(n) * 4, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail(RMSNORM_ERR_CUDA, "memset: %s", cudaGetErrorString(e));
    return RMSNORM_OK;
}

bool misaligned(const void* p, int64_t to) {
    return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(to - 1)) != 0;
}

// An argument: its array, its name, and a mark. An output may lie exactly on an
// input of the same mark (not 0): those that one thread reads before it writes.
struct Named {
    View v;
    const char* name;
    int mark;
};

int check_overlaps(const Named* outs, int nout, const Named* ins, int nin) {
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

// ---- block --------------------------------------------------------------------

int block_shapes(const rmsnorm_block_args_t* a, bool need_r) {
    if (a == nullptr) return fail(RMSNORM_ERR_NULL, "args is NULL");
    if (a->struct_size != static_cast<int32_t>(sizeof(*a)))
        return fail(RMSNORM_ERR_OPTIONS, "args.struct_size is %d, expected %d", a->struct_size,
                    static_cast<int>(sizeof(*a)));
    if (!dtype_ok(a->dtype)) return fail(RMSNORM_ERR_DTYPE, "dtype %d is not a rmsnorm_dtype_t", a->dtype);
    if (a->M < 0 || a->N <= 0 || a->N > (int64_t(1) << 31))
        return fail(RMSNORM_ERR_SHAPE, "need M >= 0 and 0 < N <= 2^31 (got M=%lld N=%lld)",
                    static_cast<long long>(a->M), static_cast<long long>(a->N));
    // A gate of no rows may have no address.
    if (a->gate ? a->gate_rows < 1 : a->M == 0 ? a->gate_rows < 0 : a->gate_rows != 0)
        return fail(RMSNORM_ERR_SHAPE, "gate_rows is %lld: rows per gate row (>= 1), 0 without a gate",
                    static_cast<long long>(a->gate_rows));
    if (!std::isfinite(a->offset) || !std::isfinite(a->alpha) || !std::isfinite(a->beta))
        return fail(RMSNORM_ERR_SCALAR, "offset, alpha and beta must be finite");
    if (need_r && (!std::isfinite(a->eps) || a->eps < 0.f))
        return fail(RMSNORM_ERR_SCALAR, "eps must be finite and >= 0 (got %g)", a->eps);
    return RMSNORM_OK;
}

// Rows of h per gate row as the kernels take them: what lies past the last row
// is left out, so that a product with it stays small (more than one stays so).
int64_t gate_rows_of(const rmsnorm_block_args_t* a) {
    return a->gate ? std::min(a->gate_rows, std::max<int64_t>(a->M, 2)) : 0;
}

int check_ld(const char* name, int64_t ld, int64_t rows, int64_t N, int64_t eb) {
    if (ld < N)
        return fail(RMSNORM_ERR_SHAPE, "the row stride of %s is %lld, below N", name,
                    static_cast<long long>(ld));
    if (rows > 0 && (rows > (int64_t(1) << 46) || ld > kSpanLimit / eb / rows))
        return fail(RMSNORM_ERR_SHAPE, "%s would span more than 2^48 bytes", name);
    return RMSNORM_OK;
}

}  // namespace
}  // namespace rmsn

using namespace rmsn;

extern "C" int rmsnorm_block_fwd(const rmsnorm_block_args_t* a, const rmsnorm_options_t* opts,
                                 void* stream) {
    int rc = block_shapes(a, true);
    if (rc != RMSNORM_OK) return rc;
    OpCfg c;
    rc = read_op_options(opts, &c);
    if (rc != RMSNORM_OK) return rc;
    if (!a->w_post && !a->w_pre)
        return fail(RMSNORM_ERR_NULL, "at least one of w_post and w_pre must be given");
    if ((a->w_pre != nullptr) != (a->y != nullptr) && a->M > 0)
        return fail(RMSNORM_ERR_NULL, "y is given exactly when w_pre is");
    if (a->M == 0) return RMSNORM_OK;
    if (!a->h || !a->r || !a->s) return fail(RMSNORM_ERR_NULL, "h, r and s must be non-NULL");
    const int64_t eb = elem_bytes(a->dtype), N = a->N, M = a->M;
    const int64_t gate_rows = gate_rows_of(a);
    const int64_t grows = a->gate ? (M + gate_rows - 1) / gate_rows : 0;
    if ((rc = check_ld("h", a->ldh, M, N, eb)) || (rc = check_ld("r", a->ldr, M, N, eb)) ||
        (rc = check_ld("s", a->lds, M, N, eb)) ||
        (a->y && (rc = check_ld("y", a->ldy, M, N, eb))) ||
        (a->gate && (rc = check_ld("gate", a->ldg, grows, N, eb))))
        return rc;
    const void* elems[] = {a->h, a->r, a->w_post, a->gate, a->w_pre, a->s, a->y};
    for (const void* p : elems)
        if (misaligned(p, eb))
            return fail(RMSNORM_ERR_ALIGN, "tensors must be aligned to the element size (%d bytes)",
                        static_cast<int>(eb));
    if (misaligned(a->rstd_post, 4) || misaligned(a->rstd_pre, 4))
        return fail(RMSNORM_ERR_ALIGN, "rstd_post and rstd_pre must be 4-byte aligned");
    auto rows = [&](const void* p, int64_t ld, int64_t n) { return View(p, N * eb).dim(n, ld * eb); };
    const Named outs[] = {{rows(a->s, a->lds, M), "s", 1},
                          {rows(a->y, a->ldy, M), "y", 1},
                          {View(a->rstd_post, M * 4), "rstd_post", 0},
                          {View(a->rstd_pre, M * 4), "rstd_pre", 0}};
    const Named ins[] = {{rows(a->h, a->ldh, M), "h", 1},
                         {rows(a->r, a->ldr, M), "r", 1},
                         {View(a->w_post, N * eb), "w_post", 0},
                         {View(a->w_pre, N * eb), "w_pre", 0},
                         {rows(a->gate, a->ldg, grows), "gate", 0}};
    rc = check_overlaps(outs, 4, ins, 5);
    if (rc != RMSNORM_OK) return rc;
    rc = finish_cfg(&c, stream);
    if (rc != RMSNORM_OK) return rc;
    const BlockP p{a->h, a->r, a->w_post, a->gate, a->w_pre, a->s, a->y, a->rstd_post, a->rstd_pre,
                   M, N, gate_rows, a->ldh, a->ldr, a->ldg, a->lds, a->ldy,
                   static_cast<float>(N), a->eps, a->offset, a->alpha, a->beta, a->dtype};
    return launched([&] { return block_fwd_run(p, c); });
}

extern "C" int rmsnorm_block_bwd_workspace_size(int64_t M, int64_t N, int dtype, int64_t* bytes) {
    if (bytes == nullptr) return fail(RMSNORM_ERR_NULL, "bytes is NULL");
    *bytes = 0;
    if (!dtype_ok(dtype)) return fail(RMSNORM_ERR_DTYPE, "dtype %d is not a rmsnorm_dtype_t", dtype);
    if (M < 0 || N <= 0 || N > (int64_t(1) << 31))
        return fail(RMSNORM_ERR_SHAPE, "need M >= 0 and 0 < N <= 2^31");
    DeviceInfo d;
    const cudaError_t e = device_info(&d);
    if (e != cudaSuccess) return fail(RMSNORM_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
    *bytes = static_cast<int64_t>(block_bwd_max_grid(M, N, d.sm_count)) * kBlockBwdRows *
             block_bwd_pitch(N) * 4;
    return RMSNORM_OK;
}

extern "C" int rmsnorm_block_bwd(const rmsnorm_block_args_t* a, const rmsnorm_block_grads_t* g,
                                 void* workspace, int64_t workspace_bytes,
                                 const rmsnorm_options_t* opts, void* stream) {
    int rc = block_shapes(a, false);
    if (rc != RMSNORM_OK) return rc;
    if (g == nullptr) return fail(RMSNORM_ERR_NULL, "grads is NULL");
    if (g->struct_size != static_cast<int32_t>(sizeof(*g)) || g->reserved != 0)
        return fail(RMSNORM_ERR_OPTIONS, "grads.struct_size is %d, expected %d (reserved 0)",
                    g->struct_size, static_cast<int>(sizeof(*g)));
    OpCfg c;
    rc = read_op_options(opts, &c);
    if (rc != RMSNORM_OK) return rc;
    if (!a->w_post && !a->w_pre)
        return fail(RMSNORM_ERR_NULL, "at least one of w_post and w_pre must be given");
    if ((a->w_post != nullptr) != (g->dw_post != nullptr) || (a->w_pre != nullptr) != (g->dw_pre != nullptr))
        return fail(RMSNORM_ERR_NULL, "dw_post and dw_pre are given exactly when w_post and w_pre are");
    const int64_t eb = elem_bytes(a->dtype), N = a->N, M = a->M;
    if (misaligned(g->dw_post, 4) || misaligned(g->dw_pre, 4))
        return fail(RMSNORM_ERR_ALIGN, "dw_post and dw_pre must be 4-byte aligned");
    if (M == 0) {
        const Named outs0[] = {{View(g->dw_post, N * 4), "dw_post", 0}, {View(g->dw_pre, N * 4), "dw_pre", 0}};
        const Named ins0[] = {{View(a->w_post, N * eb), "w_post", 0}, {View(a->w_pre, N * eb), "w_pre", 0}};
        rc = check_overlaps(outs0, 2, ins0, 2);
        if (rc == RMSNORM_OK) rc = clear_floats(g->dw_post, N, stream);
        if (rc == RMSNORM_OK) rc = clear_floats(g->dw_pre, N, stream);
        return rc;
    }
    if ((a->w_pre != nullptr) != (g->dy != nullptr))
        return fail(RMSNORM_ERR_NULL, "dy is given exactly when w_pre is");
    if (!g->dy && !g->ds) return fail(RMSNORM_ERR_NULL, "one of dy and ds must be given");
    if ((a->gate != nullptr) != (g->dgate != nullptr))
        return fail(RMSNORM_ERR_NULL, "dgate is given exactly when gate is");
    if (!a->h || !g->dh || !g->dr || !workspace)
        return fail(RMSNORM_ERR_NULL, "h, dh, dr and the workspace must be non-NULL");
    if (a->w_pre && (!a->s || !a->rstd_pre))
        return fail(RMSNORM_ERR_NULL, "s and rstd_pre must be given with w_pre");
    if (a->w_post && !a->rstd_post) return fail(RMSNORM_ERR_NULL, "rstd_post must be given with w_post");
    const void* s = a->w_pre ? a->s : nullptr;
    const int64_t gate_rows = gate_rows_of(a);
    const int64_t grows = a->gate ? (M + gate_rows - 1) / gate_rows : 0;
    if ((rc = check_ld("h", a->ldh, M, N, eb)) || (s && (rc = check_ld("s", a->lds, M, N, eb))) ||
        (g->dy && (rc = check_ld("dy", g->lddy, M, N, eb))) ||
        (g->ds && (rc = check_ld("ds", g->ldds, M, N, eb))) ||
        (rc = check_ld("dh", g->lddh, M, N, eb)) || (rc = check_ld("dr", g->lddr, M, N, eb)) ||
        (a->gate && ((rc = check_ld("gate", a->ldg, grows, N, eb)) ||
                     (rc = check_ld("dgate", g->lddg, grows, N, eb)))))
        return rc;
    const void* elems[] = {a->h, s, a->w_post, a->gate, a->w_pre, g->dy, g->ds, g->dh, g->dr, g->dgate};
    for (const void* p : elems)
        if (misaligned(p, eb))
            return fail(RMSNORM_ERR_ALIGN, "tensors must be aligned to the element size (%d bytes)",
                        static_cast<int>(eb));
    if (misaligned(a->rstd_post, 4) || misaligned(a->rstd_pre, 4))
        return fail(RMSNORM_ERR_ALIGN, "rstd_post and rstd_pre must be 4-byte aligned");
    if (misaligned(workspace, 16)) return fail(RMSNORM_ERR_ALIGN, "the workspace must be 16-byte aligned");
    auto rows = [&](const void* p, int64_t ld, int64_t n) { return View(p, N * eb).dim(n, ld * eb); };
    // The workspace is checked at the size given: the device's need is known below.
    const Named outs[] = {{rows(g->dh, g->lddh, M), "dh", 1},
                          {rows(g->dr, g->lddr, M), "dr", 1},
                          {rows(g->dgate, g->lddg, grows), "dgate", 0},
                          {View(g->dw_post, N * 4), "dw_post", 0},
                          {View(g->dw_pre, N * 4), "dw_pre", 0}};
    const Named ins[] = {{rows(a->h, a->ldh, M), "h", 1},
                         {rows(s, a->lds, M), "s", 1},
                         {rows(g->dy, g->lddy, M), "dy", 1},
                         {rows(g->ds, g->ldds, M), "ds", 1},
                         {View(a->w_post, N * eb), "w_post", 0},
                         {View(a->w_pre, N * eb), "w_pre", 0},
                         {rows(a->gate, a->ldg, grows), "gate", 0},
                         {View(a->w_post ? a->rstd_post : nullptr, M * 4), "rstd_post", 0},
                         {View(a->w_pre ? a->rstd_pre : nullptr, M * 4), "rstd_pre", 0}};
    rc = check_overlaps(outs, 5, ins, 9);
    if (rc != RMSNORM_OK) return rc;
    rc = finish_cfg(&c, stream);
    if (rc != RMSNORM_OK) return rc;
    const int64_t need = static_cast<int64_t>(block_bwd_max_grid(M, N, c.dev.sm_count)) * kBlockBwdRows *
                         block_bwd_pitch(N) * 4;
    if (workspace_bytes < need)
        return fail(RMSNORM_ERR_WORKSPACE, "workspace of %lld bytes, %lld needed",
                    static_cast<long long>(workspace_bytes), static_cast<long long>(need));
    const View ws(workspace, need);
    for (const Named& o : outs)
        if (meet(ws, o.v)) return fail(RMSNORM_ERR_OVERLAP, "the workspace overlaps %s", o.name);
    for (const Named& i : ins)
        if (meet(ws, i.v)) return fail(RMSNORM_ERR_OVERLAP, "the workspace overlaps %s", i.name);
    const BlockBwdP p{a->h, s, a->w_post, a->gate, a->w_pre, a->rstd_post, a->rstd_pre, g->dy, g->ds,
                      g->dh, g->dr, g->dgate, g->dw_post, g->dw_pre, M, N, gate_rows,
                      a->ldh, a->lds, a->ldg, g->lddy, g->ldds, g->lddh, g->lddr, g->lddg,
                      static_cast<float>(N), a->offset, a->alpha, a->beta, a->dtype,
                      static_cast<float*>(workspace)};
    return launched([&] { return block_bwd_run(p, c); });
}

// ---- rope ---------------------------------------------------------------------

namespace {

// Strides of a heads tensor: not negative, and the span within 2^48 bytes.
int check_heads(const char* name, const rmsnorm_heads_t& h, int64_t batch, int64_t seq, int64_t heads,
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

View heads_view(const rmsnorm_heads_t& h, int64_t batch, int64_t seq, int64_t heads, int64_t D, int64_t eb) {
    return View(h.ptr, D * eb)
        .dim(batch, h.batch_stride * eb)
        .dim(seq, h.token_stride * eb)
        .dim(heads, h.head_stride * eb);
}

HeadsP heads_p(const rmsnorm_heads_t& h) { return {h.ptr, h.batch_stride, h.token_stride, h.head_stride}; }

int rope_shapes(const rmsnorm_rope_args_t* a, bool fwd) {
    if (a == nullptr) return fail(RMSNORM_ERR_NULL, "args is NULL");
    if (a->struct_size != static_cast<int32_t>(sizeof(*a)) || a->reserved != 0)
        return fail(RMSNORM_ERR_OPTIONS, "args.struct_size is %d, expected %d (reserved 0)",
                    a->struct_size, static_cast<int>(sizeof(*a)));
    if (!dtype_ok(a->dtype)) return fail(RMSNORM_ERR_DTYPE, "dtype %d is not a rmsnorm_dtype_t", a->dtype);
    if (a->batch < 0 || a->seq < 0 || a->heads_q < 1 || a->heads_k < 0 || a->heads_q > (1 << 20) ||
        a->heads_k > (1 << 20) || a->head_dim < 2 || a->head_dim > 65536 || a->rotary_dim < 2 ||
        a->rotary_dim > a->head_dim || a->rotary_dim % 2 != 0)
        return fail(RMSNORM_ERR_SHAPE,
                    "need heads_q >= 1, heads_k >= 0 (at most 2^20), head_dim 2..65536 and an even "
                    "rotary_dim in 2..head_dim");
    if (a->batch > 0 && (a->batch > (int64_t(1) << 40) || a->seq > (int64_t(1) << 40) / a->batch))
        return fail(RMSNORM_ERR_SHAPE, "more than 2^40 tokens");
    if (a->interleaved != 0 && a->interleaved != 1)
        return fail(RMSNORM_ERR_OPTIONS, "interleaved is 0 or 1");
    if (!std::isfinite(a->offset) || !std::isfinite(a->magnitude))
        return fail(RMSNORM_ERR_SCALAR, "offset and magnitude must be finite");
    if (fwd && (!std::isfinite(a->eps) || a->eps < 0.f))
        return fail(RMSNORM_ERR_SCALAR, "eps must be finite and >= 0 (got %g)", a->eps);
    if (a->heads_k == 0 && (a->w_k || a->rstd_k))
        return fail(RMSNORM_ERR_NULL, "w_k and rstd_k are NULL without k");
    if (a->steps == nullptr) return fail(RMSNORM_ERR_NULL, "steps is NULL");
    if (misaligned(a->steps, 8) || misaligned(a->positions, 8))
        return fail(RMSNORM_ERR_ALIGN, "steps and positions must be 8-byte aligned");
    if (misaligned(a->rstd_q, 4) || misaligned(a->rstd_k, 4))
        return fail(RMSNORM_ERR_ALIGN, "rstd_q and rstd_k must be 4-byte aligned");
    const int64_t eb = elem_bytes(a->dtype);
    if (misaligned(a->w_q, eb) || misaligned(a->w_k, eb))
        return fail(RMSNORM_ERR_ALIGN, "w_q and w_k must be aligned to the element size");
    if (a->positions && (a->positions_stride < 0 || (a->positions_stride != 0 && a->positions_stride < a->seq) ||
                         (a->batch > 1 && a->positions_stride > kSpanLimit / 8 / (a->batch - 1))))
        return fail(RMSNORM_ERR_SHAPE, "positions_stride is 0 or at least seq");
    return RMSNORM_OK;
}

void rope_fill(const rmsnorm_rope_args_t* a, RopeP* p) {
    p->positions = a->positions;
    p->positions_stride = a->positions_stride;
    p->steps = a->steps;
    p->batch = a->batch;
    p->seq = a->seq;
    p->D = a->head_dim;
    p->R = a->rotary_dim;
    p->interleaved = a->interleaved;
    p->eps = a->eps;
    p->offset = a->offset;
    p->magnitude = a->magnitude;
    p->dtype = a->dtype;
    p->ws = nullptr;
    for (int k = 0; k < 2; ++k) {
        p->seg[k] = RopeSeg{};
        p->seg[k].heads = k == 0 ? a->heads_q : a->heads_k;
        p->seg[k].w = k == 0 ? a->w_q : a->w_k;
        p->seg[k].rstd = k == 0 ? a->rstd_q : a->rstd_k;
    }
}

}  // namespace

extern "C" int rmsnorm_rope_fwd(const rmsnorm_rope_args_t* a, const rmsnorm_options_t* opts, void* stream) {
    int rc = rope_shapes(a, true);
    if (rc != RMSNORM_OK) return rc;
    OpCfg c;
    rc = read_op_options(opts, &c);
    if (rc != RMSNORM_OK) return rc;
    const int64_t B = a->batch, S = a->seq, D = a->head_dim, eb = elem_bytes(a->dtype);
    if (B == 0 || S == 0) return RMSNORM_OK;
    const int Hq = a->heads_q, Hk = a->heads_k;
    if ((rc = check_heads("q", a->q, B, S, Hq, D, eb)) ||
        (rc = check_heads("out_q", a->out_q, B, S, Hq, D, eb)) ||
        (Hk && ((rc = check_heads("k", a->k, B, S, Hk, D, eb)) ||
                (rc = check_heads("out_k", a->out_k, B, S, Hk, D, eb)))))
        return rc;
    View qv = heads_view(a->q, B, S, Hq, D, eb), oq = heads_view(a->out_q, B, S, Hq, D, eb), kv, ok;
    if (Hk) kv = heads_view(a->k, B, S, Hk, D, eb), ok = heads_view(a->out_k, B, S, Hk, D, eb);
    const int64_t T = B * S;
    const Named outs[] = {{oq, "out_q", 1}, {ok, "out_k", 2},
                          {View(a->w_q ? a->rstd_q : nullptr, T * Hq * 4), "rstd_q", 0},
                          {View(a->w_k ? a->rstd_k : nullptr, T * Hk * 4), "rstd_k", 0}};
    const Named ins[] = {{qv, "q", 1}, {kv, "k", 2},
                         {View(a->w_q, D * eb), "w_q", 0}, {View(a->w_k, D * eb), "w_k", 0},
                         {View(a->positions, S * 8).dim(B, a->positions_stride * 8), "positions", 0},
                         {View(a->steps, a->rotary_dim / 2 * 8), "steps", 0}};
    rc = check_overlaps(outs, 4, ins, 6);
    if (rc != RMSNORM_OK) return rc;
    rc = finish_cfg(&c, stream);
    if (rc != RMSNORM_OK) return rc;
    RopeP p;
    rope_fill(a, &p);
    p.seg[0].in = heads_p(a->q);
    p.seg[0].out = heads_p(a->out_q);
    p.seg[1].in = heads_p(a->k);
    p.seg[1].out = heads_p(a->out_k);
    return launched([&] { return rope_fwd_run(p, c); });
}

extern "C" int rmsnorm_rope_bwd_workspace_size(int32_t head_dim, int64_t* bytes) {
    if (bytes == nullptr) return fail(RMSNORM_ERR_NULL, "bytes is NULL");
    *bytes = 0;
    if (head_dim < 2 || head_dim > 65536) return fail(RMSNORM_ERR_SHAPE, "head_dim is in 2..65536");
    DeviceInfo d;
    const cudaError_t e = device_info(&d);
    if (e != cudaSuccess) return fail(RMSNORM_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
    *bytes = rope_bwd_partial_rows(d.sm_count) * head_dim * 4;
    return RMSNORM_OK;
}

extern "C" int rmsnorm_rope_bwd(const rmsnorm_rope_args_t* a, const rmsnorm_rope_grads_t* g,
                                void* workspace, int64_t workspace_bytes,
                                const rmsnorm_options_t* opts, void* stream) {
    int rc = rope_shapes(a, false);
    if (rc != RMSNORM_OK) return rc;
    if (g == nullptr) return fail(RMSNORM_ERR_NULL, "grads is NULL");
    if (g->struct_size != static_cast<int32_t>(sizeof(*g)) || g->reserved != 0)
        return fail(RMSNORM_ERR_OPTIONS, "grads.struct_size is %d, expected %d (reserved 0)",
                    g->struct_size, static_cast<int>(sizeof(*g)));
    OpCfg c;
    rc = read_op_options(opts, &c);
    if (rc != RMSNORM_OK) return rc;
    const int64_t B = a->batch, S = a->seq, D = a->head_dim, eb = elem_bytes(a->dtype);
    const int Hq = a->heads_q, Hk = a->heads_k;
    if ((a->w_q != nullptr) != (g->dw_q != nullptr) || (a->w_k != nullptr) != (g->dw_k != nullptr))
        return fail(RMSNORM_ERR_NULL, "dw_q and dw_k are given exactly when w_q and w_k are");
    if (misaligned(g->dw_q, 4) || misaligned(g->dw_k, 4))
        return fail(RMSNORM_ERR_ALIGN, "dw_q and dw_k must be 4-byte aligned");
    const bool norm = a->w_q || a->w_k;
    if (B == 0 || S == 0) {
        rc = clear_floats(g->dw_q, D, stream);
        return rc == RMSNORM_OK ? clear_floats(g->dw_k, D, stream) : rc;
    }
    if ((rc = check_heads("dout_q", g->dout_q, B, S, Hq, D, eb)) ||
        (rc = check_heads("dq", g->dq, B, S, Hq, D, eb)) ||
        (a->w_q && (rc = check_heads("q", a->q, B, S, Hq, D, eb))) ||
        (Hk && ((rc = check_heads("dout_k", g->dout_k, B, S, Hk, D, eb)) ||
                (rc = check_heads("dk", g->dk, B, S, Hk, D, eb)))) ||
        (a->w_k && (rc = check_heads("k", a->k, B, S, Hk, D, eb))))
        return rc;
    if ((a->w_q && !a->rstd_q) || (a->w_k && !a->rstd_k))
        return fail(RMSNORM_ERR_NULL, "rstd_q and rstd_k must be given with w_q and w_k");
    if (norm && workspace == nullptr) return fail(RMSNORM_ERR_NULL, "the workspace is NULL");
    if (misaligned(workspace, 16)) return fail(RMSNORM_ERR_ALIGN, "the workspace must be 16-byte aligned");
    View kd, ok, xq, xk;
    if (Hk) kd = heads_view(g->dout_k, B, S, Hk, D, eb), ok = heads_view(g->dk, B, S, Hk, D, eb);
    if (a->w_q) xq = heads_view(a->q, B, S, Hq, D, eb);
    if (a->w_k) xk = heads_view(a->k, B, S, Hk, D, eb);
    const int64_t T = B * S;
    const Named outs[] = {{heads_view(g->dq, B, S, Hq, D, eb), "dq", 1}, {ok, "dk", 2},
                          {View(g->dw_q, D * 4), "dw_q", 0}, {View(g->dw_k, D * 4), "dw_k", 0}};
    const Named ins[] = {{heads_view(g->dout_q, B, S, Hq, D, eb), "dout_q", 1}, {kd, "dout_k", 2},
                         {xq, "q", 0}, {xk, "k", 0},
                         {View(a->w_q, D * eb), "w_q", 0}, {View(a->w_k, D * eb), "w_k", 0},
                         {View(a->w_q ? a->rstd_q : nullptr, T * Hq * 4), "rstd_q", 0},
                         {View(a->w_k ? a->rstd_k : nullptr, T * Hk * 4), "rstd_k", 0},
                         {View(a->positions, S * 8).dim(B, a->positions_stride * 8), "positions", 0},
                         {View(a->steps, a->rotary_dim / 2 * 8), "steps", 0}};
    rc = check_overlaps(outs, 4, ins, 10);
    if (rc != RMSNORM_OK) return rc;
    rc = finish_cfg(&c, stream);
    if (rc != RMSNORM_OK) return rc;
    if (norm) {
        const int64_t need = rope_bwd_partial_rows(c.dev.sm_count) * D * 4;
        if (workspace_bytes < need)
            return fail(RMSNORM_ERR_WORKSPACE, "workspace of %lld bytes, %lld needed",
                        static_cast<long long>(workspace_bytes), static_cast<long long>(need));
        const View ws(workspace, need);
        for (const Named& o : outs)
            if (meet(ws, o.v)) return fail(RMSNORM_ERR_OVERLAP, "the workspace overlaps %s", o.name);
        for (const Named& i : ins)
            if (meet(ws, i.v)) return fail(RMSNORM_ERR_OVERLAP, "the workspace overlaps %s", i.name);
    }
    RopeP p;
    rope_fill(a, &p);
    p.ws = static_cast<float*>(workspace);
    p.seg[0].in = heads_p(g->dout_q);
    p.seg[0].out = heads_p(g->dq);
    p.seg[0].x = heads_p(a->q);
    p.seg[0].dw = g->dw_q;
    p.seg[1].in = heads_p(g->dout_k);
    p.seg[1].out = heads_p(g->dk);
    p.seg[1].x = heads_p(a->k);
    p.seg[1].dw = g->dw_k;
    return launched([&] { return rope_bwd_run(p, c); });
}

extern "C" int rmsnorm_rope_steps(int32_t rotary_dim, double base, const rmsnorm_rope_scaling_t* sc,
                                  uint64_t* steps, float* magnitude) {
    if (steps == nullptr) return fail(RMSNORM_ERR_NULL, "steps is NULL");
    if (rotary_dim < 2 || rotary_dim > 65536 || rotary_dim % 2 != 0)
        return fail(RMSNORM_ERR_SHAPE, "rotary_dim is even and in 2..65536 (got %d)", rotary_dim);
    if (!std::isfinite(base) || base <= 1.0)
        return fail(RMSNORM_ERR_SCALAR, "base must be finite and above 1 (got %g)", base);
    int kind = RMSNORM_ROPE_PLAIN;
    if (sc != nullptr) {
        if (sc->struct_size != static_cast<int32_t>(sizeof(*sc)) || sc->kind < RMSNORM_ROPE_PLAIN ||
            sc->kind > RMSNORM_ROPE_BANDS)
            return fail(RMSNORM_ERR_OPTIONS, "scaling.struct_size or kind is not valid");
        kind = sc->kind;
        const bool ramp = kind == RMSNORM_ROPE_YARN || kind == RMSNORM_ROPE_BANDS;
        if (kind != RMSNORM_ROPE_PLAIN && !(std::isfinite(sc->factor) && sc->factor >= 1.0))
            return fail(RMSNORM_ERR_SCALAR, "scaling.factor must be finite and at least 1");
        if (ramp && !(std::isfinite(sc->length) && sc->length > 0.0 && std::isfinite(sc->beta_fast) &&
                      sc->beta_slow > 0.0 && sc->beta_fast > sc->beta_slow))
            return fail(RMSNORM_ERR_SCALAR, "scaling needs length > 0 and beta_fast > beta_slow > 0");
        if (kind == RMSNORM_ROPE_NTK && rotary_dim == 2)
            return fail(RMSNORM_ERR_SHAPE, "NTK scaling needs a rotary_dim above 2");
    }
    const double two_pi = 6.283185307179586476925286766559;
    const int half = rotary_dim / 2;
    const double R = rotary_dim;
    if (kind == RMSNORM_ROPE_NTK) {
        base *= std::pow(sc->factor, R / (R - 2.0));
        if (!std::isfinite(base)) return fail(RMSNORM_ERR_SCALAR, "the scaled base is not finite");
    }
    double lo = 0.0, hi = 0.0;
    if (kind == RMSNORM_ROPE_YARN) {
        // The pair index at which a frequency makes `turns` turns within `length`.
        auto index = [&](double turns) {
            return R * std::log(sc->length / (turns * two_pi)) / (2.0 * std::log(base));
        };
        lo = std::floor(index(sc->beta_fast));
        hi = std::ceil(index(sc->beta_slow));
        if (hi <= 0.0) {  // every pair is under beta_slow turns
            lo = -2.0;
            hi = -1.0;
        } else if (lo > R - 1.0) {  // every pair is above beta_fast turns
            hi = lo + 1.0;
        } else {
            lo = std::fmax(lo, 0.0);
            hi = std::fmin(hi, R - 1.0);
            if (hi == lo) hi += 0.001;
        }
    }
    for (int i = 0; i < half; ++i) {
        double f = std::pow(base, -2.0 * i / R);  // radians per position
        if (kind == RMSNORM_ROPE_LINEAR) {
            f /= sc->factor;
        } else if (kind == RMSNORM_ROPE_YARN) {
            const double t = std::fmin(std::fmax((i - lo) / (hi - lo), 0.0), 1.0);
            f = f / sc->factor * t + f * (1.0 - t);
        } else if (kind == RMSNORM_ROPE_BANDS) {
            const double turns = sc->length * f / two_pi;
            const double t = std::fmin(std::fmax((turns - sc->beta_slow) / (sc->beta_fast - sc->beta_slow), 0.0), 1.0);
            f = f / sc->factor * (1.0 - t) + f * t;
        }
        // At most 1/(2 pi) of a turn per position, so the product is below 2^62.
        steps[i] = static_cast<uint64_t>(std::ldexp(f / two_pi, 64) + 0.5);
    }
    if (magnitude)
        *magnitude = kind == RMSNORM_ROPE_YARN ? static_cast<float>(0.1 * std::log(sc->factor) + 1.0) : 1.f;
    return RMSNORM_OK;
}

// ---- cache --------------------------------------------------------------------

namespace {

int cache_shapes(const rmsnorm_cache_t* c, int dtype, CacheP* p) {
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

Named cache_array(const rmsnorm_cache_t* c, const CacheP& p, int which) {
    const int64_t heads = p.slots * p.heads;
    switch (which) {
        case 0: return {View(c->k_codes, heads * p.code_bytes), "k_codes", 0};
        case 1: return {View(c->k_scales, heads * p.groups), "k_scales", 0};
        case 2: return {View(c->v_codes, heads * p.code_bytes), "v_codes", 0};
        default: return {View(c->v_scales, heads * p.groups), "v_scales", 0};
    }
}

// k and v of a call: tokens of `heads` heads.
int cache_tensor(const char* name, const rmsnorm_heads_t* h, int64_t T, const CacheP& p, int k, CacheP* out,
                 View* v) {
    rmsnorm_heads_t x = *h;
    x.batch_stride = 0;
    const int64_t eb = elem_bytes(p.dtype);
    const int rc = check_heads(name, x, 1, T, p.heads, p.D, eb);
    if (rc != RMSNORM_OK) return rc;
    out->t[k] = heads_p(x);
    *v = heads_view(x, 1, T, p.heads, p.D, eb);
    return RMSNORM_OK;
}

}  // namespace

extern "C" int rmsnorm_cache_write(const rmsnorm_cache_t* cache, const rmsnorm_heads_t* k,
                                   const rmsnorm_heads_t* v, const int64_t* slots, int64_t T, int dtype,
                                   const rmsnorm_options_t* opts, void* stream) {
    CacheP p;
    int rc = cache_shapes(cache, dtype, &p);
    if (rc != RMSNORM_OK) return rc;
    OpCfg c;
    rc = read_op_options(opts, &c);
    if (rc != RMSNORM_OK) return rc;
    if (T < 0 || T > (int64_t(1) << 40)) return fail(RMSNORM_ERR_SHAPE, "T must be in 0..2^40");
    if (k == nullptr) return fail(RMSNORM_ERR_NULL, "k is NULL");
    if (v != nullptr && cache->v_codes == nullptr)
        return fail(RMSNORM_ERR_NULL, "v is given but the cache has no v_codes");
    if (T == 0) return RMSNORM_OK;
    if (slots == nullptr) return fail(RMSNORM_ERR_NULL, "slots is NULL");
    if (misaligned(slots, 8)) return fail(RMSNORM_ERR_ALIGN, "slots must be 8-byte aligned");
    View kv, vv;
    if ((rc = cache_tensor("k", k, T, p, 0, &p, &kv)) || (v && (rc = cache_tensor("v", v, T, p, 1, &p, &vv))))
        return rc;
    const Named outs[] = {cache_array(cache, p, 0), cache_array(cache, p, 1), cache_array(cache, p, 2),
                          cache_array(cache, p, 3)};
    const Named ins[] = {{kv, "k", 0}, {vv, "v", 0}, {View(slots, T * 8), "slots", 0}};
    rc = check_overlaps(outs, 4, ins, 3);
    if (rc != RMSNORM_OK) return rc;
    rc = finish_cfg(&c, stream);
    if (rc != RMSNORM_OK) return rc;
    p.codes[0] = cache->k_codes;
    p.scales[0] = cache->k_scales;
    p.codes[1] = v ? cache->v_codes : nullptr;
    p.scales[1] = v ? cache->v_scales : nullptr;
    p.slot = slots;
    p.T = T;
    return launched([&] { return cache_write_run(p, c); });
}

extern "C" int rmsnorm_cache_read(const rmsnorm_cache_t* cache, const int32_t* table, int64_t table_width,
                                  const int32_t* cu_rows, const int32_t* starts, int64_t sequences,
                                  int64_t rows, const rmsnorm_heads_t* k_out, const rmsnorm_heads_t* v_out,
                                  int dtype, const rmsnorm_options_t* opts, void* stream) {
    CacheP p;
    int rc = cache_shapes(cache, dtype, &p);
    if (rc != RMSNORM_OK) return rc;
    OpCfg c;
    rc = read_op_options(opts, &c);
    if (rc != RMSNORM_OK) return rc;
    if (rows < 0 || rows > (int64_t(1) << 31) || sequences < 0 || sequences > (int64_t(1) << 31) ||
        table_width < 0 || (sequences > 0 && table_width > (kSpanLimit / 4) / sequences))
        return fail(RMSNORM_ERR_SHAPE, "need 0 <= rows, sequences <= 2^31 and table_width >= 0");
    if (k_out == nullptr && v_out == nullptr) return fail(RMSNORM_ERR_NULL, "k_out and v_out are both NULL");
    if (v_out != nullptr && cache->v_codes == nullptr)
        return fail(RMSNORM_ERR_NULL, "v_out is given but the cache has no v_codes");
    if (rows == 0 || sequences == 0) return RMSNORM_OK;
    if (cu_rows == nullptr || (table == nullptr && table_width > 0))
        return fail(RMSNORM_ERR_NULL, "table and cu_rows must be non-NULL");
    if (misaligned(table, 4) || misaligned(cu_rows, 4) || misaligned(starts, 4))
        return fail(RMSNORM_ERR_ALIGN, "table, cu_rows and starts must be 4-byte aligned");
    View kv, vv;
    if ((k_out && (rc = cache_tensor("k_out", k_out, rows, p, 0, &p, &kv))) ||
        (v_out && (rc = cache_tensor("v_out", v_out, rows, p, 1, &p, &vv))))
        return rc;
    const Named outs[] = {{kv, "k_out", 0}, {vv, "v_out", 0}};
    const Named ins[] = {cache_array(cache, p, 0), cache_array(cache, p, 1), cache_array(cache, p, 2),
                         cache_array(cache, p, 3),
                         {View(table, sequences * table_width * 4), "table", 0},
                         {View(cu_rows, (sequences + 1) * 4), "cu_rows", 0},
                         {View(starts, sequences * 4), "starts", 0}};
    rc = check_overlaps(outs, 2, ins, 7);
    if (rc != RMSNORM_OK) return rc;
    rc = finish_cfg(&c, stream);
    if (rc != RMSNORM_OK) return rc;
    p.codes[0] = cache->k_codes;
    p.scales[0] = cache->k_scales;
    p.codes[1] = cache->v_codes;
    p.scales[1] = cache->v_scales;
    p.table = table;
    p.table_width = table_width;
    p.cu_rows = cu_rows;
    p.starts = starts;
    p.sequences = sequences;
    p.rows = rows;
    return launched([&] { return cache_read_run(p, c); });
}
