// C ABI front end of the operators that serve from the cache: attention over it, and its
// pages copied, forked, freed and compacted. Argument validation on the host before any
// CUDA call, then the launch. The operations are stated in include/rmsnorm.h.
#include "rmsnorm.h"

#include "op_checks.h"

namespace rmsn {
namespace {

constexpr int kMaxHeadDim = 512;  // of attention

// ---- pages ----------------------------------------------------------------------

void page_layout(const rmsnorm_cache_t* c, const CacheP& k, PageBytes* b) {
    uint8_t* arrays[4] = {c->k_codes, c->v_codes, c->k_scales, c->v_scales};
    b->runs = c->heads_first ? c->heads : 1;
    b->page_size = c->page_size;
    b->vectors = true;
    for (int a = 0; a < 4; ++a) {
        const int64_t head = a < 2 ? k.code_bytes : k.groups;
        b->p[a] = arrays[a];
        b->page[a] = arrays[a] ? head * c->heads * c->page_size : 0;
        b->token[a] = c->heads_first ? head : head * c->heads;
        if (b->page[a] % 16 != 0 || !aligned16(arrays[a]) || b->page[a] > (int64_t(1) << 32)) b->vectors = false;
    }
}

// The cache of a call that moves its pages.
int cache_pages(const rmsnorm_cache_t* c, CacheP* k, PagesP* p) {
    const int rc = cache_shapes(c, RMSNORM_DTYPE_BF16, k);
    if (rc != RMSNORM_OK) return rc;
    page_layout(c, *k, &p->bytes);
    p->pages = c->pages;
    return RMSNORM_OK;
}

int pages_struct(const rmsnorm_cache_pages_t* g, bool lengths, PagesP* p) {
    if (g == nullptr) return fail(RMSNORM_ERR_NULL, "pages is NULL");
    if (g->struct_size != static_cast<int32_t>(sizeof(*g)) || g->reserved != 0)
        return fail(RMSNORM_ERR_OPTIONS, "pages.struct_size is %d, expected %d (reserved 0)", g->struct_size,
                    static_cast<int>(sizeof(*g)));
    if (g->pages < 1 || g->pages > kMaxPages)
        return fail(RMSNORM_ERR_SHAPE, "pages must be in 1..2^25 (got %lld)", static_cast<long long>(g->pages));
    if (g->sequences < 0 || g->sequences > (int64_t(1) << 30) || g->table_width < 0 ||
        g->table_width > (int64_t(1) << 30))
        return fail(RMSNORM_ERR_SHAPE, "sequences and table_width must be in 0..2^30");
    const bool some = g->sequences > 0;
    if (!g->refs || (!g->table && some && g->table_width > 0) || (!g->lengths && some && lengths))
        return fail(RMSNORM_ERR_NULL, "refs, table and lengths must be non-NULL");
    if (misaligned(g->refs, 4) || misaligned(g->table, 4) || misaligned(g->lengths, 4))
        return fail(RMSNORM_ERR_ALIGN, "refs, table and lengths must be 4-byte aligned");
    p->pages = g->pages;
    p->sequences = g->sequences;
    p->width = g->table_width;
    p->refs = g->refs;
    p->table = g->table;
    p->lengths = g->lengths;
    return RMSNORM_OK;
}

// Lists of n indices.
int lists(const char* names, const int32_t* a, const int32_t* b, bool two, int64_t n) {
    if (n < 0 || n > (int64_t(1) << 30)) return fail(RMSNORM_ERR_SHAPE, "n must be in 0..2^30");
    if (n > 0 && (a == nullptr || (two && b == nullptr))) return fail(RMSNORM_ERR_NULL, "%s must be non-NULL", names);
    if (misaligned(a, 4) || misaligned(b, 4)) return fail(RMSNORM_ERR_ALIGN, "%s must be 4-byte aligned", names);
    return RMSNORM_OK;
}

Named refs_of(const rmsnorm_cache_pages_t* g, int mark) { return {View(g->refs, g->pages * 4), "refs", mark}; }
Named table_of(const rmsnorm_cache_pages_t* g, int mark) {
    return {View(g->table, g->sequences * g->table_width * 4), "table", mark};
}
Named lengths_of(const rmsnorm_cache_pages_t* g) { return {View(g->lengths, g->sequences * 4), "lengths", 0}; }

int check_workspace(const void* ws, int64_t have, int64_t need, const Named* arrays, int n) {
    if (need > 0 && ws == nullptr) return fail(RMSNORM_ERR_NULL, "the workspace is NULL");
    if (misaligned(ws, 16)) return fail(RMSNORM_ERR_ALIGN, "the workspace must be 16-byte aligned");
    if (have < need)
        return fail(RMSNORM_ERR_WORKSPACE, "workspace of %lld bytes, %lld needed", static_cast<long long>(have),
                    static_cast<long long>(need));
    const View w(ws, need);
    for (int i = 0; i < n; ++i)
        if (meet(w, arrays[i].v)) return fail(RMSNORM_ERR_OVERLAP, "the workspace overlaps %s", arrays[i].name);
    return RMSNORM_OK;
}

}  // namespace
}  // namespace rmsn

using namespace rmsn;

extern "C" int rmsnorm_cache_copy_pages(const rmsnorm_cache_t* cache, const int32_t* src, const int32_t* dst,
                                        int64_t n, const rmsnorm_options_t* opts, void* stream) {
    CacheP k;
    PagesP p{};
    int rc = cache_pages(cache, &k, &p);
    if (rc != RMSNORM_OK) return rc;
    OpCfg c;
    rc = read_op_options(opts, &c);
    if (rc != RMSNORM_OK) return rc;
    rc = lists("src and dst", src, dst, true, n);
    if (rc != RMSNORM_OK || n == 0) return rc;
    const Named outs[] = {cache_array(cache, k, 0), cache_array(cache, k, 1), cache_array(cache, k, 2),
                          cache_array(cache, k, 3)};
    const Named ins[] = {{View(src, n * 4), "src", 0}, {View(dst, n * 4), "dst", 0}};
    rc = check_overlaps(outs, 4, ins, 2);
    if (rc != RMSNORM_OK) return rc;
    rc = finish_cfg(&c, stream);
    if (rc != RMSNORM_OK) return rc;
    p.n = n;
    p.a = src;
    p.b = dst;
    return launched([&] { return pages_copy_run(p, c); });
}

extern "C" int rmsnorm_cache_pages_workspace_size(int64_t pages, int64_t sequences, int64_t n, int64_t* bytes) {
    if (bytes == nullptr) return fail(RMSNORM_ERR_NULL, "bytes is NULL");
    *bytes = 0;
    if (pages < 1 || pages > kMaxPages || sequences < 0 || sequences > (int64_t(1) << 30) || n < 0 ||
        n > (int64_t(1) << 30))
        return fail(RMSNORM_ERR_SHAPE, "need pages in 1..2^25, sequences and n in 0..2^30");
    *bytes = pages_ws_bytes(pages, sequences, n);
    return RMSNORM_OK;
}

extern "C" int rmsnorm_cache_fork(const rmsnorm_cache_t* cache, const rmsnorm_cache_pages_t* pages,
                                  const int32_t* parents, const int32_t* children, int64_t n, void* workspace,
                                  int64_t workspace_bytes, const rmsnorm_options_t* opts, void* stream) {
    CacheP k;
    PagesP p{};
    int rc = cache_pages(cache, &k, &p);
    if (rc != RMSNORM_OK || (rc = pages_struct(pages, true, &p)) != RMSNORM_OK) return rc;
    if (pages->pages != cache->pages)
        return fail(RMSNORM_ERR_SHAPE, "pages.pages is %lld, the cache has %lld", static_cast<long long>(pages->pages),
                    static_cast<long long>(cache->pages));
    OpCfg c;
    rc = read_op_options(opts, &c);
    if (rc != RMSNORM_OK) return rc;
    rc = lists("parents and children", parents, children, true, n);
    if (rc != RMSNORM_OK || n == 0) return rc;
    const Named outs[] = {cache_array(cache, k, 0), cache_array(cache, k, 1), cache_array(cache, k, 2),
                          cache_array(cache, k, 3), refs_of(pages, 0), table_of(pages, 0), lengths_of(pages)};
    const Named ins[] = {{View(parents, n * 4), "parents", 0}, {View(children, n * 4), "children", 0}};
    rc = check_overlaps(outs, 7, ins, 2);
    if (rc != RMSNORM_OK) return rc;
    const int64_t need = pages_ws_bytes(p.pages, p.sequences, n);
    if ((rc = check_workspace(workspace, workspace_bytes, need, outs, 7)) ||
        (rc = check_workspace(workspace, workspace_bytes, need, ins, 2)))
        return rc;
    rc = finish_cfg(&c, stream);
    if (rc != RMSNORM_OK) return rc;
    p.n = n;
    p.a = parents;
    p.b = children;
    p.ws = workspace;
    return launched([&] { return pages_fork_run(p, c); });
}

extern "C" int rmsnorm_cache_free(const rmsnorm_cache_pages_t* pages, const int32_t* rows, int64_t n,
                                  const rmsnorm_options_t* opts, void* stream) {
    PagesP p{};
    int rc = pages_struct(pages, true, &p);
    if (rc != RMSNORM_OK) return rc;
    OpCfg c;
    rc = read_op_options(opts, &c);
    if (rc != RMSNORM_OK) return rc;
    rc = lists("rows", rows, nullptr, false, n);
    if (rc != RMSNORM_OK || n == 0) return rc;
    const Named outs[] = {refs_of(pages, 0), table_of(pages, 0), lengths_of(pages)};
    const Named ins[] = {{View(rows, n * 4), "rows", 0}};
    rc = check_overlaps(outs, 3, ins, 1);
    if (rc != RMSNORM_OK) return rc;
    rc = finish_cfg(&c, stream);
    if (rc != RMSNORM_OK) return rc;
    p.n = n;
    p.a = rows;
    return launched([&] { return pages_free_run(p, c); });
}

extern "C" int rmsnorm_cache_compact(const rmsnorm_cache_t* cache, const rmsnorm_cache_pages_t* pages,
                                     int32_t* refs_out, int32_t* table_out, int32_t* live, void* workspace,
                                     int64_t workspace_bytes, const rmsnorm_options_t* opts, void* stream) {
    CacheP k;
    PagesP p{};
    int rc = cache_pages(cache, &k, &p);
    if (rc != RMSNORM_OK || (rc = pages_struct(pages, false, &p)) != RMSNORM_OK) return rc;
    if (pages->pages != cache->pages)
        return fail(RMSNORM_ERR_SHAPE, "pages.pages is %lld, the cache has %lld", static_cast<long long>(pages->pages),
                    static_cast<long long>(cache->pages));
    OpCfg c;
    rc = read_op_options(opts, &c);
    if (rc != RMSNORM_OK) return rc;
    const int64_t entries = p.sequences * p.width;
    if (!refs_out || !live || (!table_out && entries > 0))
        return fail(RMSNORM_ERR_NULL, "refs_out, table_out and live must be non-NULL");
    if (misaligned(refs_out, 4) || misaligned(table_out, 4) || misaligned(live, 4))
        return fail(RMSNORM_ERR_ALIGN, "refs_out, table_out and live must be 4-byte aligned");
    const Named outs[] = {cache_array(cache, k, 0), cache_array(cache, k, 1), cache_array(cache, k, 2),
                          cache_array(cache, k, 3), {View(refs_out, p.pages * 4), "refs_out", 1},
                          {View(table_out, entries * 4), "table_out", 2}, {View(live, 4), "live", 0}};
    const Named ins[] = {refs_of(pages, 1), table_of(pages, 2)};
    rc = check_overlaps(outs, 7, ins, 2);
    if (rc != RMSNORM_OK) return rc;
    const int64_t need = pages_ws_bytes(p.pages, 0, 0);
    if ((rc = check_workspace(workspace, workspace_bytes, need, outs, 7)) ||
        (rc = check_workspace(workspace, workspace_bytes, need, ins, 2)))
        return rc;
    rc = finish_cfg(&c, stream);
    if (rc != RMSNORM_OK) return rc;
    p.refs_out = refs_out;
    p.table_out = table_out;
    p.live = live;
    p.ws = workspace;
    return launched([&] { return pages_compact_run(p, c); });
}

// ---- attention ------------------------------------------------------------------

namespace {

int attention_sizes(int64_t heads, int64_t heads_q, int64_t D, int64_t sequences, int64_t rows) {
    if (heads < 1 || heads > (1 << 20) || heads_q < 1 || heads_q > (1 << 20) || heads_q % heads != 0)
        return fail(RMSNORM_ERR_SHAPE, "heads_q (%lld) must be a multiple of the cache's heads (%lld)",
                    static_cast<long long>(heads_q), static_cast<long long>(heads));
    if (D < 1 || D > kMaxHeadDim) return fail(RMSNORM_ERR_SHAPE, "head_dim must be in 1..%d for attention", kMaxHeadDim);
    if (sequences < 0 || sequences > (int64_t(1) << 30) || rows < 0 || rows > (int64_t(1) << 30) ||
        rows * heads_q > (int64_t(1) << 40))
        return fail(RMSNORM_ERR_SHAPE, "sequences and rows must be in 0..2^30 (2^40 rows of heads)");
    return RMSNORM_OK;
}

}  // namespace

extern "C" int rmsnorm_cache_attention_workspace_size(int32_t cache_heads, int32_t heads_q, int32_t head_dim,
                                                      int64_t sequences, int64_t rows, int64_t* bytes) {
    if (bytes == nullptr) return fail(RMSNORM_ERR_NULL, "bytes is NULL");
    *bytes = 0;
    const int rc = attention_sizes(cache_heads, heads_q, head_dim, sequences, rows);
    if (rc != RMSNORM_OK) return rc;
    DeviceInfo d;
    const cudaError_t e = device_info(&d);
    if (e != cudaSuccess) return fail(RMSNORM_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
    *bytes = attn_ws_bytes(cache_heads, heads_q / cache_heads, head_dim, sequences, rows, d.sm_count);
    return RMSNORM_OK;
}

extern "C" int rmsnorm_cache_attention(const rmsnorm_cache_t* cache, const rmsnorm_cache_attention_args_t* a,
                                       void* workspace, int64_t workspace_bytes, const rmsnorm_options_t* opts,
                                       void* stream) {
    if (a == nullptr) return fail(RMSNORM_ERR_NULL, "args is NULL");
    if (a->struct_size != static_cast<int32_t>(sizeof(*a)) || a->reserved != 0.f)
        return fail(RMSNORM_ERR_OPTIONS, "args.struct_size is %d, expected %d (reserved 0)", a->struct_size,
                    static_cast<int>(sizeof(*a)));
    CacheP k;
    int rc = cache_shapes(cache, a->dtype, &k);
    if (rc != RMSNORM_OK) return rc;
    if (cache->v_codes == nullptr) return fail(RMSNORM_ERR_NULL, "attention needs a cache that holds v");
    rc = attention_sizes(cache->heads, a->heads_q, cache->head_dim, a->sequences, a->rows);
    if (rc != RMSNORM_OK) return rc;
    OpCfg c;
    rc = read_op_options(opts, &c);
    if (rc != RMSNORM_OK) return rc;
    if (a->causal != 0 && a->causal != 1) return fail(RMSNORM_ERR_OPTIONS, "causal is 0 or 1");
    if (a->window < 0 || (a->window > 0 && !a->causal))
        return fail(RMSNORM_ERR_SHAPE, "window is >= 0, and needs causal");
    if (!std::isfinite(a->scale)) return fail(RMSNORM_ERR_SCALAR, "scale must be finite");
    if (a->table_width < 0 || a->table_width > (int64_t(1) << 30) ||
        (a->sequences > 0 && a->table_width > (kSpanLimit / 4) / a->sequences))
        return fail(RMSNORM_ERR_SHAPE, "table_width must be in 0..2^30");
    if (a->cu_rows == nullptr && a->rows != a->sequences)
        return fail(RMSNORM_ERR_SHAPE, "without cu_rows there is one row a sequence (%lld rows, %lld sequences)",
                    static_cast<long long>(a->rows), static_cast<long long>(a->sequences));
    if (a->rows == 0 || a->sequences == 0) return RMSNORM_OK;
    if (a->lengths == nullptr || (a->table == nullptr && a->table_width > 0))
        return fail(RMSNORM_ERR_NULL, "table and lengths must be non-NULL");
    if (misaligned(a->table, 4) || misaligned(a->lengths, 4) || misaligned(a->cu_rows, 4) || misaligned(a->lse, 4))
        return fail(RMSNORM_ERR_ALIGN, "table, lengths, cu_rows and lse must be 4-byte aligned");
    const int64_t eb = elem_bytes(a->dtype), D = cache->head_dim, H = a->heads_q;
    rmsnorm_heads_t q = a->q, o = a->out;
    q.batch_stride = o.batch_stride = 0;
    if ((rc = check_heads("q", q, 1, a->rows, H, D, eb)) || (rc = check_heads("out", o, 1, a->rows, H, D, eb)))
        return rc;
    const Named outs[] = {{heads_view(o, 1, a->rows, H, D, eb), "out", 0}, {View(a->lse, a->rows * H * 4), "lse", 0}};
    const Named ins[] = {{heads_view(q, 1, a->rows, H, D, eb), "q", 0},
                         cache_array(cache, k, 0), cache_array(cache, k, 1), cache_array(cache, k, 2),
                         cache_array(cache, k, 3),
                         {View(a->table, a->sequences * a->table_width * 4), "table", 0},
                         {View(a->lengths, a->sequences * 4), "lengths", 0},
                         {View(a->cu_rows, (a->sequences + 1) * 4), "cu_rows", 0}};
    rc = check_overlaps(outs, 2, ins, 8);
    if (rc != RMSNORM_OK) return rc;
    rc = finish_cfg(&c, stream);
    if (rc != RMSNORM_OK) return rc;
    const int64_t G = H / cache->heads;
    const int64_t need = attn_ws_bytes(cache->heads, G, D, a->sequences, a->rows, c.dev.sm_count);
    if ((rc = check_workspace(workspace, workspace_bytes, need, outs, 2)) ||
        (rc = check_workspace(workspace, workspace_bytes, need, ins, 8)))
        return rc;
    AttnP p{};
    p.format = cache->format;
    p.slots = k.slots;
    p.page_size = cache->page_size;
    p.heads = cache->heads;
    p.D = cache->head_dim;
    p.code_bytes = k.code_bytes;
    p.groups = k.groups;
    p.heads_first = cache->heads_first;
    p.codes[0] = cache->k_codes;
    p.codes[1] = cache->v_codes;
    p.scales[0] = cache->k_scales;
    p.scales[1] = cache->v_scales;
    p.q = heads_p(q);
    p.out = heads_p(o);
    p.dtype = a->dtype;
    p.heads_q = a->heads_q;
    p.G = static_cast<int>(G);
    p.causal = a->causal;
    p.window = a->window;
    p.sequences = a->sequences;
    p.rows = a->rows;
    p.width = a->table_width;
    p.table = a->table;
    p.lengths = a->lengths;
    p.cu = a->cu_rows;
    p.lse = a->lse;
    p.scale = a->scale;
    p.ws = workspace;
    return launched([&] { return attn_run(p, c); });
}
