// Attention over the quantised cache: the element-wise kernel for any head size, and the
// choice of a kernel (the operation is stated in include/rmsnorm.h).
#include "rmsnorm.h"

#include "attn_common.cuh"
#include "attn_rows.h"
#include "row_ring_host.h"

#include <algorithm>
#include <mutex>
#include <set>
#include <utility>

namespace rmsn {

// Bit 0: a token's page was not there since the last read. One word per device.
__device__ unsigned int g_attn_status;
__device__ unsigned int g_attn_late;  // bit 0: a bounded wait ran out
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
        if (s.len > s.held && threadIdx.x == 0) atomicOr(p.status, 1u);
        for (int64_t t = see.low + w; t < see.high; t += 4) {
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

// Joins the parts of slots whose tiles more than one CTA took: blockIdx.x is the slot; `wpr` warps (8 or 1) a row of a head, which take turns at the parts.
__global__ void __launch_bounds__(256) attn_join_kernel(const AttnP p, const RowsPlan r, int wpr) {
    __shared__ __align__(16) float part[8][256 + 4];  // rows of whole vectors
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int R = 8 * r.nt, DP = r.gd * 32;
    pdl_wait();
    pdl_launch_dependents();
    const int4 slot = r.entries[blockIdx.x];
    const int u = static_cast<int>(blockIdx.y) * (8 / wpr) + (wpr == 8 ? 0 : w);
    const int hk = u / R, row = u - hk * R;  // R is 8, 16 or 32
    if (slot.x < 0 || row >= slot.w || hk >= p.heads) return;
    const int x = slot.x & 0xffff, n = (slot.x >> 16) - x + 1;
    auto at = [&](int k) {  // the k-th part
        const int64_t id = k == 0 ? 2 * x + 1 : 2 * (x + k);
        return (id * p.heads + hk) * R + row;
    };
    float M = -INFINITY;
    for (int k = lane; k < n; k += 32) M = fmaxf(M, r.ml[at(k)].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float L = 0.f;
    float4 o[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    const int first = wpr == 8 ? w : 0;
    for (int k0 = first; k0 < n; k0 += 4 * wpr) {
        float2 ml[4];
        float4 v[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = k0 + i * wpr;
            ml[i] = make_float2(-INFINITY, 0.f);
            v[i][0] = v[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k >= n) continue;
            const int64_t a = at(k);
            ml[i] = r.ml[a];
            if (lane * 4 < DP) v[i][0] = *reinterpret_cast<const float4*>(r.o + a * DP + lane * 4);
            if (128 + lane * 4 < DP) v[i][1] = *reinterpret_cast<const float4*>(r.o + a * DP + 128 + lane * 4);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float f = ml[i].x == -INFINITY ? 1.f : exp2f(ml[i].x - M);  // no token: zeros
            L += f * ml[i].y;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                o[c].x = fmaf(f, v[i][c].x, o[c].x), o[c].y = fmaf(f, v[i][c].y, o[c].y);
                o[c].z = fmaf(f, v[i][c].z, o[c].z), o[c].w = fmaf(f, v[i][c].w, o[c].w);
            }
        }
    }
    const int i = (slot.z + row) / p.G, qh = hk * p.G + slot.z + row - i * p.G;
    const int64_t out_row = slot.y + i;
    auto put = [&](int d, float v) {
        if (d >= p.D) return;
        const int64_t j = out_row * p.out.st + qh * p.out.sh + d;
        if (p.dtype == kBF16) store1<kBF16>(p.out.p, j, v);
        else if (p.dtype == kFP16) store1<kFP16>(p.out.p, j, v);
        else store1<kFP32>(p.out.p, j, v);
    };
    if (wpr == 8) {
#pragma unroll
        for (int c = 0; c < 2; ++c) *reinterpret_cast<float4*>(&part[w][c * 128 + lane * 4]) = o[c];
        if (lane == 0) part[w][256] = L;
        __syncthreads();
        L = 0.f;
        for (int k = 0; k < 8; ++k) L += part[k][256];
        float v = 0.f;
        for (int k = 0; k < 8; ++k) v += part[k][threadIdx.x];
        put(threadIdx.x, L == 0.f ? 0.f : v / L);
    } else {
        const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float v[4] = {o[c].x, o[c].y, o[c].z, o[c].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) put(c * 128 + lane * 4 + k, L == 0.f ? 0.f : v[k] * inv);
        }
    }
    if (p.lse && lane == 0 && (wpr == 1 || w == 0))
        p.lse[out_row * p.heads_q + qh] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// How the row kernels take a call; false where they cannot.
int divisor_up_to(int n, int most) {
    int d = n < most ? n : most;
    while (n % d) --d;
    return d;
}

// Rows of a key head in a CTA, eights of them. 32 rows take about 1.7 times 16 rows' time, so they are
// taken together where that leaves enough fewer CTAs; with more than 96 values a head they spill.
// (GB300, us, 32 / 16 rows a CTA, 32 sequences, contexts of 8192, 8 heads, bf16: 32 rows of a head of
// 64 values in 4 bits 111 / 125, of 128 values 224 / 196, in 8 bits 265 / 304; 40 rows 415 / 284, in
// 8 bits 455 / 444, fp32 604 / 361; 17 sequences of 40 rows of 64 values, a window of 400, 21.5 / 11.5)
int rows_nt(int64_t G, int64_t gd, int64_t sequences, int64_t rows) {
    // rows of a key head that a sequence has, on average
    const int64_t n = (rows + sequences - 1) / sequences * G;
    return n <= 8 ? 1 : gd <= 3 && (n + 31) / 32 * 7 <= (n + 15) / 16 * 4 ? 4 : 2;
}

int rows_gd(int64_t D) {
    const int64_t g = (D + 31) / 32;
    return g <= 2 ? 2 : g <= 4 ? static_cast<int>(g) : g <= 6 ? 6 : 8;
}

int64_t rows_slots(int64_t G, int nt, int64_t sequences, int64_t rows) { return rows * G / (8 * nt) + sequences; }

// At most this many CTAs for all head blocks together where slots are split.
int64_t rows_ctas(int nt, int gd, int pieces, int sm_count) {
    return static_cast<int64_t>(sm_count) * (gd * nt <= 4 && pieces == 1 ? 2 : 1);
}

// t / d = t * mul >> shift for 0 <= t < 2^31: with 2^l >= d > 2^(l - 1) and mul = floor(2^(31 + l) / d) + 1,
// t * mul is above t * 2^(31 + l) / d by at most t < 2^31 <= 2^(31 + l) / d.
void reciprocal(int64_t d, uint32_t* mul, int* shift) {
    int l = 0;
    while ((int64_t(1) << l) < d) ++l;
    *shift = 31 + l;
    *mul = static_cast<uint32_t>((uint64_t(1) << *shift) / static_cast<uint64_t>(d) + 1);
}

bool rows_plan(const AttnP& p, const OpCfg& c, RowsPlan* r) {
    *r = RowsPlan{};
    if (p.D > 256 || p.G > (1 << 20) || p.slots * p.heads >= 0xffffffffLL) return false;  // tokens of heads are counted in 32 bits
    r->pages = static_cast<uint32_t>(p.slots / p.page_size);
    reciprocal(p.page_size, &r->page_mul, &r->page_shift);
    reciprocal(p.G, &r->g_mul, &r->g_shift);
    r->most_tokens = static_cast<int>(std::min<int64_t>(p.width * p.page_size, INT32_MAX - 4096));
    r->window = static_cast<int>(std::min<int64_t>(p.window, INT32_MAX));
    const uintptr_t codes = reinterpret_cast<uintptr_t>(p.codes[0]) | reinterpret_cast<uintptr_t>(p.codes[1]);
    const uintptr_t scales = reinterpret_cast<uintptr_t>(p.scales[0]) | reinterpret_cast<uintptr_t>(p.scales[1]);
    r->gd = rows_gd(p.D);
    // (GB300, us, 32 sequences of 8192 tokens, 8 heads of 80 values in 8 bits, by 4 / 16 bytes 135 / 111;
    // 4 bits, 40 bytes a token: by 4 / 8 97 / 95, two chunks of 512 queries 345 / 374)
    const uintptr_t run = codes | static_cast<uintptr_t>(p.code_bytes);
    r->narrow = p.D == r->gd * 32 && codes % 16 == 0 ? 0 : run % 16 == 0 ? 16 : 4;
    if (r->narrow == 4 && run % 4 != 0) return false;
    const int pieces = p.dtype == kFP32 ? 2 : 1;
    r->nt = rows_nt(p.G, r->gd, p.sequences, p.rows);
    r->vec_scales = p.groups == r->gd && scales % 8 == 0 && p.slots * p.heads * p.groups % 4 == 0;
    const int64_t eb = elem_bytes(p.dtype), e = vec_elems(p.dtype);
    r->vec_q = aligned16(p.q.p) && (p.rows <= 1 || p.q.st % e == 0) && (p.heads_q <= 1 || p.q.sh % e == 0) && eb > 0;
    r->vec_out = aligned16(p.out.p) && (p.rows <= 1 || p.out.st % 2 == 0) && (p.heads_q <= 1 || p.out.sh % 2 == 0);
    // q's operands of a CTA's heads lie in shared memory where registers do not hold them
    const auto most_heads = [&] {
        const int q = r->nt == 1 && pieces == 1 ? 0 : pieces * 2 * r->gd * r->nt * 256;
        const int room = r->gd > 4 ? 32768 : 65536;
        return q ? std::max(1, std::min(8, room / q)) : 8;
    };
    r->hb = divisor_up_to(p.heads, most_heads());
    int64_t slots = rows_slots(p.G, r->nt, p.sequences, p.rows);
    if (p.rows * p.G >= (int64_t(1) << 30) || p.sequences >= (int64_t(1) << 30)) return false;  // counted in 32 bits
    r->slots = static_cast<int>(slots);
    // (the sum of all slots' tiles, of 16 tokens at least, is counted in 32 bits too)
    r->split = slots <= kSplitSlots && p.sequences <= kSplitSlots &&
               slots * (r->most_tokens / 16 + 8) < (int64_t(1) << 31);
    // Where a slot has few tokens whatever the lengths (by the table's width, or the window), a CTA
    // takes all of them, with its warps side by side, and nothing is left to join; fewer heads a
    // CTA where there would be fewer CTAs than two an SM (or than the call allows). (GB300, us, split and
    // joined / so: 4 sequences of up to 509 tokens, 8 heads 11.4 / 7.9; 17 of five queries in a window
    // of 1000, 5 heads of 96 values 23.6 / 14.8)
    const int64_t tile = (p.format == RMSNORM_CACHE_E2M1 && r->gd <= 4 ? 32 : 16) * 8;
    const int64_t rows_seen = r->window ? static_cast<int64_t>(r->window) + 8 * r->nt : INT32_MAX;
    if (std::min<int64_t>(r->most_tokens, rows_seen) <= 4 * tile + 64) {
        r->split = 0;
        // (8 rows a CTA where 16 would leave one CTA an SM: GB300, us, 8 / 16, sequences of five queries
        // in a window of 1000, 5 heads: 17 of 20 rows of 96 values 14.8 / 21.0; 17 of 40 rows of 128
        // values 27.8 / 29.4, 136 of them 139 / 173; 17 of 10 rows 17.2 / 15.1)
        if (pieces == 1 && (r->gd == 3 || r->gd == 4)) r->nt = 1;
        slots = rows_slots(p.G, r->nt, p.sequences, p.rows);
        r->slots = static_cast<int>(slots);
        r->hb = divisor_up_to(p.heads, most_heads());
        int hb = r->hb;
        const int64_t most = c.max_ctas > 0 ? c.max_ctas : INT32_MAX;
        while (hb > 1 && slots * (p.heads / hb) < std::min<int64_t>(2 * c.dev.sm_count, most)) {
            hb = divisor_up_to(p.heads, hb - 1);
            if (p.heads / hb > most) break;
            r->hb = hb;
        }
    }
    r->wph = 8 / r->hb;
    // (GB300, us, at 0 / 3 / 5: 32 sequences of up to 8192 tokens, 8 heads 49.2 / 45.9 / 48.0, two of
    // up to 131072, one head 53.1 / 46.6 / 45.3)
    r->start_tiles = r->wph == 1 ? 3 : 5;
    while (r->wph & (r->wph - 1)) --r->wph;  // a power of two
    r->head_blocks = p.heads / r->hb;
    int64_t ctas = rows_ctas(r->nt, r->gd, pieces, c.dev.sm_count);
    if (c.max_ctas > 0) ctas = std::min<int64_t>(ctas, c.max_ctas);
    ctas = std::min<int64_t>(ctas, 32767);  // a slot's first and last CTA share a word
    const int64_t whole = c.max_ctas > 0 ? c.max_ctas : 1 << 24;  // CTAs that take slots whole
    r->gx = static_cast<int>(std::max<int64_t>(1, r->split ? ctas / r->head_blocks
                                                          : std::min<int64_t>(slots, whole / r->head_blocks)));
    if (r->split) {
        const int64_t rows = 2LL * r->gx * p.heads * 8 * r->nt;
        unsigned char* at = static_cast<unsigned char*>(p.ws);
        r->o = reinterpret_cast<float*>(at);
        r->ml = reinterpret_cast<float2*>(at + rows * r->gd * 32 * 4);
        r->entries = reinterpret_cast<int4*>(at + rows * (r->gd * 32 * 4 + 8));
    }
    return true;
}

// The status words' addresses on the current device, for kernels of other files.
cudaError_t status_words(AttnP* p) {
    constexpr int kDevices = 64;
    static std::atomic<unsigned int*> known[kDevices][2];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kDevices && (p->status = known[dev][0].load()) && (p->late = known[dev][1].load())) return cudaSuccess;
    void *status = nullptr, *late = nullptr;
    if ((e = cudaGetSymbolAddress(&status, g_attn_status)) != cudaSuccess) return e;
    if ((e = cudaGetSymbolAddress(&late, g_attn_late)) != cudaSuccess) return e;
    p->status = static_cast<unsigned int*>(status);
    p->late = static_cast<unsigned int*>(late);
    if (dev < kDevices) known[dev][0].store(p->status), known[dev][1].store(p->late);
    return cudaSuccess;
}

// Whether the tensor cores take a call. A wave of their blocks (one an SM, of up to 256 rows) costs
// about as much as 6500 rows in the row kernels, which also split the tokens of few blocks.
// (GB300, us, tensor cores / row kernels, 8 heads of 128 values in 4 bits, bf16, contexts of 4096:
// 16 sequences of 64 rows 82 / 112, 64 of 32 rows 323 / 207, one of 512 rows 90 / 63, of 2048 90 / 190)
constexpr int64_t kRowsOfAWave = 6500;
bool tiles_ok(const AttnP& p, const RowsPlan& r, const OpCfg& c) {
    if (p.dtype == kFP32 || p.D % 32 != 0 || p.groups < 2 || p.groups > 4 || r.narrow || !r.vec_q) return false;
    const int64_t n = (p.rows + p.sequences - 1) / p.sequences * p.G;  // rows of a sequence, on average
    const int64_t blocks = ((n + 255) / 256 * p.sequences) * p.heads;
    const int64_t waves = (blocks + c.dev.sm_count - 1) / c.dev.sm_count;
    return p.rows * p.G * p.heads >= kRowsOfAWave * waves &&
           (p.rows * p.G / 256 + p.sequences) * p.heads < (int64_t(1) << 31);
}

}  // namespace

cudaError_t allow_smem(const void* kernel, int smem) {
    static std::mutex mu;
    static std::set<std::pair<int, const void*>> done;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> guard(mu);
    if (done.count({dev, kernel})) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) done.insert({dev, kernel});
    return e;
}

cudaError_t attn_join(const AttnP& p, const RowsPlan& r, const OpCfg& c) {
    // Parts a slot on average; many are joined by eight warps.
    const int wpr = r.gx / r.slots >= 12 ? 8 : 1;
    Launch l;
    l.grid = r.slots;
    l.threads = 256;
    LaunchCfg cfg(l, c.stream, c.pdl);
    cfg.cfg.gridDim.y = static_cast<unsigned>((static_cast<int64_t>(p.heads) * 8 * r.nt * wpr + 7) / 8);
    return cudaLaunchKernelEx(&cfg.cfg, attn_join_kernel, p, r, wpr);
}

// For any type, format and alignment of such a call.
int64_t attn_ws_bytes(int64_t heads, int64_t G, int64_t D, int64_t sequences, int64_t rows, int sm_count) {
    if (D > 256 || sequences == 0 || rows == 0) return 16;
    const int gd = rows_gd(D), nt = rows_nt(G, gd, sequences, rows);
    const int64_t slots = rows_slots(G, nt, sequences, rows);
    if (slots > kSplitSlots || sequences > kSplitSlots) return 16;
    // gx * head_blocks CTAs of hb heads: the heads in all CTAs are at most 8 a CTA, or all of them once
    const int64_t parts = std::max<int64_t>(rows_ctas(nt, gd, 1, sm_count) * std::min<int64_t>(heads, 8), heads);
    return 2 * parts * 8 * nt * (gd * 32 * 4 + 8) + slots * 16;
}

cudaError_t attn_run(const AttnP& given, const OpCfg& c) {
    AttnP p = given;
    const cudaError_t e = status_words(&p);
    if (e != cudaSuccess) return e;
    g_launched.store(true);
    RowsPlan r;
    if (c.variant != RMSNORM_VARIANT_GENERIC && rows_plan(p, c, &r)) {
        if (tiles_ok(p, r, c)) return attn_tiles(p, r, c);
        const bool e4 = p.format == RMSNORM_CACHE_E4M3, wide = p.dtype == kFP32;
        const cudaError_t ran = e4 ? (wide ? attn_rows_e4m3_fp32(p, r, c) : attn_rows_e4m3(p, r, c))
                                   : (wide ? attn_rows_e2m1_fp32(p, r, c) : attn_rows_e2m1(p, r, c));
        return ran != cudaSuccess || !r.split || r.gx == 1 ? ran : attn_join(p, r, c);
    }
    if (c.variant == RMSNORM_VARIANT_CTA) return cudaErrorNotSupported;
    return p.format == RMSNORM_CACHE_E4M3 ? run_generic<RMSNORM_CACHE_E4M3>(p, c)
                                          : run_generic<RMSNORM_CACHE_E2M1>(p, c);
}

cudaError_t attn_late_read_and_clear(unsigned int* value) {
    return symbol_read_and_clear(g_attn_late, g_launched, value);
}

cudaError_t attn_status_read_and_clear(unsigned int* value) {
    return symbol_read_and_clear(g_attn_status, g_launched, value);
}

}  // namespace rmsn
