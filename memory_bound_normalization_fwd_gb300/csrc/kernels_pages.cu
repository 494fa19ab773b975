// Pages of the cache copied, forked, freed and compacted (the operations are stated in
// include/rmsnorm.h).
//
// What is moved is whole pages of the cache's four arrays: one read and one write of
// every byte, bound by HBM. What is planned is small, and has to be the same whatever the
// order in which threads run: free pages are named by rank (the i-th free page), which a
// scan gives, not by a counter that threads race for. (GB300: 6000 pages of 17 KB copied in
// 33.5 us, 89% of the rate of a copy; 16384 pages of 34 KB, 5500 of them live, compacted in 46.5, 79%,
// of which live_kernel and the start of the moves are about 5; 56 rows freed and forked in 10.5,
// three launches' latency. One CTA seeks the free pages of a fork, so a large pool whose free pages lie at its
// end takes longer: 64 children, forked and freed, 4096 pages 9.8, 65536 23.5, 262144 67, 1048576 238.)
#include "rmsnorm.h"

#include "ops.h"
#include "ops_common.cuh"
#include "row_ring_host.h"

#include <algorithm>

namespace rmsn {

// Bit 0: an index was out of range, or a sequence could not be forked, since the last
// read. One word per device.
__device__ unsigned int g_pages_status;
static std::atomic<bool> g_launched{false};  // a kernel that writes it

namespace {

__device__ __forceinline__ void report() { atomicOr(&g_pages_status, 1u); }

// n bytes by `lanes` threads (this one is `lane`), in the widest accesses that both
// addresses and n allow.
__device__ __forceinline__ void copy_bytes(uint8_t* to, const uint8_t* from, int64_t n, int lane, int lanes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(to) | reinterpret_cast<uintptr_t>(from) | static_cast<uintptr_t>(n);
    if ((a & 15) == 0) {
        for (int64_t i = lane; i < n / 16; i += lanes)
            st_stream(reinterpret_cast<uint4*>(to) + i, ld_stream(reinterpret_cast<const uint4*>(from) + i));
    } else if ((a & 3) == 0) {
        for (int64_t i = lane; i < n / 4; i += lanes)
            reinterpret_cast<uint32_t*>(to)[i] = reinterpret_cast<const uint32_t*>(from)[i];
    } else {
        for (int64_t i = lane; i < n; i += lanes) to[i] = from[i];
    }
}

// A page. Vectors of the four arrays are numbered through, `FLY` of a thread in flight.
template <int FLY>
__device__ __forceinline__ void copy_page(const PageBytes& b, int64_t from, int64_t to, int lane, int lanes) {
    if (!b.vectors) {
#pragma unroll
        for (int a = 0; a < 4; ++a)
            if (b.p[a]) copy_bytes(b.p[a] + to * b.page[a], b.p[a] + from * b.page[a], b.page[a], lane, lanes);
        return;
    }
    const int e0 = static_cast<int>(b.page[0] / 16), e1 = e0 + static_cast<int>(b.page[1] / 16);
    const int e2 = e1 + static_cast<int>(b.page[2] / 16), e3 = e2 + static_cast<int>(b.page[3] / 16);
    for (int i0 = lane; i0 < e3; i0 += lanes * FLY) {
        uint4 v[FLY];
        uint8_t* base[FLY];
        int64_t size[FLY];
        int at[FLY];
#pragma unroll
        for (int k = 0; k < FLY; ++k) {
            const int i = i0 + k * lanes;
            const int a = (i >= e0) + (i >= e1) + (i >= e2);
            base[k] = i < e3 ? (a == 0 ? b.p[0] : a == 1 ? b.p[1] : a == 2 ? b.p[2] : b.p[3]) : nullptr;
            size[k] = a == 0 ? b.page[0] : a == 1 ? b.page[1] : a == 2 ? b.page[2] : b.page[3];
            at[k] = i - (a == 0 ? 0 : a == 1 ? e0 : a == 2 ? e1 : e2);
            if (base[k]) v[k] = ld_stream(reinterpret_cast<const uint4*>(base[k] + from * size[k]) + at[k]);
        }
#pragma unroll
        for (int k = 0; k < FLY; ++k)
            if (base[k]) st_stream(reinterpret_cast<uint4*>(base[k] + to * size[k]) + at[k], v[k]);
    }
}

// ---- copy ------------------------------------------------------------------------

// A team of `team` threads (a warp or the CTA) takes a page. One page a team: CTAs that come
// free take the next ones (6000 pages of 17 KB, us: 1216 CTAs of as many pages each 36.4, so 33.8).
__global__ void __launch_bounds__(256) copy_pages_kernel(const PagesP p, int team) {
    pdl_wait();
    pdl_launch_dependents();
    const int per = 256 / team, lane = threadIdx.x & (team - 1);
    const int64_t step = static_cast<int64_t>(gridDim.x) * per;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * per + threadIdx.x / team; i < p.n; i += step) {
        const int32_t from = __ldg(p.a + i), to = __ldg(p.b + i);
        if (from < 0 || to < 0) continue;
        if (from >= p.pages || to >= p.pages) {
            if (lane == 0) report();
            continue;
        }
        copy_page<5>(p.bytes, from, to, lane, team);
    }
}

// ---- free ------------------------------------------------------------------------

// A CTA a row. An entry is taken by an exchange, so that a row named twice loses its
// references once.
__global__ void __launch_bounds__(128) free_kernel(const PagesP p) {
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t i = blockIdx.x; i < p.n; i += gridDim.x) {
        const int64_t row = __ldg(p.a + i);
        if (row < 0) continue;
        if (row >= p.sequences) {
            if (threadIdx.x == 0) report();
            continue;
        }
        int32_t* entries = p.table + row * p.width;
        for (int64_t j = threadIdx.x; j < p.width; j += 128) {
            if (entries[j] == -1) continue;
            const int32_t page = atomicExch(entries + j, -1);
            if (page < 0) continue;
            if (page >= p.pages) {
                report();
            } else if (atomicSub(p.refs + page, 1) <= 0) {
                atomicAdd(p.refs + page, 1);
                report();
            }
        }
        if (threadIdx.x == 0) p.lengths[row] = 0;
    }
}

// ---- fork ------------------------------------------------------------------------

// The plan of a fork: tokens of each child (-1: nothing is done), the free page that takes its
// last ones (-1: none), and which fork claims a row.
struct ForkPlan {
    int32_t* have;   // [n]
    int32_t* fresh;  // [n]
    int32_t* claim;  // [sequences]
};

__host__ __device__ inline ForkPlan fork_plan(void* ws, int64_t n) {
    int32_t* w = static_cast<int32_t*>(ws);
    return {w, w + n, w + 2 * n};
}

// Exclusive sum of v over the CTA's 1024 threads, in order; the total in `total`.
__device__ __forceinline__ int cta_scan(int v, int* sums, int& total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int t = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, t, off);
        if (lane >= off) t += o;
    }
    if (lane == 31) sums[w] = t;
    __syncthreads();
    int s = sums[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += o;
    }
    total = __shfl_sync(0xffffffffu, s, 31);
    const int before = w ? __shfl_sync(0xffffffffu, s, w - 1) : 0;
    __syncthreads();  // sums is free again
    return before + t - v;
}

// One CTA: it is a few thousand numbers, and what it waits for is latency. Free pages are
// sought 4096 at a time from the lowest on, until there are enough.
__global__ void __launch_bounds__(1024) fork_plan_kernel(const PagesP p) {
    __shared__ int sums[32];
    const ForkPlan f = fork_plan(p.ws, p.n);
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    auto in_table = [&](int64_t row) { return row >= 0 && row < p.sequences; };
    for (int64_t i = tid; i < p.n; i += 1024)
        if (in_table(p.b[i])) f.claim[p.b[i]] = INT32_MAX;
    __syncthreads();
    for (int64_t i = tid; i < p.n; i += 1024)
        if (in_table(p.b[i]) && p.a[i] >= 0) atomicMin(f.claim + p.b[i], static_cast<int32_t>(i));
    __syncthreads();
    int need = 0;  // free pages taken so far
    for (int64_t i0 = 0; i0 < p.n; i0 += 1024) {
        const int64_t i = i0 + tid;
        int have = -1;
        if (i < p.n && p.a[i] >= 0 && p.b[i] >= 0) {
            const int64_t parent = p.a[i], child = p.b[i];
            bool ok = in_table(parent) && in_table(child) && parent != child;
            ok = ok && p.lengths[child] == 0 && atomicAdd(f.claim + child, 0) == i;
            if (ok) {
                have = p.lengths[parent];
                const int64_t used = (static_cast<int64_t>(have) + p.bytes.page_size - 1) / p.bytes.page_size;
                ok = have >= 0 && used <= p.width;
            }
            if (!ok) {
                report();
                have = -1;
            }
        }
        const int mine = have > 0 && have % p.bytes.page_size != 0 ? 1 : 0;
        int total;
        const int rank = cta_scan(mine, sums, total);
        if (i < p.n) {
            f.have[i] = have;
            f.fresh[i] = mine ? need + rank : -1;  // its rank, until the pages are known
        }
        need += total;
    }
    // The free pages by rank.
    __syncthreads();
    int found = 0;
    for (int64_t q0 = 0; q0 < p.pages && found < need; q0 += 4096) {
        const int64_t q = q0 + 4 * tid;
        int r[4], mine = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            r[k] = q + k < p.pages ? p.refs[q + k] : 1;
            mine += r[k] <= 0;
        }
        int total;
        int rank = found + cta_scan(mine, sums, total);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (r[k] > 0) continue;
            if (rank < need) f.claim[p.sequences + rank] = static_cast<int32_t>(q + k);
            ++rank;
        }
        found += total;
    }
    __syncthreads();
    for (int64_t i = tid; i < p.n; i += 1024) {
        const int rank = f.fresh[i];
        if (rank < 0) continue;
        if (rank < found) {
            f.fresh[i] = f.claim[p.sequences + rank];
        } else {  // no free page left
            report();
            f.have[i] = -1;
        }
    }
}

// A CTA a child: its row, the references, and the tokens of the last page.
__global__ void __launch_bounds__(256) fork_kernel(const PagesP p) {
    const ForkPlan f = fork_plan(p.ws, p.n);
    const PageBytes& b = p.bytes;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t i = blockIdx.x; i < p.n; i += gridDim.x) {
        const int have = f.have[i];
        if (have < 0) continue;
        const int full = have / b.page_size, rest = have - full * b.page_size;
        const int32_t fresh = f.fresh[i];
        const int32_t* from = p.table + static_cast<int64_t>(p.a[i]) * p.width;
        int32_t* to = p.table + static_cast<int64_t>(p.b[i]) * p.width;
        for (int64_t j = threadIdx.x; j < p.width; j += 256) {
            int32_t page = -1;
            if (j < full) {
                page = from[j];
                if (page >= 0 && page < p.pages) atomicAdd(p.refs + page, 1);
                else report();
            } else if (j == full && rest) {
                page = from[j];
                if (page >= 0 && page < p.pages) {
                    page = fresh;
                    p.refs[page] = 1;
                } else {  // stays what it is; the page set aside for it stays free
                    report();
                }
            }
            to[j] = page;
        }
        if (threadIdx.x == 0) p.lengths[p.b[i]] = have;
        if (!rest) continue;
        const int32_t old = from[full];
        if (old < 0 || old >= p.pages) continue;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            if (!b.p[a]) continue;
            const int64_t run = b.token[a] * b.page_size;
            if (b.runs == 1) {
                copy_bytes(b.p[a] + fresh * b.page[a], b.p[a] + old * b.page[a], b.token[a] * rest, threadIdx.x, 256);
            } else {  // a warp a head
                for (int h = threadIdx.x >> 5; h < b.runs; h += 8)
                    copy_bytes(b.p[a] + fresh * b.page[a] + h * run, b.p[a] + old * b.page[a] + h * run,
                               b.token[a] * rest, threadIdx.x & 31, 32);
            }
        }
    }
}

// ---- compact ----------------------------------------------------------------------

// Which pages are live: a bit a page in words of 32, with the live pages of the same 1024
// before each word, and the live pages of each 1024 pages.
struct LiveMap {
    uint2* words;     // (mask, live pages before it in its thousand)
    int32_t* counts;  // of each 1024 pages
};

__host__ __device__ inline LiveMap live_map(void* ws, int64_t pages) {
    const int64_t blocks = (pages + 1023) / 1024;
    return {static_cast<uint2*>(ws), reinterpret_cast<int32_t*>(static_cast<uint2*>(ws) + blocks * 32)};
}

__global__ void __launch_bounds__(1024) live_kernel(const PagesP p) {
    __shared__ int sums[32];
    const LiveMap m = live_map(p.ws, p.pages);
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t b = blockIdx.x; b * 1024 < p.pages; b += gridDim.x) {
        const int64_t q = b * 1024 + threadIdx.x;
        const uint32_t mask = __ballot_sync(0xffffffffu, q < p.pages && p.refs[q] > 0);
        if (lane == 0) sums[w] = __popc(mask);
        __syncthreads();
        int t = sums[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, t, off);
            if (lane >= off) t += o;
        }
        if (lane == w) m.words[b * 32 + w] = make_uint2(mask, t - __popc(mask));
        if (threadIdx.x == 31) m.counts[b] = t;
        __syncthreads();  // sums is free again
    }
}

// The k-th set bit of a word that has more than k.
__device__ __forceinline__ int bit_at(uint32_t mask, int k) {
    int at = 0;
#pragma unroll
    for (int half = 16; half > 0; half >>= 1) {
        const int low = __popc(mask & ((1u << half) - 1u));
        if (k >= low) {
            k -= low;
            at += half;
            mask >>= half;
        }
    }
    return at;
}

// Ranks and selections among the live pages. before[b]: live pages before the b-th 1024
// (in shared memory).
struct Ranks {
    const uint2* words;  // in shared memory where they fit
    const int32_t* before;
    int blocks;
    __device__ __forceinline__ int64_t live_before(int64_t page) const {
        const uint2 w = words[page >> 5];
        return before[page >> 10] + static_cast<int>(w.y) + __popc(w.x & ((1u << (page & 31)) - 1u));
    }
    // The k-th live (or free) page; there are more than k.
    template <bool LIVE>
    __device__ __forceinline__ int64_t select(int64_t k) const {
        auto at_block = [&](int b) -> int64_t { return LIVE ? before[b] : b * int64_t(1024) - before[b]; };
        int lo = 0, hi = blocks - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (at_block(mid) <= k) lo = mid;
            else hi = mid - 1;
        }
        const int r = static_cast<int>(k - at_block(lo));
        const uint2* w = words + lo * int64_t(32);
        auto at_word = [&](int i) {
            const int v = static_cast<int>(w[i].y);
            return LIVE ? v : i * 32 - v;
        };
        int a = 0;
#pragma unroll
        for (int half = 16; half > 0; half >>= 1)
            if (at_word(a + half) <= r) a += half;
        const uint32_t mask = w[a].x;
        return lo * int64_t(1024) + a * 32 + bit_at(LIVE ? mask : ~mask, r - at_word(a));
    }
};

// Moves, the counts and the table. With L live pages, `stay` of them below L: the i-th
// move takes the (stay + i)-th live page to the i-th free one.
__global__ void __launch_bounds__(256) compact_kernel(const PagesP p, int team, int move_ctas, int staged) {
    extern __shared__ __align__(16) int32_t before[];  // [blocks + 1], behind it the words
    __shared__ int warp_sums[8];
    const LiveMap m = live_map(p.ws, p.pages);
    const int blocks = static_cast<int>((p.pages + 1023) / 1024), tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    // exclusive sums of the counts, a run of consecutive ones a thread
    const int run = (blocks + 255) / 256;
    int own = 0;
    for (int i = tid * run; i < min(blocks, tid * run + run); ++i) own += m.counts[i];
    int t = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, t, off);
        if ((tid & 31) >= off) t += o;
    }
    if ((tid & 31) == 31) warp_sums[tid >> 5] = t;
    __syncthreads();
    int sum = t - own;
    for (int w = 0; w < tid >> 5; ++w) sum += warp_sums[w];
    for (int i = tid * run; i < min(blocks, tid * run + run); ++i) {
        before[i] = sum;
        sum += m.counts[i];
    }
    int all = 0;
    for (int w = 0; w < 8; ++w) all += warp_sums[w];
    uint2* words = reinterpret_cast<uint2*>(before + (blocks + 4) / 4 * 4);
    if (staged)
        for (int i = tid; i < blocks * 32; i += 256) words[i] = m.words[i];
    __syncthreads();
    const int64_t L = all;
    const Ranks r{staged ? words : m.words, before, blocks};
    const int64_t stay = L < p.pages ? r.live_before(L) : L, moves = L - stay;
    if (static_cast<int>(blockIdx.x) < move_ctas) {
        // The CTA's next 256 moves are found by a thread each (by all threads for each one,
        // the searches took longer than the copies).
        __shared__ int64_t from[256], to[256];
        const int per = 256 / team, lane = tid & (team - 1);
        for (int64_t i0 = blockIdx.x; i0 < moves; i0 += static_cast<int64_t>(move_ctas) * 256) {
            const int64_t i = i0 + static_cast<int64_t>(tid) * move_ctas;
            __syncthreads();
            if (i < moves) {
                from[tid] = r.select<true>(stay + i);
                to[tid] = r.select<false>(i);
            }
            __syncthreads();
            for (int k = tid / team; k < 256 && i0 + static_cast<int64_t>(k) * move_ctas < moves; k += per)
                copy_page<4>(p.bytes, from[k], to[k], lane, team);
        }
        if (static_cast<int>(gridDim.x) > move_ctas) return;
    }
    // counts and table: by the CTAs behind, or by a single one too
    const int before_rest = static_cast<int>(gridDim.x) > move_ctas ? move_ctas : 0;
    const int64_t first = static_cast<int64_t>(blockIdx.x - before_rest) * 256 + tid;
    const int64_t step = static_cast<int64_t>(gridDim.x - before_rest) * 256;
    if (first == 0) *p.live = static_cast<int32_t>(L);
    // a move's two counts, by one thread; the others stay as they are
    for (int64_t i = first; i < moves; i += step) {
        const int64_t from = r.select<true>(stay + i), to = r.select<false>(i);
        const int32_t v = p.refs[from];
        p.refs_out[to] = v;
        p.refs_out[from] = 0;
    }
    if (p.refs_out != p.refs) {
        for (int64_t q = first; q < p.pages; q += step) {
            const bool is_live = (r.words[q >> 5].x >> (q & 31)) & 1u;
            if (is_live ? q < L : q >= L) p.refs_out[q] = p.refs[q];
        }
    }
    const int64_t entries = p.sequences * p.width;
    for (int64_t e = first; e < entries; e += step) {
        int32_t page = p.table[e];
        if (page >= p.pages) {
            report();
        } else if (page >= L && ((r.words[page >> 5].x >> (page & 31)) & 1u)) {
            page = static_cast<int32_t>(r.select<false>(r.live_before(page) - stay));
        }
        p.table_out[e] = page;
    }
}

int64_t page_bytes(const PageBytes& b) { return b.page[0] + b.page[1] + b.page[2] + b.page[3]; }

// Threads a page: a CTA where they have a vector each.
int team_of(const PageBytes& b) { return page_bytes(b) >= 256 * 16 ? 256 : 32; }

}  // namespace

int64_t pages_ws_bytes(int64_t pages, int64_t sequences, int64_t n) {
    const int64_t blocks = (pages + 1023) / 1024;
    const int64_t fork = (2 * n + sequences + n) * 4, compact = blocks * 32 * 8 + blocks * 4;
    return (std::max(fork, compact) + 15) / 16 * 16;
}

cudaError_t pages_copy_run(const PagesP& p, const OpCfg& c) {
    g_launched.store(true);
    const int team = team_of(p.bytes);
    int64_t G = std::min<int64_t>((p.n + 256 / team - 1) / (256 / team), 1 << 24);
    if (c.max_ctas > 0) G = std::min<int64_t>(G, c.max_ctas);
    return op_launch(c, copy_pages_kernel, G, 256, 0, p, team);
}

cudaError_t pages_free_run(const PagesP& p, const OpCfg& c) {
    g_launched.store(true);
    return op_launch(c, free_kernel, persistent_grid(p.n, 1, c.dev.sm_count, 16, c.max_ctas), 128, 0, p);
}

cudaError_t pages_fork_run(const PagesP& p, const OpCfg& c) {
    g_launched.store(true);
    const cudaError_t e = op_launch(c, fork_plan_kernel, 1, 1024, 0, p);
    if (e != cudaSuccess) return e;
    return op_launch(c, fork_kernel, persistent_grid(p.n, 1, c.dev.sm_count, 8, c.max_ctas), 256, 0, p);
}

cudaError_t pages_compact_run(const PagesP& p, const OpCfg& c) {
    g_launched.store(true);
    const int64_t blocks = (p.pages + 1023) / 1024;
    cudaError_t e = op_launch(c, live_kernel, persistent_grid(blocks, 1, c.dev.sm_count, 2, c.max_ctas), 1024, 0, p);
    if (e != cudaSuccess) return e;
    const int team = team_of(p.bytes);
    // Up to 128 thousand pages: the words are searched in shared memory.
    const int staged = blocks <= 128 ? 1 : 0;
    const int smem = staged ? static_cast<int>((blocks + 4) / 4 * 4) * 4 + static_cast<int>(blocks) * 32 * 8
                            : static_cast<int>(blocks + 1) * 4;
    if (!staged) {  // always to the most, so that no call lowers it for another
        e = cudaFuncSetAttribute(compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kMaxPages / 1024 + 1) * 4);
        if (e != cudaSuccess) return e;
    }
    // At most half of the pages can move; some CTAs beside take counts and table.
    int64_t move = persistent_grid((p.pages + 1) / 2, 256 / team, c.dev.sm_count, 7, c.max_ctas);
    const int64_t small = std::max(p.pages, p.sequences * p.width);
    int64_t rest = persistent_grid(small, 256, c.dev.sm_count, 1, 0);
    if (c.max_ctas > 0) {  // both together
        rest = std::min<int64_t>(rest, c.max_ctas == 1 ? 0 : std::max(1, c.max_ctas / 8));
        move = std::min<int64_t>(move, c.max_ctas - rest);
    }
    return op_launch(c, compact_kernel, move + rest, 256, smem, p, team, static_cast<int>(move), staged);
}

cudaError_t pages_status_read_and_clear(unsigned int* value) {
    return symbol_read_and_clear(g_pages_status, g_launched, value);
}

}  // namespace rmsn
