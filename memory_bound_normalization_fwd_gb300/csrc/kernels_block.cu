// The norm after a block, its gate, the scaled residual and the norm before
// the next block (the operation is stated in include/rmsnorm.h).
//
// Both norms need a whole row's sum before the row can go on, and the second
// sum is over what the first norm makes: two row reductions in sequence, with
// 2 reads and 2 writes of a row around them. The bound is HBM: 4 M N elements.
#include "rmsnorm.h"

#include "ops.h"
#include "ops_common.cuh"
#include "row_ring.cuh"
#include "row_ring_host.h"

#include <algorithm>

namespace rmsn {

// Bit 0: a bounded wait ran out since the last read. One word per device.
__device__ unsigned int g_block_status;
static std::atomic<bool> g_launched{false};  // a kernel that writes it

namespace {

// Vector kernel: row teams with a ring of h and r rows (and gate rows, where
// each row has its own) in shared memory. A thread keeps its columns of the row
// in registers between the reductions: h is read once, s once made.
// GATE: 0 none, 1 one gate row for several rows (kept in registers, read again
// where the gate row changes), 2 a gate row per row (staged like h and r).
// FULL: both norms are there and a row is exactly V vectors of every thread, which
// the compiler then knows: no test of either is left in the loop.
template <int DT, int V, int GATE, int MAXT, bool FULL>
__global__ void __launch_bounds__(MAXT) block_fwd_ring_kernel(const BlockP p, const RingShape g) {
    constexpr int E = VecElems<DT>::value;
    const bool post = FULL || p.w_post, pre = FULL || p.w_pre;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ RingShared sh;
    __shared__ __align__(16) float parts[kMaxTeams][2][kMaxTeamWarps];

    const int team = threadIdx.x / g.T, t = threadIdx.x - team * g.T;
    const int64_t me = static_cast<int64_t>(blockIdx.x) * g.teams + team;
    const int64_t r0 = me * g.q + (me < g.rem ? me : g.rem);
    const int rows = static_cast<int>(g.q) + (me < g.rem ? 1 : 0);
    Ring ring;
    ring.row_bytes = static_cast<uint32_t>(g.nvec) * 16u;
    ring.stage_bytes = ring.row_bytes * g.arrays;
    ring.base = smem_u32(smem) + static_cast<uint32_t>(team * g.stages) * ring.stage_bytes;
    ring.bars = smem_u32(&sh.bars[team][0]);
    if (t == 0) {
        for (int st = 0; st < g.stages; ++st) mbar_init(ring.bar(st), 1);
        fence_mbar_init();
        sh.give_up[team].clear();
    }
    for (int i = t; i < 2 * kMaxTeamWarps; i += g.T) parts[team][0][i] = 0.f;

    const uint4* h = static_cast<const uint4*>(p.h) + r0 * p.ldh;
    const uint4* r = static_cast<const uint4*>(p.r) + r0 * p.ldr;
    const uint4* gate = static_cast<const uint4*>(p.gate);
    uint4* s = static_cast<uint4*>(p.s) + r0 * p.lds + t;
    uint4* y = static_cast<uint4*>(p.y) + r0 * p.ldy + t;
    auto issue = [&](int row, int st) {
        ring.expect(st);
        ring.copy(st, 0, h + row * p.ldh);
        ring.copy(st, 1, r + row * p.ldr);
        if (GATE == 2) ring.copy(st, 2, gate + (r0 + row) * p.ldg);
    };
    pdl_wait();
    if (t == 0) {
        for (int k = 0; k < g.stages && k < rows; ++k) issue(k, k);
    }
    // Per column, as pairs: alpha (offset + w_post), times the gate where it stands
    // for several rows, and offset + w_pre.
    constexpr int H = E / 2;
    const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
    f2 scale[V][H], wpre[V][H];
    int64_t grow = 0;
    int64_t left = 0;  // rows until the gate row changes
    if (GATE == 1) {
        grow = r0 / p.gate_rows;
        left = (grow + 1) * p.gate_rows - r0;
    }
    auto load_scale = [&]() {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = v * g.T + t;
            const bool in = c < g.nvec;
            if (p.w_post) {
                weights2<DT>(in ? __ldg(static_cast<const uint4*>(p.w_post) + c) : zero4, p.offset, scale[v]);
#pragma unroll
                for (int e = 0; e < H; ++e) scale[v][e] = f2_mul(scale[v][e], f2_dup(p.alpha));
            } else {
#pragma unroll
                for (int e = 0; e < H; ++e) scale[v][e] = f2_dup(p.alpha);
            }
            if (GATE == 1) {
                f2 x[H];
                unpack2<DT>(in ? __ldg(gate + grow * p.ldg + c) : zero4, x);
#pragma unroll
                for (int e = 0; e < H; ++e) scale[v][e] = f2_mul(scale[v][e], x[e]);
            }
        }
    };
    load_scale();
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = v * g.T + t;
        weights2<DT>(p.w_pre && c < g.nvec ? __ldg(static_cast<const uint4*>(p.w_pre) + c) : zero4, p.offset,
                     wpre[v]);
    }
    __syncthreads();  // barriers and flags are set up
    pdl_launch_dependents();

    int st = 0, parity = 0;
    uint32_t phase = 0;
    bool dead = false;
    int row = 0;
    const f2 beta = f2_dup(p.beta);
    // Vectors of the row; those past its end stay zero.
    uint4 hv[V], rv[V], gv[V];
#pragma unroll
    for (int v = 0; v < V; ++v) hv[v] = rv[v] = gv[v] = zero4;
    for (; row < rows; ++row, s += p.lds, y += p.ldy) {
        if (GATE == 1) {
            if (left == 0) {
                ++grow;
                left = p.gate_rows;
                load_scale();
            }
            --left;
        }
        if (!mbar_wait_bounded(ring.bar(st), phase, g.limit)) sh.give_up[team].mark(row);
        f2 f[V][H];
        f2 sq = 0;
        const unsigned char* at = smem + (ring.stage(st) - smem_u32(smem)) + 16u * t;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (FULL || v * g.T + t < g.nvec) {
                const unsigned char* q = at + 16u * (v * g.T);
                hv[v] = *reinterpret_cast<const uint4*>(q);
                rv[v] = *reinterpret_cast<const uint4*>(q + ring.row_bytes);
                if (GATE == 2) gv[v] = *reinterpret_cast<const uint4*>(q + 2 * ring.row_bytes);
            }
            unpack2<DT>(hv[v], f[v]);
            if (post) {
#pragma unroll
                for (int e = 0; e < H; ++e) sq = f2_fma(f[v][e], f[v][e], sq);
            }
        }
        // Behind a row's first barrier every thread has read the stage: the
        // leader refills it.
        auto behind_first_barrier = [&]() {
            dead = sh.give_up[team].at(row);
            if (!dead && t == 0 && row + g.stages < rows) issue(row + g.stages, st);
        };
        float a = 1.f;
        if (post) {
            const float ss = team_sum(f2_sum(sq), &parts[team][parity][0], team, t, g.T);
            parity ^= 1;
            behind_first_barrier();
            if (dead) break;
            a = row_rstd(ss, p.n, p.eps);
            if (t == 0 && p.rstd_post) p.rstd_post[r0 + row] = a;
        }
        sq = 0;
        const f2 a2 = f2_dup(a);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            f2 x[H], q[H];
            if (GATE == 2) unpack2<DT>(gv[v], q);
            unpack2<DT>(rv[v], x);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                // the same bits whether the gate is a row's own or stands for several
                const f2 k = GATE == 2 ? f2_mul(scale[v][e], q[e]) : scale[v][e];
                f[v][e] = f2_fma(f2_mul(f[v][e], a2), k, f2_mul(beta, x[e]));
                sq = f2_fma(f[v][e], f[v][e], sq);
            }
        }
        float ss = f2_sum(sq);
        if (!post) {  // then w_pre is given
            ss = team_sum(ss, &parts[team][parity][0], team, t, g.T);
            parity ^= 1;
            behind_first_barrier();
            if (dead) break;
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (FULL || v * g.T + t < g.nvec) st_stream(s + v * g.T, pack2<DT>(f[v]));
        if (pre) {
            if (post) {
                ss = team_sum(ss, &parts[team][parity][0], team, t, g.T);
                parity ^= 1;
            }
            const float b = row_rstd(ss, p.n, p.eps);
            if (t == 0 && p.rstd_pre) p.rstd_pre[r0 + row] = b;
            const f2 b2 = f2_dup(b);
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int e = 0; e < H; ++e) f[v][e] = f2_mul(f2_mul(f[v][e], b2), wpre[v][e]);
                if (FULL || v * g.T + t < g.nvec) st_stream(y + v * g.T, pack2<DT>(f[v]));
            }
        }
        if (++st == g.stages) {
            st = 0;
            phase ^= 1;
        }
    }
    if (dead && t == 0) {
        atomicOr(&g_block_status, 1u);
        // Rows below row + stages were issued and may still be landing.
        for (int k = row; k < row + g.stages && k < rows; ++k) {
            mbar_wait_bounded(ring.bar(st), phase, g.drain);
            if (++st == g.stages) {
                st = 0;
                phase ^= 1;
            }
        }
    }
}

template <int DT, int GATE>
cudaError_t launch_ring(BlockP p, const OpCfg& c, bool* taken) {
    constexpr int E = VecElems<DT>::value;
    using Fn = void (*)(const BlockP, const RingShape);
    const int64_t nvec = p.N / E;
    RingPlan plan;
    *taken = false;
    // One vector per thread up to 256 threads, then two, then four.
    const int V = nvec <= 256 ? 1 : nvec <= 1024 ? 2 : nvec <= 2048 ? 4 : 0;
    if (V == 0) return cudaSuccess;
    const int T = static_cast<int>((nvec + V * 32 - 1) / (V * 32)) * 32;
    const bool wide = T > 256;
    const bool full = p.w_post && p.w_pre && nvec == static_cast<int64_t>(V) * T;
    Fn fn = nullptr;
    if (full)
        fn = V == 1   ? block_fwd_ring_kernel<DT, 1, GATE, 256, true>
             : V == 2 ? (wide ? block_fwd_ring_kernel<DT, 2, GATE, 512, true>
                              : block_fwd_ring_kernel<DT, 2, GATE, 256, true>)
                      : block_fwd_ring_kernel<DT, 4, GATE, 512, true>;
    else
        fn = V == 1   ? block_fwd_ring_kernel<DT, 1, GATE, 256, false>
             : V == 2 ? (wide ? block_fwd_ring_kernel<DT, 2, GATE, 512, false>
                              : block_fwd_ring_kernel<DT, 2, GATE, 256, false>)
                      : block_fwd_ring_kernel<DT, 4, GATE, 512, false>;
    // 64 KB of stages per SM carry the reads; more make reads and writes fight
    // (GB300, us: 16384x4096 bf16 at 64 / 96 / 128 / 192 KB 86 / 97 / 97 / 97,
    // 16384x8192 164 / 178 / 184 / 184, 65536x512 at 48 / 72 / 96 KB 52 / 46 / 46).
    if (!ring_plan(reinterpret_cast<const void*>(fn), c, p.M, static_cast<int>(nvec), T, wide ? 512 : 256,
                   GATE == 2 ? 3 : 2, 0, 64 << 10, 1, INT64_MAX, &plan))
        return cudaSuccess;
    p.ldh /= E;
    p.ldr /= E;
    p.ldg /= E;
    p.lds /= E;
    p.ldy /= E;
    *taken = true;
    return op_launch(c, fn, plan.grid, plan.threads, plan.smem, p, plan.shape);
}

// Whole vectors everywhere: rows, strides and addresses.
bool vectors(const BlockP& p) {
    const int64_t e = vec_elems(p.dtype);
    const void* ptrs[] = {p.h, p.r, p.w_post, p.gate, p.w_pre, p.s, p.y};
    for (const void* q : ptrs)
        if (!aligned16(q)) return false;
    const int64_t sizes[] = {p.N, p.ldh, p.ldr, p.lds, p.gate ? p.ldg : 0, p.y ? p.ldy : 0};
    for (int64_t n : sizes)
        if (n % e != 0) return false;
    return true;
}

// Element-wise kernel for rows that no other takes: one CTA per row, three
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

// Rows that are not whole vectors (any N, stride and alignment), of up to 512 V
// columns: a CTA per row, element loads, a thread's columns t, t + T, ... kept in
// registers between the reductions, so that h and r are read once. The scales stay in
// registers, the next row (and its gate row, where one gate does not stand for all
// rows) is loaded while this one is reduced, and a load is one instruction (GB300,
// us, against the kernel below: 18503x708 bf16 60 -> 44, 23493x987 fp32 92 -> 72,
// 16384x777 bf16 with a gate row per 100 rows 74 -> 57).
template <int DT, int V>
__global__ void __launch_bounds__(512) block_fwd_columns_kernel(const BlockP p) {
    using Raw = typename Elem<DT>::T;
    __shared__ __align__(16) float part[2][kMaxTeamWarps];
    int parity = 0;
    const int t = threadIdx.x, T = blockDim.x, N = static_cast<int>(p.N);
    const bool row_gate = p.gate && p.gate_rows < p.M;
    Raw rh[V], rr[V], rg[V];
    // Byte offsets of the thread's columns (past the row's end: of the last one): a
    // row's base is the same for all threads.
    uint32_t off[V];
    bool in[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        in[v] = v * T + t < N;
        off[v] = static_cast<uint32_t>(min(v * T + t, N - 1)) * static_cast<uint32_t>(sizeof(Raw));
    }
    auto load_raw = [&](const void* x, int64_t base, Raw (&out)[V]) {
        const char* q = static_cast<const char*>(x) + base * static_cast<int64_t>(sizeof(Raw));
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] = *reinterpret_cast<const Raw*>(q + off[v]);
    };
    auto store = [&](void* x, int64_t base, int v, float f) {
        char* q = static_cast<char*>(x) + base * static_cast<int64_t>(sizeof(Raw));
        *reinterpret_cast<Raw*>(q + off[v]) = Elem<DT>::store(f);
    };
    auto fetch = [&](int64_t row) {
        load_raw(p.h, row * p.ldh, rh);
        load_raw(p.r, row * p.ldr, rr);
        if (row_gate) load_raw(p.gate, row / p.gate_rows * p.ldg, rg);
    };
    for (int i = t; i < 2 * kMaxTeamWarps; i += T) (&part[0][0])[i] = 0.f;
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    fetch(blockIdx.x);
    float scale[V], wpre[V];  // alpha (offset + w_post), times a gate for all rows
    if (p.w_post) load_columns<DT, V>(p.w_post, 0, t, T, N, scale);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        scale[v] = p.w_post ? p.alpha * (p.offset + scale[v]) : p.alpha;
        wpre[v] = 0.f;
    }
    if (p.gate && !row_gate) {
        float q[V];
        load_columns<DT, V>(p.gate, 0, t, T, N, q);
#pragma unroll
        for (int v = 0; v < V; ++v) scale[v] *= q[v];
    }
    if (p.w_pre) {
        load_columns<DT, V>(p.w_pre, 0, t, T, N, wpre);
#pragma unroll
        for (int v = 0; v < V; ++v) wpre[v] += p.offset;
    }
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        float f[V], r[V], k[V], ss = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            f[v] = in[v] ? Elem<DT>::load(rh[v]) : 0.f;
            r[v] = in[v] ? Elem<DT>::load(rr[v]) : 0.f;
            // the same bits whether the gate is a row's own or stands for all
            k[v] = row_gate ? scale[v] * Elem<DT>::load(rg[v]) : scale[v];
        }
        if (row + gridDim.x < p.M) fetch(row + gridDim.x);
        float a = 1.f;
        if (p.w_post) {
#pragma unroll
            for (int v = 0; v < V; ++v) ss = fmaf(f[v], f[v], ss);
            ss = team_sum(ss, &part[parity][0], 0, t, T);
            parity ^= 1;
            a = row_rstd(ss, p.n, p.eps);
            if (t == 0 && p.rstd_post) p.rstd_post[row] = a;
            ss = 0.f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            f[v] = fmaf(f[v] * a, k[v], p.beta * r[v]);
            if (in[v]) {
                store(p.s, row * p.lds, v, f[v]);
                ss = fmaf(f[v], f[v], ss);
            }
        }
        if (p.w_pre) {
            ss = team_sum(ss, &part[parity][0], 0, t, T);
            parity ^= 1;
            const float b = row_rstd(ss, p.n, p.eps);
            if (t == 0 && p.rstd_pre) p.rstd_pre[row] = b;
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (in[v]) store(p.y, row * p.ldy, v, f[v] * b * wpre[v]);
        }
    }
}

// The same for longer rows of up to 1024 V columns, a row at a time.
template <int DT, int V>
__global__ void __launch_bounds__(1024) block_fwd_wide_columns_kernel(const BlockP p) {
    __shared__ float part[2 * 32];
    int parity = 0;
    const int t = threadIdx.x, T = blockDim.x, N = static_cast<int>(p.N);
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        float f[V], r[V], w[V], ss[1] = {0.f};
        load_columns<DT, V>(p.h, row * p.ldh, t, T, N, f);
        load_columns<DT, V>(p.r, row * p.ldr, t, T, N, r);
        float a = 1.f;
        if (p.w_post) {
#pragma unroll
            for (int v = 0; v < V; ++v) ss[0] = fmaf(f[v], f[v], ss[0]);
            block_sums<1>(ss, part, parity);
            a = row_rstd(ss[0], p.n, p.eps);
            if (t == 0 && p.rstd_post) p.rstd_post[row] = a;
            ss[0] = 0.f;
            load_columns<DT, V>(p.w_post, 0, t, T, N, w);
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] = f[v] * a * (p.alpha * (p.offset + w[v]));
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] *= p.alpha;
        }
        if (p.gate) {
            load_columns<DT, V>(p.gate, row / p.gate_rows * p.ldg, t, T, N, w);
#pragma unroll
            for (int v = 0; v < V; ++v) f[v] *= w[v];
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int j = v * T + t;
            f[v] = fmaf(p.beta, r[v], f[v]);
            if (j < N) {
                store1<DT>(p.s, row * p.lds + j, f[v]);
                ss[0] = fmaf(f[v], f[v], ss[0]);
            }
        }
        if (p.w_pre) {
            load_columns<DT, V>(p.w_pre, 0, t, T, N, w);
            block_sums<1>(ss, part, parity);
            const float b = row_rstd(ss[0], p.n, p.eps);
            if (t == 0 && p.rstd_pre) p.rstd_pre[row] = b;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int j = v * T + t;
                if (j < N) store1<DT>(p.y, row * p.ldy + j, f[v] * b * (p.offset + w[v]));
            }
        }
    }
}

template <int DT, int V, bool WIDE>
cudaError_t launch_columns(const BlockP& p, const OpCfg& c) {
    auto fn = WIDE ? block_fwd_wide_columns_kernel<DT, V> : block_fwd_columns_kernel<DT, WIDE ? 4 : V>;
    const int T = static_cast<int>((p.N + V * 32 - 1) / (V * 32)) * 32;
    const int occ = occupancy(reinterpret_cast<const void*>(fn), T, 0);
    return op_launch(c, fn, persistent_grid(p.M, 1, c.dev.sm_count, occ, c.max_ctas), T, 0, p);
}

template <int DT>
cudaError_t run(const BlockP& p, const OpCfg& c) {
    if (c.variant != RMSNORM_VARIANT_GENERIC && vectors(p)) {
        bool taken = false;
        const cudaError_t e = !p.gate              ? launch_ring<DT, 0>(p, c, &taken)
                              : p.gate_rows == 1 ? launch_ring<DT, 2>(p, c, &taken)
                                                   : launch_ring<DT, 1>(p, c, &taken);
        if (taken) return e;
    }
    if (c.variant == RMSNORM_VARIANT_CTA) return cudaErrorNotSupported;
    if (p.N <= 512 * 4) return launch_columns<DT, 4, false>(p, c);
    if (p.N <= 1024 * 4) return launch_columns<DT, 4, true>(p, c);
    if (p.N <= 1024 * 8) return launch_columns<DT, 8, true>(p, c);
    int T = 32;
    while (T < 512 && static_cast<int64_t>(T) * 4 < p.N) T <<= 1;
    auto fn = block_fwd_generic_kernel<DT>;
    const int occ = occupancy(reinterpret_cast<const void*>(fn), T, 0);
    return op_launch(c, fn, persistent_grid(p.M, 1, c.dev.sm_count, occ, c.max_ctas), T, 0, p);
}

}  // namespace

cudaError_t block_fwd_run(const BlockP& p, const OpCfg& c) {
    g_launched.store(true);
    switch (p.dtype) {
        case kBF16: return run<kBF16>(p, c);
        case kFP16: return run<kFP16>(p, c);
        default: return run<kFP32>(p, c);
    }
}

cudaError_t block_status_read_and_clear(unsigned int* value) {
    return symbol_read_and_clear(g_block_status, g_launched, value);
}

}  // namespace rmsn
