// Backward of the block operator (the formulas are in include/rmsnorm.h).
//
// One reduction per row: with u = dy (offset + w_pre), k2 = rstd_pre, n2 = k2 s,
// a = alpha gate (offset + w_post),
//
//   c2 = sum u n2,   A = sum a h (ds + k2 u),   B = sum a h n2
//   t  = ds + k2 u - e n2           e = k2 c2 / N
//   sum a h t = A - e B             (what the norm after the block subtracts)
//
// so both norms' row sums come from one pass. (n2 is of the size of 1 whatever s is;
// with s itself, rows of an RMS below 1e-13 would need k2^3 and sums of products that
// are past fp32's range where the gradients are not.) Sums over rows: P = sum of
// t h rstd_post over the rows of one gate row gives that row's dgate
// (alpha (offset + w_post) P) and its part of dw_post (alpha gate P), so one
// column sum serves both.
//
// Rows are split over the CTAs in contiguous ranges. A gate row whose rows all
// lie in one CTA's range is finished there; the others leave a partial row
// per CTA (a CTA's range starts and ends in at most two such gate rows).
// A second launch sums the partial rows in CTA order.
#include "rmsnorm.h"

#include "cluster.cuh"
#include "ops.h"
#include "ops_common.cuh"
#include "row_ring.cuh"
#include "row_ring_host.h"

#include <algorithm>

namespace rmsn {

// Bit 0: a bounded wait ran out since the last read. One word per device.
__device__ unsigned int g_block_bwd_status;
static std::atomic<bool> g_launched{false};  // a kernel that writes it

namespace {

__host__ __device__ inline int64_t range_begin(int64_t b, int64_t grid, int64_t M) {
    return b * (M / grid) + (b < M % grid ? b : M % grid);
}
// The CTA whose range holds a row.
__host__ __device__ inline int64_t range_owner(int64_t row, int64_t grid, int64_t M) {
    const int64_t q = M / grid, big = M % grid;
    return row < big * (q + 1) ? row / (q + 1) : big + (row - big * (q + 1)) / q;
}

constexpr int kCtasPerSM = 8;   // most CTAs of the kernels without teams
constexpr int kShortRow = 256;  // columns of a team of one warp

// Workspace: four areas of `slots` partial rows of `pitch` floats: dw_post and
// dw_pre (a row per CTA), gate sums that begin with a range, gate sums that
// begin inside it (a row per range: of a CTA, or of a team).
__device__ inline float* partial(float* ws, int area, int64_t i, int64_t slots, int64_t pitch) {
    return ws + (area * slots + i) * pitch;
}

// Vector kernel: row teams (row_ring.cuh) with the rows of h, s, dy, ds, and of
// the gate where each row has its own, staged in shared memory.
// GATE: 0 none, 1 one gate row for several rows, 2 a gate row per row.
// A thread owns V vectors of columns, eight columns. In registers per column: the
// scales, the sums over rows (P and dw_pre; GATE 2: dw_post and dw_pre), and of the
// current row t without its -e n2, s and h between the two passes. With a gate row
// for several rows dw_post changes only where the gate row ends: its sums are in
// shared memory, a thread's own. The arithmetic is on pairs (f32x2): scalar code
// took three times the instructions and was bound by them (16384 x 4096 bf16: 564
// warp instructions per 8 columns of 32 lanes).
// WIDE: a row's columns are more than 512 threads of eight; the CTAs of a cluster
// take a slice each, and send their row sums into each other's shared memory. (Sixteen columns per thread in one CTA spilled: 8192 x
// 8192 bf16 192 us, 8192 x 5000 241 us.)
// PARTS: kAll, kPreOnly: both norms (the one before alone) and ds are there and a
// row is exactly V vectors of every thread, which the compiler then knows: no test of
// them is left in the loop. kAny: tests.
constexpr int kAny = 0, kAll = 1, kPreOnly = 2;
template <int DT, int GATE, int PARTS, bool WIDE>
__global__ void __launch_bounds__(512) block_bwd_ring_kernel(const BlockBwdP p, const RingShape g) {
    constexpr int E = VecElems<DT>::value;
    constexpr bool FULL = PARTS != kAny;
    const bool post = PARTS == kAll || (PARTS == kAny && p.w_post);
    const bool prenorm = FULL || p.w_pre, has_ds = FULL || p.ds;
    constexpr int V = 8 / E;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ RingShared sh;
    __shared__ __align__(16) float parts[kMaxTeams][2][4 * kMaxTeamWarps];
    __shared__ float4 peers[2][8];  // WIDE: the sums of the cluster's CTAs, and their arrival
    __shared__ uint64_t peer_bars[2];

    const int team = threadIdx.x / g.T, t = threadIdx.x - team * g.T;
    // WIDE: this CTA's slice of the row begins at vector first_vec.
    const int rank = WIDE ? static_cast<int>(cluster_rank()) : 0;
    const int first_vec = WIDE ? rank * g.slice : 0;
    const int nvec = WIDE ? min(g.slice, g.nvec - first_vec) : g.nvec;
    const int64_t group = WIDE ? blockIdx.x / g.cluster : blockIdx.x;
    const int64_t me = group * g.teams + team;
    const int64_t r0 = me * g.q + (me < g.rem ? me : g.rem);
    const int rows = static_cast<int>(g.q) + (me < g.rem ? 1 : 0);
    Ring ring;
    ring.row_bytes = static_cast<uint32_t>(nvec) * 16u;
    ring.stage_bytes = ring.row_bytes * g.arrays;
    ring.base = smem_u32(smem) + static_cast<uint32_t>(team * g.stages) * ring.stage_bytes;
    ring.bars = smem_u32(&sh.bars[team][0]);
    // dw_post sums of GATE 1, [V * E / 4][threads] float4 behind the rings.
    float4* post_sums = reinterpret_cast<float4*>(smem + g.sums_at);
    if (t == 0) {
        for (int st = 0; st < g.stages; ++st) mbar_init(ring.bar(st), 1);
        if (WIDE) {
            mbar_init(smem_u32(&peer_bars[0]), 1);
            mbar_init(smem_u32(&peer_bars[1]), 1);
        }
        fence_mbar_init();
        sh.give_up[team].clear();
    }
    for (int i = t; i < 2 * 4 * kMaxTeamWarps; i += g.T) parts[team][0][i] = 0.f;
    const bool need_h = post || GATE != 0;
    // Which array of a stage each tensor is.
    int n_arrays = 0;
    const int ih = need_h ? n_arrays++ : 0;
    const int is = prenorm ? n_arrays++ : 0;
    const int idy = prenorm ? n_arrays++ : 0;
    const int ids = has_ds ? n_arrays++ : 0;
    const int ig = n_arrays;
    auto issue = [&](int row, int st) {
        const int64_t i = r0 + row;
        ring.expect(st);
        if (need_h) ring.copy(st, ih, static_cast<const uint4*>(p.h) + first_vec + i * p.ldh);
        if (prenorm) {
            ring.copy(st, is, static_cast<const uint4*>(p.s) + first_vec + i * p.lds);
            ring.copy(st, idy, static_cast<const uint4*>(p.dy) + first_vec + i * p.lddy);
        }
        if (has_ds) ring.copy(st, ids, static_cast<const uint4*>(p.ds) + first_vec + i * p.ldds);
        if (GATE == 2) ring.copy(st, ig, static_cast<const uint4*>(p.gate) + first_vec + i * p.ldg);
    };
    pdl_wait();
    if (t == 0) {
        for (int k = 0; k < g.stages && k < rows; ++k) issue(k, k);
    }
    constexpr int H = E / 2;
    const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
    const uint4* w_post = p.w_post ? static_cast<const uint4*>(p.w_post) + first_vec : nullptr;
    const uint4* w_pre = p.w_pre ? static_cast<const uint4*>(p.w_pre) + first_vec : nullptr;
    const uint4* gate = static_cast<const uint4*>(p.gate) + first_vec;
    // Per column, as pairs: a = alpha gate (offset + w_post) (GATE 2: without the
    // gate) and offset + w_pre.
    f2 a[V][H], wpre[V][H];
    int64_t grow = 0, left = 0;
    if (GATE == 1) {
        grow = r0 / p.gate_rows;
        left = (grow + 1) * p.gate_rows - r0;
    }
    auto column = [&](int v) { return v * g.T + t; };
    // alpha (offset + w_post) of a vector of columns.
    auto post_scale = [&](int v, f2* o) {
        const int c = column(v);
        if (post) {
            weights2<DT>(c < nvec ? __ldg(w_post + c) : zero4, p.offset, o);
#pragma unroll
            for (int e = 0; e < H; ++e) o[e] = f2_mul(o[e], f2_dup(p.alpha));
        } else {
#pragma unroll
            for (int e = 0; e < H; ++e) o[e] = f2_dup(p.alpha);
        }
    };
    auto gate_row = [&](int v, f2* o) {
        const int c = column(v);
        unpack2<DT>(c < nvec ? __ldg(gate + grow * p.ldg + c) : zero4, o);
    };
    auto load_scale = [&]() {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            post_scale(v, a[v]);
            if (GATE == 1) {
                f2 x[H];
                gate_row(v, x);
#pragma unroll
                for (int e = 0; e < H; ++e) a[v][e] = f2_mul(a[v][e], x[e]);
            }
        }
    };
    load_scale();
    f2 P[V][H], pre[V][H];  // GATE 2: P is dw_post without its alpha
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = column(v);
        weights2<DT>(w_pre && c < nvec ? __ldg(w_pre + c) : zero4, p.offset, wpre[v]);
#pragma unroll
        for (int e = 0; e < H; ++e) P[v][e] = pre[v][e] = 0;
    }
    if (GATE == 1) {
#pragma unroll
        for (int i = 0; i < V * E / 4; ++i)
            post_sums[i * blockDim.x + threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (WIDE) cluster_sync();  // the others run before anything is written to them
    else __syncthreads();

    int st = 0, parity = 0;
    uint32_t phase = 0;
    bool dead = false, lost = false;
    int row = 0, dead_row = 0;
    const f2 beta = f2_dup(p.beta);
    const float inv_n = 1.f / p.n;
    const float* rstd_post = p.rstd_post + r0;
    const float* rstd_pre = p.rstd_pre + r0;
    float k1_next = post ? __ldg(rstd_post) : 1.f;
    float k2_next = prenorm ? __ldg(rstd_pre) : 0.f;
    uint4* dr = static_cast<uint4*>(p.dr) + r0 * p.lddr + first_vec + t;
    uint4* dh = static_cast<uint4*>(p.dh) + r0 * p.lddh + first_vec + t;
    uint4* dgate = static_cast<uint4*>(p.dgate) + (GATE == 2 ? r0 * p.lddg + first_vec + t : 0);
    // Vectors of the row; those past its end stay zero.
    uint4 hv[V], sv[V], gv[V], dyv[V], dsv[V];
#pragma unroll
    for (int v = 0; v < V; ++v) hv[v] = sv[v] = gv[v] = dyv[v] = dsv[v] = zero4;
    const uint32_t oh = 16u * t + ih * ring.row_bytes, os = 16u * t + is * ring.row_bytes;
    const uint32_t ody = 16u * t + idy * ring.row_bytes, ods = 16u * t + ids * ring.row_bytes;
    const uint32_t og = 16u * t + ig * ring.row_bytes;
    for (; row < rows; ++row, dr += p.lddr, dh += p.lddh) {
        if (GATE == 1 && left == 0) {
            ++grow;
            left = p.gate_rows;
            load_scale();
        }
        if (!(WIDE && dead) && !mbar_wait_bounded(ring.bar(st), phase, g.limit)) sh.give_up[team].mark(row);
        const float k1 = k1_next, k2 = k2_next;
        if (row + 1 < rows) {  // the next row's, a global load ahead of its use
            if (post) k1_next = __ldg(rstd_post + row + 1);
            if (prenorm) k2_next = __ldg(rstd_pre + row + 1);
        }
        f2 t0[V][H];
        f2 us = 0, aht = 0, ahs = 0;
        const f2 k22 = f2_dup(k2);
        const uint32_t at = ring.stage(st);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (FULL || column(v) < nvec) {
                const uint32_t q = at + 16u * (v * g.T);
                if (need_h) hv[v] = lds16(q + oh);
                if (prenorm) {
                    sv[v] = lds16(q + os);
                    dyv[v] = lds16(q + ody);
                }
                if (has_ds) dsv[v] = lds16(q + ods);
                if (GATE == 2) gv[v] = lds16(q + og);
            }
            unpack2<DT>(dsv[v], t0[v]);
            f2 s[H];
            unpack2<DT>(sv[v], s);
            if (prenorm) {
                f2 dy[H];
                unpack2<DT>(dyv[v], dy);
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    const f2 u = f2_mul(dy[e], wpre[v][e]);
                    t0[v][e] = f2_fma(k22, u, t0[v][e]);
                    s[e] = f2_mul(s[e], k22);  // n2
                    us = f2_fma(u, s[e], us);
                    pre[v][e] = f2_fma(dy[e], s[e], pre[v][e]);
                }
            }
            if (post) {
                f2 h[H], x[H];
                unpack2<DT>(hv[v], h);
                if (GATE == 2) unpack2<DT>(gv[v], x);
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    f2 ah = f2_mul(a[v][e], h[e]);
                    if (GATE == 2) ah = f2_mul(ah, x[e]);
                    aht = f2_fma(ah, t0[v][e], aht);
                    ahs = f2_fma(ah, s[e], ahs);
                }
            }
        }
        float sums[3] = {f2_sum(us), f2_sum(aht), f2_sum(ahs)};
        team_sums3(sums, &parts[team][parity][0], team, t, g.T);
        parity ^= 1;
        if (!(WIDE && dead)) {
            dead = sh.give_up[team].at(row);
            if (WIDE) dead_row = row;
        }
        if (!dead && t == 0 && row + g.stages < rows) issue(row + g.stages, st);
        if (WIDE) {
            // Slot and barrier of this row, used again two rows on: a CTA sends a row's
            // sums when all its threads have read those of the row before. A CTA that
            // gave up says so, stores nothing more, and so do the others from the next
            // row on; but all of them send and receive to the last row, so that nothing
            // is on its way to a CTA that has ended.
            const int slot = row & 1;
            const uint32_t bar = smem_u32(&peer_bars[slot]);
            if (t == 0) mbar_arrive_expect_tx(bar, 16u * g.cluster);
            if (t < g.cluster)
                st_async_peer_f4(smem_u32(&peers[slot][rank]), bar, t, sums[0], sums[1], sums[2], dead ? 1.f : 0.f);
            if (!lost && !mbar_wait_bounded(bar, (row >> 1) & 1, g.drain)) {
                lost = true;
                sh.give_up[team].mark(row + 1);
            }
            float4 x = peers[slot][0];  // added in rank order, so that all get the same
            for (int i = 1; i < g.cluster; ++i) {
                const float4 z = peers[slot][i];
                x.x += z.x;
                x.y += z.y;
                x.z += z.z;
                x.w += z.w;
            }
            sums[0] = x.x;
            sums[1] = x.y;
            sums[2] = x.z;
            if (x.w != 0.f) sh.give_up[team].mark(row + 1);
            if (dead) continue;
        } else if (dead) {
            break;
        }
        const float e2 = k2 * (sums[0] * inv_n);
        const float f = k1 * (k1 * (fmaf(-e2, sums[2], sums[1]) * inv_n));
        const f2 me2 = f2_dup(-(e2 * k2)), k12 = f2_dup(k1), mf = f2_dup(-(k1 * f));  // me2: of s
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool in = FULL || column(v) < nvec;
            f2 s[H], h[H], x[H], o[H];
            unpack2<DT>(sv[v], s);
            unpack2<DT>(hv[v], h);
            if (GATE == 2) unpack2<DT>(gv[v], x);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                t0[v][e] = f2_fma(me2, s[e], t0[v][e]);
                o[e] = f2_mul(beta, t0[v][e]);
            }
            if (in) st_stream(dr + v * g.T, pack2<DT>(o));
            if (GATE == 2) {
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    const f2 th = f2_mul(t0[v][e], f2_mul(h[e], k12));
                    P[v][e] = f2_fma(th, x[e], P[v][e]);
                    o[e] = f2_mul(a[v][e], th);
                }
                if (in) st_stream(dgate + v * g.T, pack2<DT>(o));
            } else if (need_h) {
#pragma unroll
                for (int e = 0; e < H; ++e) P[v][e] = f2_fma(t0[v][e], f2_mul(h[e], k12), P[v][e]);
            }
#pragma unroll
            for (int e = 0; e < H; ++e) {
                f2 q = f2_mul(a[v][e], k12);
                if (GATE == 2) q = f2_mul(q, x[e]);
                o[e] = f2_mul(q, t0[v][e]);
                if (post) o[e] = f2_fma(mf, h[e], o[e]);
            }
            if (in) st_stream(dh + v * g.T, pack2<DT>(o));
        }
        if (GATE == 2) dgate += p.lddg;
        if (GATE == 1 && (--left == 0 || row + 1 == rows)) {
            // The end of a gate row's rows here: their P into dw_post's sums, and
            // out as dgate where they are all of the gate row's rows.
            const int64_t first = grow * p.gate_rows;
            const int64_t last = first + p.gate_rows < p.M ? first + p.gate_rows : p.M;
            const bool whole = first >= r0 && last <= r0 + rows;
            float* out = partial(p.ws, first > r0 ? 3 : 2, me, g.slots, block_bwd_pitch(p.N)) + first_vec * E;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = column(v);
                const bool in = c < nvec;
                f2 q[H], o[H];
                gate_row(v, q);
                post_scale(v, o);
#pragma unroll
                for (int i = 0; i < E / 4; ++i) {
                    const f2 p0 = P[v][2 * i], p1 = P[v][2 * i + 1];
                    float4& acc = post_sums[(v * (E / 4) + i) * blockDim.x + threadIdx.x];
                    const float4 x = acc;
                    const float2 lo = f2_get(f2_fma(p0, q[2 * i], f2_make(x.x, x.y)));
                    const float2 hi = f2_get(f2_fma(p1, q[2 * i + 1], f2_make(x.z, x.w)));
                    acc = make_float4(lo.x, lo.y, hi.x, hi.y);
                    const float2 u = f2_get(p0), w = f2_get(p1);
                    if (in && !whole)
                        reinterpret_cast<float4*>(out)[c * (E / 4) + i] = make_float4(u.x, u.y, w.x, w.y);
                }
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    o[e] = f2_mul(o[e], P[v][e]);
                    P[v][e] = 0;
                }
                if (in && whole)
                    static_cast<uint4*>(p.dgate)[grow * p.lddg + first_vec + c] = pack2<DT>(o);
            }
        }
        if (++st == g.stages) {
            st = 0;
            phase ^= 1;
        }
    }
    if ((dead || lost) && t == 0) {
        atomicOr(&g_block_bwd_status, 1u);
        // Rows below the one given up at + stages were issued and may still be landing
        // (its stage and phase are still the current ones).
        if (!WIDE) dead_row = row;
        for (int i = dead_row; dead && i < dead_row + g.stages && i < rows; ++i) {
            mbar_wait_bounded(ring.bar(st), phase, g.drain);
            if (++st == g.stages) {
                st = 0;
                phase ^= 1;
            }
        }
    }
    if (WIDE) cluster_sync();  // nobody writes to a CTA that has ended
    pdl_launch_dependents();
    // The teams' column sums, added in team order through the rings' memory,
    // into the CTA's partial rows.
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (which == 0 ? !w_post : !w_pre) continue;
        float4* all = reinterpret_cast<float4*>(smem);
        __syncthreads();  // the rings, or the sums of the round before, are done with
#pragma unroll
        for (int i = 0; i < V * E / 4; ++i) {
            const int v = i / (E / 4), e = 2 * (i % (E / 4));
            const float2 lo = f2_get(which == 0 ? P[v][e] : pre[v][e]);
            const float2 hi = f2_get(which == 0 ? P[v][e + 1] : pre[v][e + 1]);
            float4 x = make_float4(lo.x, lo.y, hi.x, hi.y);
            if (which == 0 && GATE == 1) x = post_sums[i * blockDim.x + threadIdx.x];
            if (which == 0) x = make_float4(p.alpha * x.x, p.alpha * x.y, p.alpha * x.z, p.alpha * x.w);
            if (g.teams > 1) all[i * blockDim.x + threadIdx.x] = x;
            else {
                const int c = (i / (E / 4)) * g.T + t;
                if (c < nvec)
                    reinterpret_cast<float4*>(partial(p.ws, which, group, g.slots, block_bwd_pitch(p.N)) + first_vec * E)
                        [c * (E / 4) + i % (E / 4)] = x;
            }
        }
        if (g.teams == 1) continue;
        __syncthreads();
        if (team == 0) {
#pragma unroll
            for (int i = 0; i < V * E / 4; ++i) {
                const int c = (i / (E / 4)) * g.T + t;
                float4 x = all[i * blockDim.x + t];
                for (int k = 1; k < g.teams; ++k) {
                    const float4 z = all[i * blockDim.x + k * g.T + t];
                    x.x += z.x;
                    x.y += z.y;
                    x.z += z.z;
                    x.w += z.w;
                }
                if (c < nvec)
                    reinterpret_cast<float4*>(partial(p.ws, which, group, g.slots, block_bwd_pitch(p.N)) + first_vec * E)
                        [c * (E / 4) + i % (E / 4)] = x;
            }
        }
    }
}

// Element-wise kernel for rows that no other takes; a thread owns the columns
// tid, tid + T, ... and keeps their sums in the CTA's partial rows.
template <int DT>
__global__ void __launch_bounds__(512) block_bwd_generic_kernel(const BlockBwdP p, int64_t slots) {
    __shared__ float part[2 * 3 * 32];
    int parity = 0;
    const int tid = threadIdx.x, T = blockDim.x;
    const int64_t G = gridDim.x, b = blockIdx.x, pitch = block_bwd_pitch(p.N);
    const int64_t r0 = range_begin(b, G, p.M), r1 = range_begin(b + 1, G, p.M);
    float* acc_post = partial(p.ws, 0, b, slots, pitch);
    float* acc_pre = partial(p.ws, 1, b, slots, pitch);
    const bool per_element = p.gate && p.gate_rows == 1;
    const bool grouped = p.gate && !per_element;
    pdl_wait();
    for (int64_t j = tid; j < p.N; j += T) {
        if (p.w_post) acc_post[j] = 0.f;
        if (p.w_pre) acc_pre[j] = 0.f;
    }
    float* acc_gate = nullptr;
    for (int64_t row = r0; row < r1; ++row) {
        const int64_t h0 = row * p.ldh, s0 = row * p.lds, dy0 = row * p.lddy, ds0 = row * p.ldds;
        const int64_t grow = p.gate ? row / p.gate_rows : 0;
        const int64_t g0 = grow * p.ldg;
        if (grouped && (row == r0 || row % p.gate_rows == 0)) {
            acc_gate = partial(p.ws, row == r0 ? 2 : 3, b, slots, pitch);
            for (int64_t j = tid; j < p.N; j += T) acc_gate[j] = 0.f;
        }
        const float k1 = p.w_post ? p.rstd_post[row] : 1.f;
        const float k2 = p.w_pre ? p.rstd_pre[row] : 0.f;
        auto scale = [&](int64_t j) {  // a
            float a = p.alpha;
            if (p.gate) a *= load1<DT>(p.gate, g0 + j);
            if (p.w_post) a *= p.offset + load1<DT>(p.w_post, j);
            return a;
        };
        float v[3] = {0.f, 0.f, 0.f};
        for (int64_t j = tid; j < p.N; j += T) {
            const float s = p.w_pre ? load1<DT>(p.s, s0 + j) * k2 : 0.f;  // n2
            const float u = p.w_pre ? load1<DT>(p.dy, dy0 + j) * (p.offset + load1<DT>(p.w_pre, j)) : 0.f;
            const float d = p.ds ? load1<DT>(p.ds, ds0 + j) : 0.f;
            v[0] = fmaf(u, s, v[0]);
            if (p.w_post) {
                const float ah = scale(j) * load1<DT>(p.h, h0 + j);
                v[1] = fmaf(ah, fmaf(k2, u, d), v[1]);
                v[2] = fmaf(ah, s, v[2]);
            }
        }
        block_sums<3>(v, part, parity);
        const float e = k2 * (v[0] / p.n);
        const float f = k1 * (k1 * (fmaf(-e, v[2], v[1]) / p.n));
        for (int64_t j = tid; j < p.N; j += T) {
            float t = p.ds ? load1<DT>(p.ds, ds0 + j) : 0.f;
            const float a = scale(j);
            const float h = load1<DT>(p.h, h0 + j);
            if (p.w_pre) {
                const float s = load1<DT>(p.s, s0 + j) * k2, dy = load1<DT>(p.dy, dy0 + j);
                t = fmaf(k2, dy * (p.offset + load1<DT>(p.w_pre, j)), t);
                t = fmaf(-e, s, t);
                acc_pre[j] = fmaf(dy, s, acc_pre[j]);
            }
            const float th = t * (h * k1);
            store1<DT>(p.dr, row * p.lddr + j, p.beta * t);
            store1<DT>(p.dh, row * p.lddh + j, p.w_post ? k1 * fmaf(a, t, -h * f) : a * t);
            if (per_element) {
                const float gw = p.alpha * th;
                store1<DT>(p.dgate, row * p.lddg + j,
                           p.w_post ? gw * (p.offset + load1<DT>(p.w_post, j)) : gw);
                if (p.w_post) acc_post[j] = fmaf(gw, load1<DT>(p.gate, g0 + j), acc_post[j]);
            } else if (grouped) {
                acc_gate[j] += th;
            } else if (p.w_post) {
                acc_post[j] = fmaf(p.alpha, th, acc_post[j]);
            }
        }
        if (grouped && (row + 1 == r1 || (row + 1) % p.gate_rows == 0)) {
            const int64_t first = grow * p.gate_rows;
            const int64_t last = first + p.gate_rows < p.M ? first + p.gate_rows : p.M;
            const bool whole = first >= r0 && last <= r1;
            for (int64_t j = tid; j < p.N; j += T) {
                const float q = p.alpha * acc_gate[j];
                if (p.w_post) acc_post[j] = fmaf(q, load1<DT>(p.gate, g0 + j), acc_post[j]);
                if (whole)
                    store1<DT>(p.dgate, grow * p.lddg + j,
                               p.w_post ? q * (p.offset + load1<DT>(p.w_post, j)) : q);
            }
        }
    }
    pdl_launch_dependents();
}

// Rows that are not whole vectors (any N, stride and alignment), of up to 512 V
// columns: a CTA per range of rows, element loads, a thread's columns t, t + T, ...
// of the row, its scales and the sums in registers (dw_post's sums with a gate row
// for several rows in shared memory). The next row is loaded into registers while
// this one is reduced, and a load is one instruction (GB300, us, against the kernel
// below: 18503x708 bf16 105 -> 72, 23493x987 fp32 161 -> 112, 16384x777 bf16 117 ->
// 76).
template <int DT, int V>
__global__ void __launch_bounds__(512) block_bwd_columns_kernel(const BlockBwdP p, int64_t slots) {
    using Raw = typename Elem<DT>::T;
    extern __shared__ __align__(16) float post[];  // [V][T]
    __shared__ __align__(16) float part[2][4 * kMaxTeamWarps];
    int parity = 0;
    const int t = threadIdx.x, T = blockDim.x, N = static_cast<int>(p.N);
    const int64_t G = gridDim.x, b = blockIdx.x, pitch = block_bwd_pitch(p.N);
    const int64_t r0 = range_begin(b, G, p.M), r1 = range_begin(b + 1, G, p.M);
    const bool per_element = p.gate && p.gate_rows == 1;
    const bool grouped = p.gate && !per_element;
    const float inv_n = 1.f / p.n;
    Raw rh[V], rs[V], rdy[V], rds[V];
    // Byte offsets of the thread's columns (past the row's end: of the last one): a
    // row's base is the same for all threads, and a load is one instruction.
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
        if (p.ds) load_raw(p.ds, row * p.ldds, rds);
        if (p.w_pre) {
            load_raw(p.s, row * p.lds, rs);
            load_raw(p.dy, row * p.lddy, rdy);
        }
    };
    auto unpacked = [&](const Raw (&x)[V], float (&out)[V]) {  // zero past the row's end
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] = in[v] ? Elem<DT>::load(x[v]) : 0.f;
    };
    for (int i = t; i < 2 * 4 * kMaxTeamWarps; i += T) part[0][i] = 0.f;
    __syncthreads();
    pdl_wait();
    fetch(r0);
    float P[V], pre[V];  // P: sums of t h rstd_post (times the gate where a row has its own)
    float a[V], wpre[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        P[v] = pre[v] = wpre[v] = 0.f;
        if (grouped) post[v * T + t] = 0.f;
    }
    if (p.w_pre) {
        load_columns<DT, V>(p.w_pre, 0, t, T, N, wpre);
#pragma unroll
        for (int v = 0; v < V; ++v) wpre[v] += p.offset;
    }
    int64_t grow = grouped ? r0 / p.gate_rows : 0;
    int64_t left = grouped ? (grow + 1) * p.gate_rows - r0 : 0;
    float k1_next = p.w_post ? __ldg(p.rstd_post + r0) : 1.f;
    float k2_next = p.w_pre ? __ldg(p.rstd_pre + r0) : 0.f;
    // alpha (offset + w_post) of the thread's columns.
    auto post_scale = [&](float (&o)[V]) {
        if (p.w_post) load_columns<DT, V>(p.w_post, 0, t, T, N, o);
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = p.w_post ? p.alpha * (p.offset + o[v]) : p.alpha;
    };
    // a: times the gate row, but where each row has its own.
    auto load_scale = [&]() {
        post_scale(a);
        if (!grouped) return;
        float q[V];
        load_columns<DT, V>(p.gate, grow * p.ldg, t, T, N, q);
#pragma unroll
        for (int v = 0; v < V; ++v) a[v] *= q[v];
    };
    load_scale();
    for (int64_t row = r0; row < r1; ++row) {
        const float k1 = k1_next, k2 = k2_next;
        if (row + 1 < r1) {
            if (p.w_post) k1_next = __ldg(p.rstd_post + row + 1);
            if (p.w_pre) k2_next = __ldg(p.rstd_pre + row + 1);
        }
        float t0[V], h[V], s[V], q[V], sums[3] = {0.f, 0.f, 0.f};
        unpacked(rh, h);
        if (per_element) {
            Raw x[V];
            load_raw(p.gate, row * p.ldg, x);
            unpacked(x, q);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            t0[v] = s[v] = 0.f;
            if (!per_element) q[v] = 1.f;
        }
        if (p.ds) unpacked(rds, t0);
        if (p.w_pre) {
            float dy[V];
            unpacked(rs, s);
            unpacked(rdy, dy);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float u = dy[v] * wpre[v];
                t0[v] = fmaf(k2, u, t0[v]);
                s[v] *= k2;  // n2
                sums[0] = fmaf(u, s[v], sums[0]);
                pre[v] = fmaf(dy[v], s[v], pre[v]);
            }
        }
        if (row + 1 < r1) fetch(row + 1);
        if (p.w_post) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float ah = a[v] * q[v] * h[v];
                sums[1] = fmaf(ah, t0[v], sums[1]);
                sums[2] = fmaf(ah, s[v], sums[2]);
            }
        }
        team_sums3(sums, &part[parity][0], 0, t, T);
        parity ^= 1;
        const float e = k2 * (sums[0] * inv_n);
        const float f = k1 * (k1 * (fmaf(-e, sums[2], sums[1]) * inv_n));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            t0[v] = fmaf(-e, s[v], t0[v]);
            const float th = t0[v] * (h[v] * k1);
            if (!in[v]) continue;
            const float aq = a[v] * q[v];
            store(p.dr, row * p.lddr, v, p.beta * t0[v]);
            store(p.dh, row * p.lddh, v, p.w_post ? k1 * fmaf(aq, t0[v], -h[v] * f) : aq * t0[v]);
            if (per_element) store(p.dgate, row * p.lddg, v, a[v] * th);
            P[v] = fmaf(th, q[v], P[v]);
        }
        if (grouped && (--left == 0 || row + 1 == r1)) {
            const int64_t first = grow * p.gate_rows;
            const int64_t last = first + p.gate_rows < p.M ? first + p.gate_rows : p.M;
            const bool whole = first >= r0 && last <= r1;
            float* out = partial(p.ws, first > r0 ? 3 : 2, b, slots, pitch);
            load_columns<DT, V>(p.gate, grow * p.ldg, t, T, N, q);
            post_scale(t0);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int j = v * T + t;
                if (j < N) {
                    post[j] = fmaf(P[v], q[v], post[j]);
                    if (whole) store1<DT>(p.dgate, grow * p.lddg + j, t0[v] * P[v]);
                    else out[j] = P[v];
                }
                P[v] = 0.f;
            }
            ++grow;
            left = p.gate_rows;
            if (row + 1 < r1) load_scale();
        }
    }
    pdl_launch_dependents();
    float* acc_post = partial(p.ws, 0, b, slots, pitch);
    float* acc_pre = partial(p.ws, 1, b, slots, pitch);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int j = v * T + t;
        if (j >= N) continue;
        if (p.w_post) acc_post[j] = p.alpha * (grouped ? post[j] : P[v]);
        if (p.w_pre) acc_pre[j] = pre[v];
    }
}

// The same for longer rows of up to 1024 V columns, whose next row and scales would
// not fit into registers (4096x3001 bf16 106 us, with them 152): a CTA per range of rows, element loads, a thread's columns t, t + T, ...
// of the row and of the sums in registers (dw_post's with a gate row for several
// rows in shared memory).
template <int DT, int V>
__global__ void __launch_bounds__(1024) block_bwd_wide_columns_kernel(const BlockBwdP p, int64_t slots) {
    extern __shared__ __align__(16) float post[];  // [V][T]
    __shared__ float part[2 * 3 * 32];
    int parity = 0;
    const int t = threadIdx.x, T = blockDim.x, N = static_cast<int>(p.N);
    const int64_t G = gridDim.x, b = blockIdx.x, pitch = block_bwd_pitch(p.N);
    const int64_t r0 = range_begin(b, G, p.M), r1 = range_begin(b + 1, G, p.M);
    const bool per_element = p.gate && p.gate_rows == 1;
    const bool grouped = p.gate && !per_element;
    const float inv_n = 1.f / p.n;
    pdl_wait();
    float P[V], pre[V];  // P: sums of t h rstd_post (times the gate where a row has its own)
#pragma unroll
    for (int v = 0; v < V; ++v) {
        P[v] = pre[v] = 0.f;
        if (grouped) post[v * T + t] = 0.f;
    }
    int64_t grow = grouped ? r0 / p.gate_rows : 0;
    int64_t left = grouped ? (grow + 1) * p.gate_rows - r0 : 0;
    float k1_next = p.w_post ? __ldg(p.rstd_post + r0) : 1.f;
    float k2_next = p.w_pre ? __ldg(p.rstd_pre + r0) : 0.f;
    // alpha gate (offset + w_post) of the thread's columns; `wp` without the gate.
    auto scales = [&](int64_t row, float (&a)[V], bool with_gate) {
        if (p.w_post) {
            load_columns<DT, V>(p.w_post, 0, t, T, N, a);
#pragma unroll
            for (int v = 0; v < V; ++v) a[v] = p.alpha * (p.offset + a[v]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) a[v] = p.alpha;
        }
        if (with_gate && p.gate) {
            float q[V];
            load_columns<DT, V>(p.gate, (per_element ? row : grow) * p.ldg, t, T, N, q);
#pragma unroll
            for (int v = 0; v < V; ++v) a[v] *= q[v];
        }
    };
    for (int64_t row = r0; row < r1; ++row) {
        const float k1 = k1_next, k2 = k2_next;
        if (row + 1 < r1) {
            if (p.w_post) k1_next = __ldg(p.rstd_post + row + 1);
            if (p.w_pre) k2_next = __ldg(p.rstd_pre + row + 1);
        }
        float t0[V], h[V], s[V], a[V], sums[3] = {0.f, 0.f, 0.f};
        load_columns<DT, V>(p.h, row * p.ldh, t, T, N, h);
        if (p.ds) {
            load_columns<DT, V>(p.ds, row * p.ldds, t, T, N, t0);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) t0[v] = 0.f;
        }
        if (p.w_pre) {
            float dy[V];
            load_columns<DT, V>(p.s, row * p.lds, t, T, N, s);
            load_columns<DT, V>(p.dy, row * p.lddy, t, T, N, dy);
            load_columns<DT, V>(p.w_pre, 0, t, T, N, a);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float u = dy[v] * (p.offset + a[v]);
                t0[v] = fmaf(k2, u, t0[v]);
                s[v] *= k2;  // n2
                sums[0] = fmaf(u, s[v], sums[0]);
                pre[v] = fmaf(dy[v], s[v], pre[v]);
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = 0.f;
        }
        scales(row, a, true);
        if (p.w_post) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float ah = a[v] * h[v];
                sums[1] = fmaf(ah, t0[v], sums[1]);
                sums[2] = fmaf(ah, s[v], sums[2]);
            }
        }
        block_sums<3>(sums, part, parity);
        const float e = k2 * (sums[0] * inv_n);
        const float f = k1 * (k1 * (fmaf(-e, sums[2], sums[1]) * inv_n));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int j = v * T + t;
            t0[v] = fmaf(-e, s[v], t0[v]);
            s[v] = t0[v] * (h[v] * k1);  // what P sums
            if (j < N) {
                store1<DT>(p.dr, row * p.lddr + j, p.beta * t0[v]);
                store1<DT>(p.dh, row * p.lddh + j, p.w_post ? k1 * fmaf(a[v], t0[v], -h[v] * f) : a[v] * t0[v]);
            }
        }
        if (per_element) {
            load_columns<DT, V>(p.gate, row * p.ldg, t, T, N, h);
            scales(row, a, false);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int j = v * T + t;
                if (j < N) {
                    store1<DT>(p.dgate, row * p.lddg + j, a[v] * s[v]);
                    P[v] = fmaf(s[v], h[v], P[v]);
                }
            }
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v * T + t < N) P[v] += s[v];
        }
        if (grouped && (--left == 0 || row + 1 == r1)) {
            const int64_t first = grow * p.gate_rows;
            const int64_t last = first + p.gate_rows < p.M ? first + p.gate_rows : p.M;
            const bool whole = first >= r0 && last <= r1;
            float* out = partial(p.ws, first > r0 ? 3 : 2, b, slots, pitch);
            load_columns<DT, V>(p.gate, grow * p.ldg, t, T, N, h);
            scales(row, a, false);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int j = v * T + t;
                if (j < N) {
                    post[j] = fmaf(P[v], h[v], post[j]);
                    if (whole) store1<DT>(p.dgate, grow * p.lddg + j, a[v] * P[v]);
                    else out[j] = P[v];
                }
                P[v] = 0.f;
            }
            ++grow;
            left = p.gate_rows;
        }
    }
    pdl_launch_dependents();
    float* acc_post = partial(p.ws, 0, b, slots, pitch);
    float* acc_pre = partial(p.ws, 1, b, slots, pitch);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int j = v * T + t;
        if (j >= N) continue;
        if (p.w_post) acc_post[j] = p.alpha * (grouped ? post[j] : P[v]);
        if (p.w_pre) acc_pre[j] = pre[v];
    }
}

template <int DT>
cudaError_t finish(const BlockBwdP& p, const OpCfg& c, int64_t slots, int64_t G, int64_t R);

template <int DT, int V, bool WIDE>
cudaError_t launch_columns(const BlockBwdP& p, const OpCfg& c) {
    auto fn = WIDE ? block_bwd_wide_columns_kernel<DT, V> : block_bwd_columns_kernel<DT, WIDE ? 4 : V>;
    const int T = static_cast<int>((p.N + V * 32 - 1) / (V * 32)) * 32;
    const int smem = p.gate && p.gate_rows > 1 ? V * T * 4 : 0;  // at most 32 KB
    const int occ = occupancy(reinterpret_cast<const void*>(fn), T, smem);
    const int64_t slots = block_bwd_max_grid(p.M, p.N, c.dev.sm_count);
    const int64_t G = std::min<int64_t>(
        slots, persistent_grid(p.M, 1, c.dev.sm_count, std::min(occ, kCtasPerSM), c.max_ctas));
    const cudaError_t e = op_launch(c, fn, G, T, smem, p, slots);
    return e != cudaSuccess ? e : finish<DT>(p, c, slots, G, G);
}

// Sums of the partial rows in order: dw_post and dw_pre over the G CTAs, and
// the gate rows that more than one of the R ranges worked on. Latency is what this
// launch costs, so a CTA sums 32 columns only: groups of eight threads, as many as
// there are eights of partial rows (16 to 64), take every so many-th partial row,
// eight loads in flight each, and meet by shuffles and then in shared memory in a
// fixed order. blockIdx.y: 0 dw_post, 1 dw_pre, then gate rows.
// `flat`: gate rows are short and many, each in few ranges. Then the CTAs behind
// the first two rows of the grid go over the borders between ranges instead, a thread
// per border and four columns: a gate row is summed at the first border inside it.
template <int DT>
__global__ void __launch_bounds__(512) block_bwd_finish_kernel(const BlockBwdP p, int64_t slots, int64_t G,
                                                               int64_t R, bool flat) {
    __shared__ float4 red[16][8];
    const int64_t pitch = block_bwd_pitch(p.N);
    auto put_gate = [&](int64_t grow, int64_t j, float s) {
        s *= p.alpha;
        if (p.w_post) s *= p.offset + load1<DT>(p.w_post, j);
        store1<DT>(p.dgate, grow * p.lddg + j, s);
    };
    if (flat && blockIdx.y >= 2) {
        const int64_t nv = (p.N + 3) / 4, all = (R - 1) * nv;
        const int64_t me = (static_cast<int64_t>(blockIdx.y - 2) * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x;
        pdl_wait();
        for (int64_t i = me; i < all; i += static_cast<int64_t>(gridDim.y - 2) * gridDim.x * blockDim.x) {
            const int64_t b = 1 + i / nv, j4 = i - (b - 1) * nv;
            const int64_t begin = range_begin(b, R, p.M), before = range_begin(b - 1, R, p.M);
            const int64_t grow = begin / p.gate_rows, first = grow * p.gate_rows;
            if (first == begin || before > first) continue;  // no gate row is split, or not first here
            const int64_t last = first + p.gate_rows < p.M ? first + p.gate_rows : p.M;
            float4 x = reinterpret_cast<const float4*>(
                partial(p.ws, before < first ? 3 : 2, b - 1, slots, pitch))[j4];
            for (int64_t k = b, at = begin; at < last; at = range_begin(++k, R, p.M)) {
                const float4 z = reinterpret_cast<const float4*>(partial(p.ws, 2, k, slots, pitch))[j4];
                x.x += z.x;
                x.y += z.y;
                x.z += z.z;
                x.w += z.w;
            }
            const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j4 * 4 + e < p.N) put_gate(grow, j4 * 4 + e, v[e]);
        }
        return;
    }
    const int lane = threadIdx.x & 7, w = threadIdx.x >> 3, groups = blockDim.x >> 3;
    const int64_t j4 = static_cast<int64_t>(blockIdx.x) * 8 + lane;
    pdl_wait();
    for (int64_t item = blockIdx.y;; item += gridDim.y) {
        const int64_t grow = item - 2;
        if (item >= 2 && (flat || !p.gate || p.gate_rows == 1 || grow * p.gate_rows >= p.M)) return;
        int64_t b0 = 0, b1 = G;
        int area = static_cast<int>(item), area0 = area;
        if (item < 2) {
            if (!(item == 0 ? p.dw_post : p.dw_pre)) continue;
        } else {
            const int64_t first = grow * p.gate_rows;
            const int64_t last = first + p.gate_rows < p.M ? first + p.gate_rows : p.M;
            b0 = range_owner(first, R, p.M);
            b1 = range_owner(last - 1, R, p.M) + 1;
            if (b1 - b0 == 1) continue;  // finished by the range itself
            area = 2;
            area0 = range_begin(b0, R, p.M) < first ? 3 : 2;
        }
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j4 * 4 < p.N) {
            auto at = [&](int64_t b) {
                return reinterpret_cast<const float4*>(
                    partial(p.ws, b == b0 ? area0 : area, b, slots, pitch))[j4];
            };
            auto add = [&](const float4& z) {
                x.x += z.x;
                x.y += z.y;
                x.z += z.z;
                x.w += z.w;
            };
            int64_t b = b0 + w;
            while (b < b1) {
                float4 z[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    z[k] = b + groups * k < b1 ? at(b + groups * k) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 8; ++k) add(z[k]);
                b += groups * 8;
            }
        }
#pragma unroll
        for (int off = 8; off < 32; off <<= 1) {
            x.x += __shfl_xor_sync(0xffffffffu, x.x, off);
            x.y += __shfl_xor_sync(0xffffffffu, x.y, off);
            x.z += __shfl_xor_sync(0xffffffffu, x.z, off);
            x.w += __shfl_xor_sync(0xffffffffu, x.w, off);
        }
        __syncthreads();
        if ((threadIdx.x & 31) < 8) red[threadIdx.x >> 5][lane] = x;
        __syncthreads();
        if (threadIdx.x < 32) {
            float s = 0.f;
#pragma unroll 4
            for (int k = 0; k < groups / 4; ++k) s += reinterpret_cast<const float*>(&red[k][0])[threadIdx.x];
            const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x;
            if (j < p.N) {
                if (item < 2) {
                    (item == 0 ? p.dw_post : p.dw_pre)[j] = s;
                } else {
                    put_gate(grow, j, s);
                }
            }
        }
    }
}

template <int DT>
cudaError_t finish(const BlockBwdP& p, const OpCfg& c, int64_t slots, int64_t G, int64_t R) {
    const int64_t grows = p.gate && p.gate_rows > 1 ? (p.M + p.gate_rows - 1) / p.gate_rows : 0;
    if (!p.dw_post && !p.dw_pre && grows == 0) return cudaSuccess;
    Launch l;
    l.grid = static_cast<int>((p.N + 31) / 32);
    // Gate rows in eight ranges or fewer each go with the borders (GB300, us, the whole
    // backward: 4096x4096 bf16 with a gate row per 3 rows 157 -> 51, 8231x272 fp32 with
    // one per 2 rows 56 -> 24).
    const bool flat = grows * 8 >= R;
    const int64_t most = grows && !flat ? std::max(G, R) : G;  // partial rows of a sum
    l.threads = most <= 128 ? 128 : most <= 256 ? 256 : 512;
    LaunchCfg cfg(l, c.stream, c.pdl);
    const int64_t borders = ((R - 1) * ((p.N + 3) / 4) + l.threads - 1) / l.threads;  // CTAs of them
    const int64_t gates = flat && grows ? (borders + l.grid - 1) / l.grid : grows;
    cfg.cfg.gridDim.y = static_cast<unsigned>(std::min<int64_t>(2 + gates, 1024));
    return cudaLaunchKernelEx(&cfg.cfg, block_bwd_finish_kernel<DT>, p, slots, G, R, flat && grows > 0);
}

template <int DT, int GATE>
cudaError_t launch_ring(const BlockBwdP& in, const OpCfg& c, bool* taken) {
    constexpr int E = VecElems<DT>::value, V = 8 / E;  // eight columns per thread
    using Fn = void (*)(const BlockBwdP, const RingShape);
    const int64_t nvec = in.N / E;
    *taken = false;
    int cluster = 1;
    while (cluster <= 8 && nvec > 512 * V * cluster) cluster *= 2;
    if (cluster > 8) return cudaSuccess;
    const int slice = static_cast<int>((nvec + cluster - 1) / cluster);
    const int T = (slice + V * 32 - 1) / (V * 32) * 32;
    const bool full = in.w_pre && in.ds && nvec == static_cast<int64_t>(V) * T * cluster;
    const int parts = full && in.w_post ? kAll : full && GATE == 0 ? kPreOnly : kAny;
    constexpr int PRE = GATE == 0 ? kPreOnly : kAny;
    const Fn fn = cluster > 1 ? (parts == kAll   ? block_bwd_ring_kernel<DT, GATE, kAll, true>
                                 : parts == kAny ? block_bwd_ring_kernel<DT, GATE, kAny, true>
                                                 : block_bwd_ring_kernel<DT, GATE, PRE, true>)
                              : (parts == kAll   ? block_bwd_ring_kernel<DT, GATE, kAll, false>
                                 : parts == kAny ? block_bwd_ring_kernel<DT, GATE, kAny, false>
                                                 : block_bwd_ring_kernel<DT, GATE, PRE, false>);
    const int arrays = (in.w_post || GATE ? 1 : 0) + (in.w_pre ? 2 : 0) + (in.ds ? 1 : 0) + (GATE == 2 ? 1 : 0);
    const int64_t slots = block_bwd_max_grid(in.M, in.N, c.dev.sm_count);
    RingPlan plan;
    const int extra = GATE == 1 ? V * E * 4 : 0;
    // 128 KB of stages per SM (GB300, us: 16384x4096 bf16 at 64 / 96 / 128 / 192
    // KB 147 / 130 / 129 / 132, 65536x512 91 / 87 / 88 / 88).
    if (!ring_plan(reinterpret_cast<const void*>(fn), c, in.M, slice, T, 512, arrays, extra, 128 << 10, cluster,
                   slots, &plan))
        return cudaSuccess;
    // The teams' sums meet in the rings' memory: with a row per team it may be
    // smaller than they are.
    plan.shape.sums_at = std::max(plan.smem - extra * plan.threads, plan.threads * V * E * 4);
    plan.smem = plan.shape.sums_at + extra * plan.threads;
    plan.shape.slots = slots;
    plan.shape.nvec = static_cast<int>(nvec);
    const int64_t groups = plan.grid / cluster, ranges = groups * plan.shape.teams;
    // A gate row in more than a thousand ranges costs the second launch more than short
    // rows of few gain here: a range is a warp's, in the kernel below a CTA's (GB300, us,
    // here / there, bf16, one gate row for all: 4096x64 14.6 / 11.0, 8231x128 17.1 / 14.3,
    // 32768x16 28.5 / 26.1; 65536x64 44.6 / 49.8, 8231x256 15.9 / 18.4; 8231x128 with one
    // per 100 rows 12.6 / 14.5, without 10.3 / 12.8).
    if (GATE == 1 && c.variant == RMSNORM_VARIANT_AUTO && in.N <= 128 && in.M < 12 * ranges &&
        ranges > 1024 * ((in.M + in.gate_rows - 1) / in.gate_rows))
        return cudaSuccess;
    BlockBwdP p = in;
    p.ldh /= E;
    p.lds /= E;
    p.ldg /= E;
    p.lddy /= E;
    p.ldds /= E;
    p.lddh /= E;
    p.lddr /= E;
    p.lddg /= E;
    *taken = true;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    if (c.pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    cfg.gridDim = dim3(static_cast<unsigned>(plan.grid));
    cfg.blockDim = dim3(static_cast<unsigned>(plan.threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(plan.smem);
    cfg.stream = c.stream;
    cfg.attrs = attr;
    cfg.numAttrs = n;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p, plan.shape);
    return e != cudaSuccess ? e : finish<DT>(in, c, slots, groups, ranges);
}

bool vectors(const BlockBwdP& p) {
    const int64_t e = vec_elems(p.dtype);
    const void* ptrs[] = {p.h, p.s, p.w_post, p.gate, p.w_pre, p.dy, p.ds, p.dh, p.dr, p.dgate};
    for (const void* q : ptrs)
        if (!aligned16(q)) return false;
    const int64_t sizes[] = {p.N, p.ldh, p.w_pre ? p.lds : 0, p.gate ? p.ldg : 0, p.dy ? p.lddy : 0,
                             p.ds ? p.ldds : 0, p.lddh, p.lddr, p.gate ? p.lddg : 0};
    for (int64_t n : sizes)
        if (n % e != 0) return false;
    return true;
}

template <int DT>
cudaError_t run(const BlockBwdP& p, const OpCfg& c) {
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
    auto fn = block_bwd_generic_kernel<DT>;
    const int occ = occupancy(reinterpret_cast<const void*>(fn), T, 0);
    const int64_t slots = block_bwd_max_grid(p.M, p.N, c.dev.sm_count);
    const int64_t G = std::min<int64_t>(
        slots, persistent_grid(p.M, 1, c.dev.sm_count, std::min(occ, kCtasPerSM), c.max_ctas));
    const cudaError_t e = op_launch(c, fn, G, T, 0, p, slots);
    return e != cudaSuccess ? e : finish<DT>(p, c, slots, G, G);
}

}  // namespace

int block_bwd_max_grid(int64_t M, int64_t N, int sm_count) {
    // Up to eight ranges per SM, or 24 of short rows, where a team is a warp; for very
    // long rows fewer, so that the partial rows stay within about 256 MB.
    const int64_t rows = (int64_t(1) << 28) / (kBlockBwdRows * 4 * block_bwd_pitch(N));
    const int64_t per_sm = N <= kShortRow ? 24 : kCtasPerSM;
    const int64_t g = std::min<int64_t>(M, std::min<int64_t>(per_sm * sm_count, std::max<int64_t>(rows, 1)));
    return static_cast<int>(std::max<int64_t>(g, 1));
}

cudaError_t block_bwd_run(const BlockBwdP& p, const OpCfg& c) {
    g_launched.store(true);
    switch (p.dtype) {
        case kBF16: return run<kBF16>(p, c);
        case kFP16: return run<kFP16>(p, c);
        default: return run<kFP32>(p, c);
    }
}

cudaError_t block_bwd_status_read_and_clear(unsigned int* value) {
    return symbol_read_and_clear(g_block_bwd_status, g_launched, value);
}

}  // namespace rmsn
