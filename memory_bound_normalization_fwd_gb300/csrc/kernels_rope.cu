// Rotary positions on the heads of q and k after each head's RMSNorm, and the
// backward of the two (the operation is stated in include/rmsnorm.h).
//
// Angles. A frequency is held as the fraction of a turn per position times
// 2^64, so position * step modulo 2^64 is the phase, exact for any position:
// its top 32 bits as a signed number are the angle in half turns times 2^31,
// and sincospif of that needs no range reduction. The phase is off by 2^-32
// turns and its fp32 value by 2^-25 half turns.
#include "rmsnorm.h"

#include "ops.h"
#include "ops_common.cuh"

#include <algorithm>
#include <map>
#include <mutex>
#include <utility>

namespace rmsn {
namespace {

// cos and sin (times magnitude) of pair i at a position.
__device__ __forceinline__ float2 turn(int64_t position, uint64_t step, float magnitude) {
    const uint64_t phase = static_cast<uint64_t>(position) * step;
    const float x = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
    float s, c;
    sincospif(x, &s, &c);
    return make_float2(c * magnitude, s * magnitude);
}

__device__ __forceinline__ int64_t position_of(const RopeP& p, int64_t b, int64_t s) {
    return p.positions ? p.positions[b * p.positions_stride + s] : s;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Vector kernels. A head is nv = head_dim / E vectors of 16 bytes; a lane takes two
// of them, so that both values of every pair are in one thread: vectors i and
// i + R/(2E) of the rotated part in the half layout, 2i and 2i + 1 when interleaved
// and behind R. L lanes (a power of two, 1..32) make a head; the row sum of a
// head's norm is a butterfly over them.
//
// The cos and sin of a token serve all of its heads, so a CTA takes whole tokens
// of one tensor (a tile), makes their tables in shared memory once, and walks the
// tile's heads, whose vectors it copies into shared memory a few steps ahead.
// Bound by HBM: one read and one write of every head (backward with the norm:
// two reads).
//
// Tables: cos and sin of pair i of a tile's token at [token][0][i] and [token][1][i].
// The arithmetic is on pairs of values (f32x2).
struct RopeTile {
    int L;           // lanes per head
    int log2L;
    int nv;          // vectors per head
    int pairs;       // vectors per half of the rotated part (half layout: R / (2E))
    int tokens[2];   // tokens per tile, q and k
    int64_t tiles[2];
    int64_t ctas[2]; // CTAs of q, of k
    float inv_d;     // 1 / head_dim
};

// The two vectors of lane l: a in [0, nv), b in [0, nv) or past it (none).
__device__ __forceinline__ void lane_vectors(const RopeTile& g, bool interleaved, int l, int& a, int& b) {
    if (interleaved || l >= g.pairs) {
        a = 2 * l;  // behind the rotated part 2 pairs is even, so 2l starts there
        b = a + 1;
    } else {
        a = l;
        b = l + g.pairs;
    }
}

// Turns a lane's values by SIGN * angle, on tables `cs` (cos) and `sn` (sin) of the
// token. Half layout: x and z hold the first and the second values of the same
// pairs. Interleaved: a pair is one f2 of x or z.
template <int DT, bool INTER, int SIGN>
__device__ __forceinline__ void turn_lane(const RopeTile& g, const float* cs, const float* sn, int l, f2* x, f2* z,
                                          int R) {
    constexpr int E = VecElems<DT>::value, H = E / 2;
    if (!INTER) {
        if (l < g.pairs) {
#pragma unroll
            for (int i = 0; i < H; i += 2) {
                const float4 c4 = *reinterpret_cast<const float4*>(cs + l * E + 2 * i);
                const float4 s4 = *reinterpret_cast<const float4*>(sn + l * E + 2 * i);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const f2 c = k == 0 ? f2_make(c4.x, c4.y) : f2_make(c4.z, c4.w);
                    const float s0 = k == 0 ? s4.x : s4.z, s1 = k == 0 ? s4.y : s4.w;
                    const f2 ps = f2_make(s0, s1), ns = f2_make(-s0, -s1);
                    const f2 a = x[i + k], b = z[i + k];
                    x[i + k] = f2_fma(b, SIGN > 0 ? ns : ps, f2_mul(a, c));
                    z[i + k] = f2_fma(a, SIGN > 0 ? ps : ns, f2_mul(b, c));
                }
            }
        }
    } else {
        // pairs of vector 2l: l E + i; of vector 2l + 1: E / 2 further
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            f2* y = k == 0 ? x : z;
            const int first = (2 * l + k) * H;
            if (first < R / 2) {  // the rotated part may end inside the vector
#pragma unroll
                for (int i = 0; i < H; i += 2) {
                    const float2 c2 = *reinterpret_cast<const float2*>(cs + first + i);
                    const float2 s2 = *reinterpret_cast<const float2*>(sn + first + i);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        if (first + i + q >= R / 2) continue;
                        const float c = q == 0 ? c2.x : c2.y, s = SIGN * (q == 0 ? s2.x : s2.y);
                        const float2 v = f2_get(y[i + q]);
                        y[i + q] = f2_make(fmaf(v.x, c, -v.y * s), fmaf(v.y, c, v.x * s));
                    }
                }
            }
        }
    }
}

__device__ __forceinline__ float lanes_sum(float v, int L) {
    for (int off = L >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// cos and sin of the tile's tokens into shared memory, `pad` entries of each per
// token (those past the rotated part are read with whole vectors, not used).
__device__ __forceinline__ void make_tables(const RopeP& p, int64_t tok0, int n, int pad, float* table) {
    const int half = p.R / 2;
    for (int i = threadIdx.x; i < n * pad; i += 256) {
        const int tk = i / pad, j = i - tk * pad;
        float2 cs = make_float2(0.f, 0.f);
        if (j < half) {
            const int64_t tkn = tok0 + tk;
            const int64_t b = p.batch == 1 ? 0 : tkn / p.seq;
            cs = turn(position_of(p, b, tkn - b * p.seq), __ldg(p.steps + j), p.magnitude);
        }
        table[2 * tk * pad + j] = cs.x;
        table[(2 * tk + 1) * pad + j] = cs.y;
    }
}

// Asynchronous copies into shared memory that the copying thread alone reads
// back (cp.async: any stride, no registers, no barrier).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A team's way through the CTA's tiles: in step s of a tile it takes unit
// s * teams + team (unit = token of the tile * heads + head), without divisions.
struct Walk {
    int64_t tile, tok0;
    int n;          // tokens of the tile; 0: past the last tile
    int step, steps;
    int tok, h;     // this step's token of the tile and head; none where tok >= n

    __device__ __forceinline__ void enter(const RopeTile& g, int which, int64_t tokens, int team, int teams,
                                          int heads) {
        tok0 = tile * g.tokens[which];
        n = tile < g.tiles[which] ? static_cast<int>(min(static_cast<int64_t>(g.tokens[which]), tokens - tok0)) : 0;
        steps = (n * heads + teams - 1) / teams;
        step = 0;
        tok = 0;
        h = team;
        while (h >= heads) {
            h -= heads;
            ++tok;
        }
    }
    __device__ __forceinline__ void advance(const RopeTile& g, int which, int64_t tokens, int team, int teams,
                                            int heads) {
        if (++step == steps) {
            tile += g.ctas[which];
            enter(g, which, tokens, team, teams, heads);
            return;
        }
        h += teams;
        while (h >= heads) {
            h -= heads;
            ++tok;
        }
    }
    __device__ __forceinline__ bool live() const { return tok < n; }
    // Offset of the step's head.
    __device__ __forceinline__ int64_t at(const RopeP& p, const HeadsP& x) const {
        const int64_t tkn = tok0 + tok;
        if (p.batch == 1) return tkn * x.st + h * x.sh;
        const int64_t b = tkn / p.seq;
        return b * x.sb + (tkn - b * p.seq) * x.st + h * x.sh;
    }
};

constexpr int kSteps = 3;  // steps of a thread's copies in flight

// Shared memory of a CTA: the tables, then [kSteps][vectors][256] 16-byte slots and
// (backward with the norm) [kSteps][256] floats.
__host__ __device__ constexpr int tile_slots(int vectors) { return kSteps * vectors * 256 * 16; }

// Forward over tiles.
template <int DT, bool INTER, bool NORM>
__global__ void __launch_bounds__(256) rope_fwd_tile_kernel(const RopeP p, const RopeTile g, int pad, int table_bytes) {
    constexpr int E = VecElems<DT>::value, H = E / 2;
    extern __shared__ __align__(16) unsigned char smem[];
    float* table = reinterpret_cast<float*>(smem);
    const int which = blockIdx.x >= g.ctas[0];
    const RopeSeg& sg = p.seg[which];
    const int heads = sg.heads;
    const int l = threadIdx.x & (g.L - 1);
    const int team = threadIdx.x >> g.log2L, teams = 256 >> g.log2L;
    int va, vb;
    lane_vectors(g, INTER, l, va, vb);
    const bool has_a = va < g.nv, has_b = vb < g.nv;
    const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
    const bool norm = NORM && sg.w;
    const int64_t tokens = p.batch * p.seq;
    const uint4* in = static_cast<const uint4*>(sg.in.p) + va;
    uint4* out = static_cast<uint4*>(sg.out.p) + va;
    const int vd = vb - va;
    unsigned char* slots = smem + table_bytes + threadIdx.x * 16;
    for (int k = 0; k < 2 * kSteps; ++k) *reinterpret_cast<uint4*>(slots + k * 4096) = zero4;
    const uint32_t slot0 = static_cast<uint32_t>(__cvta_generic_to_shared(slots));
    Walk ahead;
    ahead.tile = blockIdx.x - (which ? g.ctas[0] : 0);
    ahead.enter(g, which, tokens, team, teams, heads);
    Walk at = ahead;
    int put = 0, take = 0;
    auto fetch = [&]() {
        if (ahead.n > 0) {
            if (ahead.live()) {
                const uint4* x = in + ahead.at(p, sg.in);
                if (has_a) copy16(slot0 + (2 * put) * 4096, x);
                if (has_b) copy16(slot0 + (2 * put + 1) * 4096, x + vd);
            }
            ahead.advance(g, which, tokens, team, teams, heads);
        }
        copies_commit();
        put = put + 1 == kSteps ? 0 : put + 1;
    };
    pdl_wait();
    pdl_launch_dependents();
#pragma unroll
    for (int k = 0; k < kSteps; ++k) fetch();
    f2 wa[H], wb[H];
    if (norm) {
        const uint4* w = static_cast<const uint4*>(sg.w);
        weights2<DT>(has_a ? __ldg(w + va) : zero4, p.offset, wa);
        weights2<DT>(has_b ? __ldg(w + vb) : zero4, p.offset, wb);
    }
    while (at.n > 0) {
        if (at.step == 0) {  // a new tile
            __syncthreads();  // the tables of the tile before are read
            make_tables(p, at.tok0, at.n, pad, table);
            __syncthreads();
        }
        copies_wait<kSteps - 1>();
        f2 x[H], z[H];
        unpack2<DT>(*reinterpret_cast<const uint4*>(slots + (2 * take) * 4096), x);
        unpack2<DT>(*reinterpret_cast<const uint4*>(slots + (2 * take + 1) * 4096), z);
        take = take + 1 == kSteps ? 0 : take + 1;
        fetch();
        const bool live = at.live();
        if (norm) {
            f2 sq = 0;
#pragma unroll
            for (int e = 0; e < H; ++e) sq = f2_fma(x[e], x[e], sq);
#pragma unroll
            for (int e = 0; e < H; ++e) sq = f2_fma(z[e], z[e], sq);
            const float ss = lanes_sum(f2_sum(sq), g.L);
            const float r = rsqrtf(fmaf(ss, g.inv_d, p.eps));
            if (l == 0 && sg.rstd && live) sg.rstd[(at.tok0 + at.tok) * heads + at.h] = r;
            const f2 r2 = f2_dup(r);
#pragma unroll
            for (int e = 0; e < H; ++e) {
                x[e] = f2_mul(f2_mul(x[e], r2), wa[e]);
                z[e] = f2_mul(f2_mul(z[e], r2), wb[e]);
            }
        }
        if (live) {
            const float* cs = table + 2 * at.tok * pad;
            turn_lane<DT, INTER, 1>(g, cs, cs + pad, l, x, z, p.R);
            uint4* y = out + at.at(p, sg.out);
            if (has_a) st_stream(y, pack2<DT>(x));
            if (has_b) st_stream(y + vd, pack2<DT>(z));
        }
        at.advance(g, which, tokens, team, teams, heads);
    }
    copies_wait<0>();
}

// Backward over tiles: turned back, then the norm's backward, with the weights'
// gradients of a lane's columns summed in registers over all the heads it sees,
// and over the CTA's teams (in order) into one partial row.
template <int DT, bool INTER, bool NORM>
__global__ void __launch_bounds__(256) rope_bwd_tile_kernel(const RopeP p, const RopeTile g, int pad, int table_bytes) {
    constexpr int E = VecElems<DT>::value, H = E / 2, NV = NORM ? 4 : 2;
    extern __shared__ __align__(16) unsigned char smem[];
    float* table = reinterpret_cast<float*>(smem);
    const int which = blockIdx.x >= g.ctas[0];
    const RopeSeg& sg = p.seg[which];
    const int heads = sg.heads;
    const int l = threadIdx.x & (g.L - 1);
    const int team = threadIdx.x >> g.log2L, teams = 256 >> g.log2L;
    int va, vb;
    lane_vectors(g, INTER, l, va, vb);
    const bool has_a = va < g.nv, has_b = vb < g.nv;
    const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
    const bool norm = NORM && sg.w;
    const int64_t tokens = p.batch * p.seq;
    const uint4* in = static_cast<const uint4*>(sg.in.p) + va;
    const uint4* xin = static_cast<const uint4*>(sg.x.p) + va;
    uint4* out = static_cast<uint4*>(sg.out.p) + va;
    const int vd = vb - va;
    unsigned char* slots = smem + table_bytes + threadIdx.x * 16;
    for (int k = 0; k < NV * kSteps; ++k) *reinterpret_cast<uint4*>(slots + k * 4096) = zero4;
    float* rs = reinterpret_cast<float*>(smem + table_bytes + tile_slots(NV)) + threadIdx.x;
    const uint32_t slot0 = static_cast<uint32_t>(__cvta_generic_to_shared(slots));
    const uint32_t rs0 = static_cast<uint32_t>(__cvta_generic_to_shared(rs));
    const int64_t cta = blockIdx.x - (which ? g.ctas[0] : 0);
    Walk ahead;
    ahead.tile = cta;
    ahead.enter(g, which, tokens, team, teams, heads);
    Walk at = ahead;
    int put = 0, take = 0;
    auto fetch = [&]() {
        if (ahead.n > 0) {
            if (ahead.live()) {
                const uint4* d = in + ahead.at(p, sg.in);
                if (has_a) copy16(slot0 + (NV * put) * 4096, d);
                if (has_b) copy16(slot0 + (NV * put + 1) * 4096, d + vd);
                if (norm) {
                    const uint4* x = xin + ahead.at(p, sg.x);
                    if (has_a) copy16(slot0 + (NV * put + 2) * 4096, x);
                    if (has_b) copy16(slot0 + (NV * put + 3) * 4096, x + vd);
                    copy4(rs0 + put * 1024, sg.rstd + (ahead.tok0 + ahead.tok) * heads + ahead.h);
                }
            }
            ahead.advance(g, which, tokens, team, teams, heads);
        }
        copies_commit();
        put = put + 1 == kSteps ? 0 : put + 1;
    };
    pdl_wait();
#pragma unroll
    for (int k = 0; k < kSteps; ++k) fetch();
    f2 wa[H], wb[H], da[H], db[H];
#pragma unroll
    for (int e = 0; e < H; ++e) da[e] = db[e] = 0;
    if (norm) {
        const uint4* w = static_cast<const uint4*>(sg.w);
        weights2<DT>(has_a ? __ldg(w + va) : zero4, p.offset, wa);
        weights2<DT>(has_b ? __ldg(w + vb) : zero4, p.offset, wb);
    }
    while (at.n > 0) {
        if (at.step == 0) {  // a new tile
            __syncthreads();  // the tables of the tile before are read
            make_tables(p, at.tok0, at.n, pad, table);
            __syncthreads();
        }
        copies_wait<kSteps - 1>();
        f2 ta[H], tb[H];
        uint4 xa = zero4, xb = zero4;
        unpack2<DT>(*reinterpret_cast<const uint4*>(slots + (NV * take) * 4096), ta);
        unpack2<DT>(*reinterpret_cast<const uint4*>(slots + (NV * take + 1) * 4096), tb);
        float r = 0.f;
        if (norm) {
            xa = *reinterpret_cast<const uint4*>(slots + (NV * take + 2) * 4096);
            xb = *reinterpret_cast<const uint4*>(slots + (NV * take + 3) * 4096);
            r = rs[take * 256];
        }
        take = take + 1 == kSteps ? 0 : take + 1;
        fetch();
        const bool live = at.live();
        const float* cs = table + 2 * (live ? at.tok : 0) * pad;
        turn_lane<DT, INTER, -1>(g, cs, cs + pad, l, ta, tb, p.R);
        if (norm) {
            f2 x[H], z[H], c2 = 0;
            unpack2<DT>(xa, x);
            unpack2<DT>(xb, z);
            const f2 r2 = f2_dup(r);
            if (live) {  // past the tile's last unit a slot holds an older one's values
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    const f2 gx = f2_mul(ta[e], x[e]), gz = f2_mul(tb[e], z[e]);
                    da[e] = f2_fma(gx, r2, da[e]);
                    db[e] = f2_fma(gz, r2, db[e]);
                    c2 = f2_fma(gx, wa[e], c2);
                    c2 = f2_fma(gz, wb[e], c2);
                }
            }
            const float c = lanes_sum(f2_sum(c2), g.L);
            const f2 mf = f2_dup(-(r * r * r * (c * g.inv_d)));
#pragma unroll
            for (int e = 0; e < H; ++e) {
                ta[e] = f2_fma(f2_mul(ta[e], r2), wa[e], f2_mul(x[e], mf));
                tb[e] = f2_fma(f2_mul(tb[e], r2), wb[e], f2_mul(z[e], mf));
            }
        }
        if (live) {
            uint4* y = out + at.at(p, sg.out);
            if (has_a) st_stream(y, pack2<DT>(ta));
            if (has_b) st_stream(y + vd, pack2<DT>(tb));
        }
        at.advance(g, which, tokens, team, teams, heads);
    }
    copies_wait<0>();
    pdl_launch_dependents();
    if (!norm) return;
    // A warp's teams meet by shuffles, the warps in order in shared memory:
    // [8 warps][L lanes][2E].
    __syncthreads();  // the tables are read
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < H; ++e) {
        float2 a = f2_get(da[e]), b = f2_get(db[e]);
        for (int off = g.L; off < 32; off <<= 1) {
            a.x += __shfl_xor_sync(0xffffffffu, a.x, off);
            a.y += __shfl_xor_sync(0xffffffffu, a.y, off);
            b.x += __shfl_xor_sync(0xffffffffu, b.x, off);
            b.y += __shfl_xor_sync(0xffffffffu, b.y, off);
        }
        if (lane < g.L) {
            float2* part = reinterpret_cast<float2*>(table) + (w * g.L + lane) * E;
            part[e] = a;
            part[H + e] = b;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < g.L * 2 * E; i += 256) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += table[k * g.L * 2 * E + i];
        int a, b;
        lane_vectors(g, INTER, i / (2 * E), a, b);
        const int e = i % (2 * E);
        const int j = e < E ? a * E + e : b * E + e - E;
        if (j < p.D) p.ws[(which ? g.ctas[0] + cta : cta) * p.D + j] = t;
    }
}

// Element-wise kernels: any head size, alignment and stride; one warp per head
// of a token (head index over q's and then k's heads). A lane owns the pairs
// lane, lane + 32, ... and the values behind rotary_dim in the same way, reads
// both values of a pair before it writes them, and no lane reads another's, so
// the outputs may lie on the inputs.
struct Unit {
    int seg;
    int64_t b, s, h, token;
};

__device__ __forceinline__ Unit unit_of(const RopeP& p, int64_t u) {
    const int H = p.seg[0].heads + p.seg[1].heads;
    Unit o;
    o.token = u / H;
    o.h = u - o.token * H;
    o.seg = o.h >= p.seg[0].heads;
    if (o.seg) o.h -= p.seg[0].heads;
    o.b = o.token / p.seq;
    o.s = o.token - o.b * p.seq;
    return o;
}

__device__ __forceinline__ int64_t at(const HeadsP& h, const Unit& u) {
    return u.b * h.sb + u.s * h.st + u.h * h.sh;
}

template <int DT>
__global__ void __launch_bounds__(256) rope_fwd_generic_kernel(const RopeP p) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
    const int64_t units = p.batch * p.seq * (p.seg[0].heads + p.seg[1].heads);
    const int half = p.R / 2;
    pdl_wait();
    pdl_launch_dependents();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < units; i += warps) {
        const Unit u = unit_of(p, i);
        const RopeSeg& g = p.seg[u.seg];
        const int64_t x0 = at(g.in, u), y0 = at(g.out, u);
        float r = 1.f;
        if (g.w) {
            float ss = 0.f;
            for (int j = lane; j < p.D; j += 32) {
                const float f = load1<DT>(g.in.p, x0 + j);
                ss = fmaf(f, f, ss);
            }
            r = row_rstd(warp_sum(ss), static_cast<float>(p.D), p.eps);
            if (lane == 0 && g.rstd) g.rstd[u.token * g.heads + u.h] = r;
        }
        auto x = [&](int j) {
            const float f = load1<DT>(g.in.p, x0 + j);
            return g.w ? f * r * (p.offset + load1<DT>(g.w, j)) : f;
        };
        const int64_t pos = position_of(p, u.b, u.s);
        __syncwarp();  // every lane's reads for the sum before the first write
        for (int j = lane; j < half; j += 32) {
            const float2 cs = turn(pos, p.steps[j], p.magnitude);
            const int a = p.interleaved ? 2 * j : j, b = p.interleaved ? 2 * j + 1 : j + half;
            const float xa = x(a), xb = x(b);
            store1<DT>(g.out.p, y0 + a, fmaf(xa, cs.x, -xb * cs.y));
            store1<DT>(g.out.p, y0 + b, fmaf(xb, cs.x, xa * cs.y));
        }
        for (int j = p.R + lane; j < p.D; j += 32) store1<DT>(g.out.p, y0 + j, x(j));
    }
}

// Backward: the gradient turned back, then the norm's backward. A warp keeps
// the weights' gradient sums of the heads it sees in its own two partial rows.
template <int DT>
__global__ void __launch_bounds__(256) rope_bwd_generic_kernel(const RopeP p) {
    const int lane = threadIdx.x & 31;
    const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
    const int64_t me = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t units = p.batch * p.seq * (p.seg[0].heads + p.seg[1].heads);
    const int half = p.R / 2;
    pdl_wait();
    for (int k = 0; k < 2; ++k) {
        if (!p.seg[k].w) continue;
        float* acc = p.ws + (k * warps + me) * p.D;
        for (int j = lane; j < half; j += 32) acc[j] = acc[half + j] = 0.f;
        for (int j = p.R + lane; j < p.D; j += 32) acc[j] = 0.f;
    }
    for (int64_t i = me; i < units; i += warps) {
        const Unit u = unit_of(p, i);
        const RopeSeg& g = p.seg[u.seg];
        const int64_t d0 = at(g.in, u), o0 = at(g.out, u), x0 = at(g.x, u);
        const int64_t pos = position_of(p, u.b, u.s);
        // The gradient of the normed head at pair j (as its two values) and
        // behind rotary_dim.
        auto back = [&](int j) {
            const float2 cs = turn(pos, p.steps[j], p.magnitude);
            const int a = p.interleaved ? 2 * j : j, b = p.interleaved ? 2 * j + 1 : j + half;
            const float da = load1<DT>(g.in.p, d0 + a), db = load1<DT>(g.in.p, d0 + b);
            return make_float2(fmaf(da, cs.x, db * cs.y), fmaf(db, cs.x, -da * cs.y));
        };
        float r = 1.f, f = 0.f;
        if (g.w) {
            r = g.rstd[u.token * g.heads + u.h];
            float c = 0.f;
            for (int j = lane; j < half; j += 32) {
                const int a = p.interleaved ? 2 * j : j, b = p.interleaved ? 2 * j + 1 : j + half;
                const float2 d = back(j);
                c = fmaf(d.x * (p.offset + load1<DT>(g.w, a)), load1<DT>(g.x.p, x0 + a), c);
                c = fmaf(d.y * (p.offset + load1<DT>(g.w, b)), load1<DT>(g.x.p, x0 + b), c);
            }
            for (int j = p.R + lane; j < p.D; j += 32)
                c = fmaf(load1<DT>(g.in.p, d0 + j) * (p.offset + load1<DT>(g.w, j)),
                         load1<DT>(g.x.p, x0 + j), c);
            f = r * r * (warp_sum(c) / static_cast<float>(p.D));
        }
        float* acc = p.ws + (u.seg * warps + me) * p.D;
        auto put = [&](int j, int slot, float d) {
            if (g.w) {
                const float x = load1<DT>(g.x.p, x0 + j);
                acc[slot] = fmaf(d, x * r, acc[slot]);
                d = r * fmaf(d, p.offset + load1<DT>(g.w, j), -x * f);
            }
            store1<DT>(g.out.p, o0 + j, d);
        };
        for (int j = lane; j < half; j += 32) {
            const float2 d = back(j);
            // sums are kept at j and half + j (this lane's), whatever the layout
            put(p.interleaved ? 2 * j : j, j, d.x);
            put(p.interleaved ? 2 * j + 1 : j + half, half + j, d.y);
        }
        for (int j = p.R + lane; j < p.D; j += 32) put(j, j, load1<DT>(g.in.p, d0 + j));
    }
    pdl_launch_dependents();
}

// dw_q and dw_k: sums of the partial rows in order. blockIdx.y is the tensor, with
// rows[0] rows of q and then rows[1] of k. `paired`: a row holds the first value of
// pair i at i, the second at half + i (the element-wise kernel's); else columns.
struct RopeRows {
    int64_t n[2];
};
__global__ void __launch_bounds__(256) rope_dw_kernel(const RopeP p, RopeRows rows, int paired) {
    __shared__ float part[8][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, half = p.R / 2;
    const int slot = static_cast<int>(blockIdx.x) * 32 + lane;
    pdl_wait();
    if (!p.seg[blockIdx.y].w) return;
    float t = 0.f;
    if (slot < p.D) {
        const float* q = p.ws + (blockIdx.y ? rows.n[0] : 0) * p.D + slot;
        const int64_t n = rows.n[blockIdx.y];
        int64_t i = w;
        for (; i + 24 < n; i += 32) {
            const float a = q[i * p.D], b = q[(i + 8) * p.D], c = q[(i + 16) * p.D], d = q[(i + 24) * p.D];
            t += a;
            t += b;
            t += c;
            t += d;
        }
        for (; i < n; i += 8) t += q[i * p.D];
    }
    part[w][lane] = t;
    __syncthreads();
    if (w == 0 && slot < p.D) {
        t = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += part[k][lane];
        const int j = !paired || !p.interleaved || slot >= p.R ? slot
                      : slot < half ? 2 * slot : 2 * (slot - half) + 1;
        p.seg[blockIdx.y].dw[j] = t;
    }
}

constexpr int kGenericCtasPerSM = 8;

int64_t generic_grid(const RopeP& p, const OpCfg& c) {
    const int64_t units = p.batch * p.seq * (p.seg[0].heads + p.seg[1].heads);
    return persistent_grid(units, 8, c.dev.sm_count, kGenericCtasPerSM, c.max_ctas);
}

// Table entries per token: the rotated pairs, up to whole vectors.
int table_pad(const RopeP& p) { return (p.R / 2 + 3) / 4 * 4; }

// Whether every head is whole 16-byte vectors that the tile kernels can pair up,
// and how: lanes per head, tokens per tile, CTAs.
bool tiles(const RopeP& p, const OpCfg& c, bool bwd, int ctas_per_sm, RopeTile* g) {
    const int E = vec_elems(p.dtype);
    if (p.D % E != 0 || p.D > 64 * E) return false;
    // Half layout: both halves whole vectors. Interleaved: any even rotary_dim.
    if (!p.interleaved && p.R % (2 * E) != 0) return false;
    for (int k = 0; k < 2; ++k) {
        const RopeSeg& s = p.seg[k];
        if (s.heads == 0) continue;
        const HeadsP* hs[] = {&s.in, &s.out, bwd && s.w ? &s.x : nullptr};
        for (const HeadsP* h : hs) {
            if (!h) continue;
            if (!aligned16(h->p) || (p.batch > 1 && h->sb % E) || (p.seq > 1 && h->st % E) ||
                (s.heads > 1 && h->sh % E))
                return false;
        }
        if (!aligned16(s.w)) return false;
    }
    g->nv = p.D / E;
    g->inv_d = 1.f / static_cast<float>(p.D);
    g->pairs = p.interleaved ? 0 : p.R / (2 * E);
    g->L = 1;
    g->log2L = 0;
    while (g->L * 2 < g->nv) {
        g->L <<= 1;
        ++g->log2L;
    }
    const int teams = 256 / g->L;
    const int64_t tokens = p.batch * p.seq;
    int64_t work[2] = {0, 0};
    for (int k = 0; k < 2; ++k) {
        const int64_t heads = p.seg[k].heads;
        g->tokens[k] = 1;
        g->tiles[k] = 0;
        if (heads == 0) continue;
        // A tile is about four steps of the CTA's teams, as far as the tokens reach
        // every SM and their tables 16 KB.
        int64_t n = std::max<int64_t>(1, 4 * teams / heads);
        n = std::min<int64_t>(n, std::max<int64_t>(1, tokens / (2 * c.dev.sm_count)));
        n = std::min<int64_t>(n, std::max<int64_t>(1, 2048 / table_pad(p)));
        g->tokens[k] = static_cast<int>(n);
        g->tiles[k] = (tokens + n - 1) / n;
        work[k] = heads;
    }
    // CTAs in proportion to the heads.
    int64_t cap = static_cast<int64_t>(c.dev.sm_count) * ctas_per_sm;
    if (c.max_ctas > 0) cap = std::min<int64_t>(cap, std::max(c.max_ctas, 2));
    g->ctas[0] = std::min(g->tiles[0], std::max<int64_t>(1, cap * work[0] / (work[0] + work[1])));
    g->ctas[1] = work[1] ? std::min(g->tiles[1], std::max<int64_t>(1, cap - g->ctas[0])) : 0;
    return true;
}

// Shared memory a tile kernel is given for its tables: 16 KB, one token's where
// that is more.
int table_bytes(const RopeP& p) { return std::max(16384, table_pad(p) * 8); }

// Opts a kernel into `smem` bytes on the current device, once; the CTAs per SM.
int tile_occupancy(const void* fn, int smem) {
    static std::mutex mu;
    static std::map<std::pair<int, const void*>, int> done;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    {
        std::lock_guard<std::mutex> guard(mu);
        int& have = done[{dev, fn}];
        if (have < smem) {
            if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return 0;
            have = smem;
        }
    }
    return occupancy(fn, 256, smem);
}

template <int DT, bool INTER, bool NORM>
cudaError_t fwd_tiles(RopeP p, const OpCfg& c, bool* taken) {
    auto fn = rope_fwd_tile_kernel<DT, INTER, NORM>;
    RopeTile g;
    const int tb = table_bytes(p), smem = tb + tile_slots(2);
    const int occ = tile_occupancy(reinterpret_cast<const void*>(fn), smem);
    *taken = occ > 0 && tiles(p, c, false, occ, &g);
    if (!*taken) return cudaSuccess;
    constexpr int E = VecElems<DT>::value;
    for (RopeSeg& s : p.seg)
        for (HeadsP* h : {&s.in, &s.out}) h->sb /= E, h->st /= E, h->sh /= E;
    return op_launch(c, fn, g.ctas[0] + g.ctas[1], 256, smem, p, g, table_pad(p), tb);
}

cudaError_t launch_dw(const RopeP& p, const OpCfg& c, int64_t rows_q, int64_t rows_k, int paired) {
    Launch l;
    l.grid = (p.D + 31) / 32;
    l.threads = 256;
    LaunchCfg cfg(l, c.stream, c.pdl);
    cfg.cfg.gridDim.y = 2;
    return cudaLaunchKernelEx(&cfg.cfg, rope_dw_kernel, p, RopeRows{{rows_q, rows_k}}, paired);
}

template <int DT, bool INTER, bool NORM>
cudaError_t bwd_tiles(RopeP p, const OpCfg& c, bool* taken) {
    auto fn = rope_bwd_tile_kernel<DT, INTER, NORM>;
    RopeTile g;
    constexpr int E = VecElems<DT>::value;
    // The sums of the weights' gradients meet where the tables were (16 KB at most).
    const int tb = table_bytes(p), smem = tb + tile_slots(NORM ? 4 : 2) + (NORM ? kSteps * 1024 : 0);
    const int occ = tile_occupancy(reinterpret_cast<const void*>(fn), smem);
    *taken = occ > 0 && tiles(p, c, true, std::min(8, occ), &g);
    if (!*taken) return cudaSuccess;
    for (RopeSeg& s : p.seg)
        for (HeadsP* h : {&s.in, &s.out, &s.x}) h->sb /= E, h->st /= E, h->sh /= E;
    const cudaError_t e = op_launch(c, fn, g.ctas[0] + g.ctas[1], 256, smem, p, g, table_pad(p), tb);
    return e != cudaSuccess || !NORM ? e : launch_dw(p, c, g.ctas[0], g.ctas[1], 0);
}

template <int DT>
cudaError_t fwd(const RopeP& p, const OpCfg& c) {
    if (c.variant != RMSNORM_VARIANT_GENERIC) {
        bool taken = false;
        const bool norm = p.seg[0].w || p.seg[1].w;
        const cudaError_t e =
            p.interleaved ? (norm ? fwd_tiles<DT, true, true>(p, c, &taken) : fwd_tiles<DT, true, false>(p, c, &taken))
                          : (norm ? fwd_tiles<DT, false, true>(p, c, &taken) : fwd_tiles<DT, false, false>(p, c, &taken));
        if (taken) return e;
    }
    if (c.variant == RMSNORM_VARIANT_CTA) return cudaErrorNotSupported;
    return op_launch(c, rope_fwd_generic_kernel<DT>, generic_grid(p, c), 256, 0, p);
}

template <int DT>
cudaError_t bwd(const RopeP& p, const OpCfg& c) {
    const bool norm = p.seg[0].w || p.seg[1].w;
    if (c.variant != RMSNORM_VARIANT_GENERIC) {
        bool taken = false;
        const cudaError_t e =
            p.interleaved ? (norm ? bwd_tiles<DT, true, true>(p, c, &taken) : bwd_tiles<DT, true, false>(p, c, &taken))
                          : (norm ? bwd_tiles<DT, false, true>(p, c, &taken) : bwd_tiles<DT, false, false>(p, c, &taken));
        if (taken) return e;
    }
    if (c.variant == RMSNORM_VARIANT_CTA) return cudaErrorNotSupported;
    const int64_t G = generic_grid(p, c);
    const cudaError_t e = op_launch(c, rope_bwd_generic_kernel<DT>, G, 256, 0, p);
    return e != cudaSuccess || !norm ? e : launch_dw(p, c, G * 8, G * 8, 1);
}

}  // namespace

int64_t rope_bwd_partial_rows(int sm_count) {
    return 2LL * sm_count * kGenericCtasPerSM * 8;
}

cudaError_t rope_fwd_run(const RopeP& p, const OpCfg& c) {
    switch (p.dtype) {
        case kBF16: return fwd<kBF16>(p, c);
        case kFP16: return fwd<kFP16>(p, c);
        default: return fwd<kFP32>(p, c);
    }
}

cudaError_t rope_bwd_run(const RopeP& p, const OpCfg& c) {
    switch (p.dtype) {
        case kBF16: return bwd<kBF16>(p, c);
        case kFP16: return bwd<kFP16>(p, c);
        default: return bwd<kFP32>(p, c);
    }
}

}  // namespace rmsn
