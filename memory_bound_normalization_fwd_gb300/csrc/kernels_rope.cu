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
// tile's heads. The first heads' loads are issued before the tables are made.
// Bound by HBM: one read and one write of every head (backward with the norm:
// two reads).
struct RopeTile {
    int L;           // lanes per head
    int log2L;
    int nv;          // vectors per head
    int pairs;       // vectors per half of the rotated part (half layout: R / (2E))
    int tokens[2];   // tokens per tile, q and k
    int64_t tiles[2];
    int64_t ctas[2]; // CTAs of q, of k
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

// Turns the values of a lane by sign * angle. tab: cos and sin of the token's
// pairs (float2 per pair).
template <int DT, bool INTER>
__device__ __forceinline__ void turn_lane(const RopeTile& g, const float2* tab, int l, float sign, float* x,
                                          float* z, int R) {
    constexpr int E = VecElems<DT>::value;
    if (!INTER) {
        if (l < g.pairs) {
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                const float4 c = *reinterpret_cast<const float4*>(tab + l * E + e);
                const float s0 = sign * c.y, s1 = sign * c.w;
                const float a0 = x[e], a1 = x[e + 1], b0 = z[e], b1 = z[e + 1];
                x[e] = fmaf(a0, c.x, -b0 * s0);
                z[e] = fmaf(b0, c.x, a0 * s0);
                x[e + 1] = fmaf(a1, c.z, -b1 * s1);
                z[e + 1] = fmaf(b1, c.z, a1 * s1);
            }
        }
    } else {
        // pairs of vector 2l: (2l E / 2) + i; of vector 2l + 1: E / 2 further
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float* y = k == 0 ? x : z;
            if ((2 * l + k) * E < R) {
                const float2* q = tab + (2 * l + k) * (E / 2);
#pragma unroll
                for (int i = 0; i < E / 2; i += 2) {
                    const float4 c = *reinterpret_cast<const float4*>(q + i);
                    const float s0 = sign * c.y, s1 = sign * c.w;
                    const float a0 = y[2 * i], b0 = y[2 * i + 1], a1 = y[2 * i + 2], b1 = y[2 * i + 3];
                    y[2 * i] = fmaf(a0, c.x, -b0 * s0);
                    y[2 * i + 1] = fmaf(b0, c.x, a0 * s0);
                    y[2 * i + 2] = fmaf(a1, c.z, -b1 * s1);
                    y[2 * i + 3] = fmaf(b1, c.z, a1 * s1);
                }
            }
        }
    }
}

__device__ __forceinline__ float lanes_sum(float v, int L) {
    for (int off = L >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Forward over tiles. UNROLL heads of a thread are in flight at once.
template <int DT, bool INTER, bool NORM, int UNROLL>
__global__ void __launch_bounds__(256) rope_fwd_tile_kernel(const RopeP p, const RopeTile g) {
    constexpr int E = VecElems<DT>::value;
    extern __shared__ __align__(16) float2 table[];
    const int which = blockIdx.x >= g.ctas[0];
    const RopeSeg& sg = p.seg[which];
    const int half = p.R / 2;
    const int l = threadIdx.x & (g.L - 1);
    const int team = threadIdx.x >> g.log2L, teams = 256 >> g.log2L;
    int va, vb;
    lane_vectors(g, INTER, l, va, vb);
    const bool has_a = va < g.nv, has_b = vb < g.nv;
    const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
    pdl_wait();
    pdl_launch_dependents();
    float wa[E], wb[E];
    if (NORM && sg.w) {
        const uint4* w = static_cast<const uint4*>(sg.w);
        weights_vec<DT>(has_a ? __ldg(w + va) : zero4, p.offset, wa);
        weights_vec<DT>(has_b ? __ldg(w + vb) : zero4, p.offset, wb);
    }
    const int64_t tokens = p.batch * p.seq;
    const int64_t cta = blockIdx.x - (which ? g.ctas[0] : 0);
    for (int64_t tile = cta; tile < g.tiles[which]; tile += g.ctas[which]) {
        const int64_t tok0 = tile * g.tokens[which];
        const int n = static_cast<int>(min(static_cast<int64_t>(g.tokens[which]), tokens - tok0));
        const int units = n * sg.heads;
        uint4 xa[UNROLL], xb[UNROLL];
        int64_t out_at[UNROLL], head_at[UNROLL];
        int tok[UNROLL];
        auto fetch = [&](int u0) {
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) {
                const int u = u0 + k * teams;
                xa[k] = xb[k] = zero4;
                if (u < units) {
                    const int tk = u / sg.heads, h = u - tk * sg.heads;
                    const int64_t tkn = tok0 + tk;
                    const int64_t b = p.batch == 1 ? 0 : tkn / p.seq, s = tkn - b * p.seq;
                    const uint4* x = static_cast<const uint4*>(sg.in.p) + b * sg.in.sb + s * sg.in.st + h * sg.in.sh;
                    if (has_a) xa[k] = ld_stream(x + va);
                    if (has_b) xb[k] = ld_stream(x + vb);
                    out_at[k] = b * sg.out.sb + s * sg.out.st + h * sg.out.sh;
                    head_at[k] = tkn * sg.heads + h;
                    tok[k] = tk;
                }
            }
        };
        fetch(team);
        for (int i = threadIdx.x; i < n * half; i += 256) {
            const int tk = i / half, j = i - tk * half;
            const int64_t tkn = tok0 + tk;
            const int64_t b = p.batch == 1 ? 0 : tkn / p.seq;
            table[i] = turn(position_of(p, b, tkn - b * p.seq), __ldg(p.steps + j), p.magnitude);
        }
        __syncthreads();
        for (int u0 = team; u0 - team < units; u0 += UNROLL * teams) {
            if (u0 != team) fetch(u0);
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) {
                float x[E], z[E];
                unpack_vec<DT>(xa[k], x);
                unpack_vec<DT>(xb[k], z);
                if (NORM && sg.w) {
                    float ss = sumsq_vec<DT>(xb[k], sumsq_vec<DT>(xa[k], 0.f));
                    ss = lanes_sum(ss, g.L);
                    const float r = row_rstd(ss, static_cast<float>(p.D), p.eps);
                    if (l == 0 && sg.rstd && u0 + k * teams < units) sg.rstd[head_at[k]] = r;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        x[e] = x[e] * r * wa[e];
                        z[e] = z[e] * r * wb[e];
                    }
                }
                if (u0 + k * teams < units) {
                    turn_lane<DT, INTER>(g, table + tok[k] * half, l, 1.f, x, z, p.R);
                    uint4* y = static_cast<uint4*>(sg.out.p) + out_at[k];
                    if (has_a) st_stream(y + va, pack_vec<DT>(x));
                    if (has_b) st_stream(y + vb, pack_vec<DT>(z));
                }
            }
        }
        __syncthreads();  // the tables are read before the next tile's are made
    }
}

// Backward over tiles: turned back, then the norm's backward, with the weights'
// gradients of a lane's columns summed in registers over all the heads it sees,
// and over the CTA's teams (in order) into one partial row.
template <int DT, bool INTER, bool NORM, int UNROLL>
__global__ void __launch_bounds__(256) rope_bwd_tile_kernel(const RopeP p, const RopeTile g) {
    constexpr int E = VecElems<DT>::value;
    extern __shared__ __align__(16) float2 table[];
    const int which = blockIdx.x >= g.ctas[0];
    const RopeSeg& sg = p.seg[which];
    const int half = p.R / 2;
    const int l = threadIdx.x & (g.L - 1);
    const int team = threadIdx.x >> g.log2L, teams = 256 >> g.log2L;
    int va, vb;
    lane_vectors(g, INTER, l, va, vb);
    const bool has_a = va < g.nv, has_b = vb < g.nv;
    const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
    const bool norm = NORM && sg.w;
    pdl_wait();
    float wa[E], wb[E], da[E], db[E];
#pragma unroll
    for (int e = 0; e < E; ++e) da[e] = db[e] = 0.f;
    if (norm) {
        const uint4* w = static_cast<const uint4*>(sg.w);
        weights_vec<DT>(has_a ? __ldg(w + va) : zero4, p.offset, wa);
        weights_vec<DT>(has_b ? __ldg(w + vb) : zero4, p.offset, wb);
    }
    const float inv_d = 1.f / static_cast<float>(p.D);
    const int64_t tokens = p.batch * p.seq;
    const int64_t cta = blockIdx.x - (which ? g.ctas[0] : 0);
    for (int64_t tile = cta; tile < g.tiles[which]; tile += g.ctas[which]) {
        const int64_t tok0 = tile * g.tokens[which];
        const int n = static_cast<int>(min(static_cast<int64_t>(g.tokens[which]), tokens - tok0));
        const int units = n * sg.heads;
        uint4 ga[UNROLL], gb[UNROLL], xa[UNROLL], xb[UNROLL];
        float rs[UNROLL];
        int64_t out_at[UNROLL];
        int tok[UNROLL];
        auto fetch = [&](int u0) {
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) {
                const int u = u0 + k * teams;
                ga[k] = gb[k] = xa[k] = xb[k] = zero4;
                rs[k] = 0.f;
                tok[k] = 0;
                if (u < units) {
                    const int tk = u / sg.heads, h = u - tk * sg.heads;
                    const int64_t tkn = tok0 + tk;
                    const int64_t b = p.batch == 1 ? 0 : tkn / p.seq, s = tkn - b * p.seq;
                    const uint4* d = static_cast<const uint4*>(sg.in.p) + b * sg.in.sb + s * sg.in.st + h * sg.in.sh;
                    if (has_a) ga[k] = ld_stream(d + va);
                    if (has_b) gb[k] = ld_stream(d + vb);
                    if (norm) {
                        const uint4* x = static_cast<const uint4*>(sg.x.p) + b * sg.x.sb + s * sg.x.st + h * sg.x.sh;
                        if (has_a) xa[k] = ld_stream(x + va);
                        if (has_b) xb[k] = ld_stream(x + vb);
                        rs[k] = __ldg(sg.rstd + tkn * sg.heads + h);
                    }
                    out_at[k] = b * sg.out.sb + s * sg.out.st + h * sg.out.sh;
                    tok[k] = tk;
                }
            }
        };
        fetch(team);
        for (int i = threadIdx.x; i < n * half; i += 256) {
            const int tk = i / half, j = i - tk * half;
            const int64_t tkn = tok0 + tk;
            const int64_t b = p.batch == 1 ? 0 : tkn / p.seq;
            table[i] = turn(position_of(p, b, tkn - b * p.seq), __ldg(p.steps + j), p.magnitude);
        }
        __syncthreads();
        for (int u0 = team; u0 - team < units; u0 += UNROLL * teams) {
            if (u0 != team) fetch(u0);
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) {
                float ta[E], tb[E];
                unpack_vec<DT>(ga[k], ta);
                unpack_vec<DT>(gb[k], tb);
                turn_lane<DT, INTER>(g, table + tok[k] * half, l, -1.f, ta, tb, p.R);
                if (norm) {
                    float x[E], z[E], c = 0.f;
                    unpack_vec<DT>(xa[k], x);
                    unpack_vec<DT>(xb[k], z);
                    const float r = rs[k];
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float gx = ta[e] * x[e], gz = tb[e] * z[e];
                        da[e] = fmaf(gx, r, da[e]);
                        db[e] = fmaf(gz, r, db[e]);
                        c = fmaf(gx, wa[e], c);
                        c = fmaf(gz, wb[e], c);
                    }
                    c = lanes_sum(c, g.L);
                    const float f = r * r * r * (c * inv_d);
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        ta[e] = fmaf(r * ta[e], wa[e], -f * x[e]);
                        tb[e] = fmaf(r * tb[e], wb[e], -f * z[e]);
                    }
                }
                if (u0 + k * teams < units) {
                    uint4* y = static_cast<uint4*>(sg.out.p) + out_at[k];
                    if (has_a) st_stream(y + va, pack_vec<DT>(ta));
                    if (has_b) st_stream(y + vb, pack_vec<DT>(tb));
                }
            }
        }
        __syncthreads();  // the tables are read before the next tile's are made
    }
    pdl_launch_dependents();
    if (!norm) return;
    // A warp's teams meet by shuffles, the warps in order in shared memory:
    // [8 warps][L lanes][2E].
    float* part = reinterpret_cast<float*>(table);
    for (int off = g.L; off < 32; off <<= 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            da[e] += __shfl_xor_sync(0xffffffffu, da[e], off);
            db[e] += __shfl_xor_sync(0xffffffffu, db[e], off);
        }
    }
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane < g.L) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
            part[(w * g.L + lane) * 2 * E + e] = da[e];
            part[(w * g.L + lane) * 2 * E + E + e] = db[e];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < g.L * 2 * E; i += 256) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += part[k * g.L * 2 * E + i];
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

// Whether every head is whole 16-byte vectors that the tile kernels can pair up,
// and how: lanes per head, tokens per tile, CTAs.
bool tiles(const RopeP& p, const OpCfg& c, bool bwd, int ctas_per_sm, RopeTile* g) {
    const int E = vec_elems(p.dtype);
    if (p.D % E != 0 || p.D > 64 * E) return false;
    // Half layout: both halves whole vectors; interleaved: the rotated part is.
    if (p.R % (p.interleaved ? E : 2 * E) != 0) return false;
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
        // A tile fills the CTA's teams about twice, as far as the tokens reach
        // every SM and their tables 16 KB.
        int64_t n = std::max<int64_t>(1, 2 * teams / heads);
        n = std::min<int64_t>(n, std::max<int64_t>(1, tokens * 2 / c.dev.sm_count));
        n = std::min<int64_t>(n, std::max<int64_t>(1, 2048 / (p.R / 2)));
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

template <int DT, bool INTER, bool NORM>
cudaError_t fwd_tiles(RopeP p, const OpCfg& c, bool* taken) {
    auto fn = rope_fwd_tile_kernel<DT, INTER, NORM, 2>;
    RopeTile g;
    const int occ = std::max(1, occupancy(reinterpret_cast<const void*>(fn), 256, 16384));
    *taken = tiles(p, c, false, occ, &g);
    if (!*taken) return cudaSuccess;
    constexpr int E = VecElems<DT>::value;
    for (RopeSeg& s : p.seg)
        for (HeadsP* h : {&s.in, &s.out}) h->sb /= E, h->st /= E, h->sh /= E;
    const int smem = std::max(g.tokens[0], g.tokens[1]) * (p.R / 2) * 8;
    return op_launch(c, fn, g.ctas[0] + g.ctas[1], 256, smem, p, g);
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
    auto fn = rope_bwd_tile_kernel<DT, INTER, NORM, 2>;
    RopeTile g;
    const int occ = std::min(8, std::max(1, occupancy(reinterpret_cast<const void*>(fn), 256, 16384)));
    *taken = tiles(p, c, true, occ, &g);
    if (!*taken) return cudaSuccess;
    constexpr int E = VecElems<DT>::value;
    for (RopeSeg& s : p.seg)
        for (HeadsP* h : {&s.in, &s.out, &s.x}) h->sb /= E, h->st /= E, h->sh /= E;
    const int smem = std::max(std::max(g.tokens[0], g.tokens[1]) * (p.R / 2) * 8,
                              NORM ? 8 * g.L * 2 * E * 4 : 0);
    const cudaError_t e = op_launch(c, fn, g.ctas[0] + g.ctas[1], 256, smem, p, g);
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
