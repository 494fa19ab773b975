// Rotary positions on the heads of q and k after each head's RMSNorm, and the
// backward of the two (the operation is stated in include/rmsnorm.h).
//
// Angles. A frequency is held as the fraction of a turn per position times
// 2^64, so position * step modulo 2^64 is the phase, exact for any position.
// The nearest quarter turn is taken off it in integers, so what becomes an fp32
// value (off by 2^-23 of itself) is at most an eighth of a turn, and cos and sin
// keep all their bits however near to zero they are.
#include "rmsnorm.h"

#include "ops.h"
#include "ops_common.cuh"

#include <algorithm>
#include <map>
#include <mutex>
#include <utility>

namespace rmsn {
namespace {

// cos and sin (times magnitude) of two pairs at their positions: the Taylor series of sin and
// cos of y quarter turns, |y| <= 1/2, to y^9 and y^10 (what is left out is below 2^-28),
// then turned by the quarters. The large term comes last, in one rounding. The same bits
// for every type and kernel. (The hardware's approximations, whose error does not shrink
// with sin, put fp16 outputs off by up to 16 half steps. GB300, us, those / this, bf16
// with norms: 64 tokens of 40 heads of 128 2.68 / 2.69, 16384 tokens 56.5 / 56.6, backward
// 83.1 / 84.2, 16384 of 20 heads of 80 with 20 turned 45.4 / 46.3. sincospif of the same
// rest: 3.05, 58.9, 86.1, 51.2; one angle at a time from a 64-bit conversion: 3.0, 57.9,
// 84.9, 48.2.)
__device__ __forceinline__ void turn2(int64_t position0, int64_t position1, uint64_t step0, uint64_t step1,
                                      float magnitude, f2& c, f2& s) {
    constexpr double q = 1.57079632679489661923;  // a quarter turn
    constexpr double q2 = q * q;
    constexpr float s1 = static_cast<float>(q), s1_rest = static_cast<float>(q - s1);
    constexpr float s3 = static_cast<float>(-q * q2 / 6), s5 = static_cast<float>(q * q2 * q2 / 120);
    constexpr float s7 = static_cast<float>(-q * q2 * q2 * q2 / 5040);
    constexpr float s9 = static_cast<float>(q * q2 * q2 * q2 * q2 / 362880);
    constexpr float c2 = static_cast<float>(-q2 / 2), c4 = static_cast<float>(q2 * q2 / 24);
    constexpr float c6 = static_cast<float>(-q2 * q2 * q2 / 720), c8 = static_cast<float>(q2 * q2 * q2 * q2 / 40320);
    constexpr float c10 = static_cast<float>(-q2 * q2 * q2 * q2 * q2 / 3628800);
    uint32_t quarter[2];  // the nearest quarter in the top two bits
    float hi[2], lo[2];   // what is left, in quarter turns times 2^32 and 2^64
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint64_t phase = static_cast<uint64_t>(k == 0 ? position0 : position1) * (k == 0 ? step0 : step1);
        const uint64_t near = phase + (uint64_t(1) << 29);  // so that lo is signed
        quarter[k] = static_cast<uint32_t>(near >> 32) + 0x20000000u;
        hi[k] = static_cast<float>(static_cast<int32_t>(near >> 30));
        lo[k] = static_cast<float>(static_cast<int32_t>(phase << 2));
    }
    const f2 y = f2_fma(f2_make(lo[0], lo[1]), f2_dup(0x1p-64f), f2_mul(f2_make(hi[0], hi[1]), f2_dup(0x1p-32f)));
    const f2 z = f2_mul(y, y);
    auto series = [&](f2 x, float a) { return f2_fma(z, x, f2_dup(a)); };
    const f2 sn = f2_fma(y, f2_dup(s1), f2_mul(y, series(series(series(series(f2_dup(s9), s7), s5), s3), s1_rest)));
    const f2 cn = series(series(series(series(series(f2_dup(c10), c8), c6), c4), c2), 1.f);
    const float2 sv = f2_get(f2_mul(sn, f2_dup(magnitude))), cv = f2_get(f2_mul(cn, f2_dup(magnitude)));
    float cs[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t sb = __float_as_uint(k == 0 ? sv.x : sv.y), cb = __float_as_uint(k == 0 ? cv.x : cv.y);
        const uint32_t h = quarter[k];
        const bool odd = h & 0x40000000u;
        // cos is negated in the quarters 1 and 2, sin in 2 and 3
        cs[0][k] = __uint_as_float((odd ? sb : cb) ^ ((h ^ (h << 1)) & 0x80000000u));
        cs[1][k] = __uint_as_float((odd ? cb : sb) ^ (h & 0x80000000u));
    }
    c = f2_make(cs[0][0], cs[0][1]);
    s = f2_make(cs[1][0], cs[1][1]);
}

__device__ __forceinline__ float2 turn(int64_t position, uint64_t step, float magnitude) {
    f2 c, s;
    turn2(position, position, step, step, magnitude, c, s);
    return make_float2(f2_get(c).x, f2_get(s).x);
}

__device__ __forceinline__ int64_t position_of(const RopeP& p, int64_t b, int64_t s) {
    return p.positions ? p.positions[b * p.positions_stride + s] : s;
}

// Several axes: the axis of pair j, whose position turns it. Pairs take the axes by
// sections (from `cut` to `cut`), or in turn: j % axes while that axis has pairs left,
// the first axis otherwise. Computed, so that no map can hold an axis that is not there.
__device__ __forceinline__ int axis_of(const RopeP& p, int j) {
    if (!p.in_turn) return (j >= p.cut[0]) + (j >= p.cut[1]) + (j >= p.cut[2]);
    const int i = j / p.axes, a = j - i * p.axes;
    return a != 0 && i < p.cut[a - 1] ? a : 0;
}
__device__ __forceinline__ int64_t position_of(const RopeP& p, int64_t b, int64_t s, int j) {
    if (p.axes <= 1) return position_of(p, b, s);
    return __ldg(p.positions + axis_of(p, j) * p.axis_stride + b * p.positions_stride + s);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Vector kernels. A head is nv = head_dim / E vectors of 16 bytes; L lanes (a power
// of two, 1..32: a team) make a head, two vectors each, and a row sum of the head's
// norm is a butterfly over them. LAYOUT says which two vectors a lane takes:
//   kHalves      i and i + R/(2E) of the rotated part, so that both values of a pair
//                are in one thread
//   kInterleaved i and i + L: a pair lies inside a vector
//   kExchange    i and i + L, halves that are not whole vectors but even: the other
//                values of pairs are read from a copy of the head in shared memory
//
// A unit is a token with some of its heads, and a team takes one unit after
// another: the cos and sin of a lane's pairs depend on the token alone, so a lane
// makes its own once per unit and keeps them in registers over the unit's heads;
// no table, no barrier. What is left per head is two loads, the arithmetic on pairs
// of values (f32x2) and two stores. Bound by HBM: one read and one write of every
// head (backward with the norm: two reads).
// (Tables of a CTA's tokens in shared memory, made once for all heads, took twice
// the instructions per head: 16384 tokens of 40 heads of 128 bf16 with norms 90 to
// 114 us in several forms.)
constexpr int kHalves = 0, kInterleaved = 1, kExchange = 2;
// Heads of a team on their way into shared memory at a time. (Held in registers
// instead, they cost the backward with norms its occupancy: 100 against 83 us at
// 16384x40x128 bf16; three ahead 84, four 86.)
constexpr int kAhead = 2;

struct RopeUnits {
    int L;           // lanes per head
    int log2L;
    int nv;          // vectors per head
    int pairs;       // kHalves: vectors per half of the rotated part
    int per[2];      // heads of a unit, q and k
    int chunks[2];   // units of a token
    int64_t units[2];
    int64_t ctas[2]; // CTAs of q, of k
    float inv_d;     // 1 / head_dim
    int slots_at;    // byte offset of the copies in shared memory (backward)
};

// The two vectors of lane l (past nv: none). Lanes of a team take neighbouring
// vectors: the copies go past L1, and would fetch a sector twice for two lanes.
template <int LAYOUT>
__device__ __forceinline__ void lane_vectors(const RopeUnits& g, int l, int& a, int& b) {
    if (LAYOUT != kHalves) {
        a = l;
        b = l + g.L;
    } else if (l < g.pairs) {
        a = l;
        b = l + g.pairs;
    } else {  // behind the rotated part
        a = l + g.pairs;
        b = l + g.L;
    }
}

// A lane's place: its two vectors and its cos and sin.
template <int DT, int LAYOUT>
struct Lane {
    static constexpr int E = VecElems<DT>::value, H = E / 2;
    static constexpr int N = LAYOUT == kExchange ? 2 * E : E;  // cos and sin of a lane
    int l, va, vb;
    bool has_a, has_b;
    f2 c[N / 2], s[N / 2];

    __device__ __forceinline__ Lane(const RopeUnits& g) {
        l = threadIdx.x & (g.L - 1);
        lane_vectors<LAYOUT>(g, l, va, vb);
        has_a = va < g.nv;
        has_b = vb < g.nv;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) c[i] = s[i] = 0;  // a team without a unit turns zeros
    }
    // The value (kExchange) or pair that the lane's n-th cos and sin are for.
    __device__ __forceinline__ int index(int n) const {
        return LAYOUT == kHalves ? l * E + n : n < N / 2 ? va * (N / 2) + n : vb * (N / 2) + n - N / 2;
    }
    // kExchange: the sines come with the sign that the other value of the pair takes.
    // With several axes a pair's position comes from its axis: a lane's loads are a few
    // neighbouring ones per unit, from L1. (GB300, us, three axes / one: 16384 tokens of 40 heads of
    // 128 bf16 without norms 60 / 58, 84% of the rate of a copy; backward of 16381 of 48 heads with norms
    // 107 / 101, 84%; 64 tokens of 40 heads 3.4 / 2.9.)
    template <int SIGN, bool AXES>
    __device__ __forceinline__ void angles(const RopeP& p, const RopeUnits& g, int64_t b, int64_t s) {
        angles<SIGN, AXES>(p, g, b, s, AXES ? 0 : position_of(p, b, s));
    }
    template <int SIGN, bool AXES>
    __device__ __forceinline__ void angles(const RopeP& p, const RopeUnits& g, int64_t bi, int64_t si,
                                           int64_t position) {
        if (LAYOUT == kHalves ? l >= g.pairs : va * E >= p.R) return;
        const int half = p.R / 2;
#pragma unroll
        for (int n = 0; n < N; n += 2) {
            uint64_t step[2];  // 0: an angle that is not used
            int64_t at[2];
            uint32_t flip[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                int j = index(n + k);
                const bool second = LAYOUT == kExchange && j >= half;
                if (second) j -= half;
                step[k] = LAYOUT == kHalves || j < half ? __ldg(p.steps + j) : 0;
                at[k] = AXES ? position_of(p, bi, si, j < half ? j : 0) : position;
                flip[k] = LAYOUT == kExchange && second == (SIGN < 0) ? 0x80000000u : 0u;
            }
            turn2(at[0], at[1], step[0], step[1], p.magnitude, c[n / 2], s[n / 2]);
            if (LAYOUT == kExchange) {
                const float2 v = f2_get(s[n / 2]);
                s[n / 2] = f2_make(__uint_as_float(__float_as_uint(v.x) ^ flip[0]),
                                   __uint_as_float(__float_as_uint(v.y) ^ flip[1]));
            }
        }
    }
    // The lane's values turned by SIGN times the angle; `row`: the team's room for a
    // head in shared memory (kExchange).
    template <int SIGN>
    __device__ __forceinline__ void turned(const RopeP& p, const RopeUnits& g, f2* x, f2* z, float* row) const {
        const int half = p.R / 2;
        if (LAYOUT == kHalves) {
            if (l >= g.pairs) return;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float2 sv = f2_get(s[i]), a = f2_get(x[i]), b = f2_get(z[i]);
                const float2 ca = f2_get(f2_mul(x[i], c[i])), cb = f2_get(f2_mul(z[i], c[i]));
                if (SIGN > 0) {
                    x[i] = f2_make(fmaf(-b.x, sv.x, ca.x), fmaf(-b.y, sv.y, ca.y));
                    z[i] = f2_make(fmaf(a.x, sv.x, cb.x), fmaf(a.y, sv.y, cb.y));
                } else {
                    x[i] = f2_make(fmaf(b.x, sv.x, ca.x), fmaf(b.y, sv.y, ca.y));
                    z[i] = f2_make(fmaf(-a.x, sv.x, cb.x), fmaf(-a.y, sv.y, cb.y));
                }
            }
        } else if (LAYOUT == kInterleaved) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                f2* y = k == 0 ? x : z;
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const int n = k * H + i;
                    if (index(n) >= half) continue;  // the rotated part may end in a vector
                    const float2 cp = f2_get(c[n / 2]), sp = f2_get(s[n / 2]), v = f2_get(y[i]);
                    const float cv = n & 1 ? cp.y : cp.x, sv = SIGN * (n & 1 ? sp.y : sp.x);
                    y[i] = f2_make(fmaf(-v.y, sv, v.x * cv), fmaf(v.x, sv, v.y * cv));
                }
            }
        } else {
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                f2* y = k == 0 ? x : z;
                const int first = (k == 0 ? va : vb) * E;
                if (first < p.R) {
#pragma unroll
                    for (int i = 0; i < H; ++i) *reinterpret_cast<float2*>(row + first + 2 * i) = f2_get(y[i]);
                }
            }
            __syncwarp();
            // half is even, so two values and their two others lie side by side
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                f2* y = k == 0 ? x : z;
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    const int j = (k == 0 ? va : vb) * E + 2 * i;
                    if (j >= p.R) continue;
                    const float2 o = *reinterpret_cast<const float2*>(row + (j < half ? j + half : j - half));
                    y[i] = f2_fma(f2_make(o.x, o.y), s[k * H + i], f2_mul(y[i], c[k * H + i]));
                }
            }
        }
    }
};

__device__ __forceinline__ float lanes_sum(float v, int L) {
    if (L > 8) {
        if (L > 16) v += __shfl_xor_sync(0xffffffffu, v, 16);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
    }
    if (L > 4) v += __shfl_xor_sync(0xffffffffu, v, 4);
    if (L > 2) v += __shfl_xor_sync(0xffffffffu, v, 2);
    if (L > 1) v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v;
}

// A unit: its token and heads.
struct Unit {
    int64_t b, s, token;
    int h, n;  // first head, heads (0: no unit)
    __device__ __forceinline__ Unit(const RopeP& p, const RopeUnits& g, int which, int heads, int64_t u) {
        const int chunks = g.chunks[which];
        int chunk;
        if (g.units[which] < (int64_t(1) << 31)) {  // 32-bit division
            const int t = static_cast<int>(u) / chunks;
            chunk = static_cast<int>(u) - t * chunks;
            token = t;
        } else {
            token = u / chunks;
            chunk = static_cast<int>(u - token * chunks);
        }
        b = p.batch == 1 ? 0 : token / p.seq;
        s = token - b * p.seq;
        h = chunk * g.per[which];
        n = u < g.units[which] ? min(g.per[which], heads - h) : 0;
    }
    __device__ __forceinline__ int64_t at(const HeadsP& x) const { return b * x.sb + s * x.st + h * x.sh; }
};

// Asynchronous copies into shared memory that the copying thread alone reads
// back (cp.async: any stride, no registers, no barrier).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Forward.
template <int DT, int LAYOUT, bool NORM, bool AXES>
__global__ void __launch_bounds__(256) rope_fwd_kernel(const RopeP p, const RopeUnits g) {
    using Ln = Lane<DT, LAYOUT>;
    constexpr int H = Ln::H, S = kAhead;
    extern __shared__ __align__(16) float rows[];
    const int which = blockIdx.x >= g.ctas[0];
    const RopeSeg sg = p.seg[which];
    Ln ln(g);
    const int team = threadIdx.x >> g.log2L, teams = 256 >> g.log2L;
    float* row = rows + team * p.D;
    const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
    const bool norm = NORM && sg.w;
    const int vd = ln.vb - ln.va, per = g.per[which];
    const unsigned char* slots = reinterpret_cast<const unsigned char*>(rows) + g.slots_at + threadIdx.x * 16;
    const uint32_t slot0 = static_cast<uint32_t>(__cvta_generic_to_shared(slots));
    for (int k = 0; k < S * 2; ++k)  // lanes past the head's end read zeros
        *reinterpret_cast<uint4*>(const_cast<unsigned char*>(slots) + k * 4096) = zero4;
    pdl_wait();
    pdl_launch_dependents();
    f2 wa[H], wb[H];
    if (norm) {
        const uint4* w = static_cast<const uint4*>(sg.w);
        weights2<DT>(ln.has_a ? __ldg(w + ln.va) : zero4, p.offset, wa);
        weights2<DT>(ln.has_b ? __ldg(w + ln.vb) : zero4, p.offset, wb);
    }
    const int64_t first = (blockIdx.x - (which ? g.ctas[0] : 0)) * teams;
    for (int64_t u0 = first; u0 < g.units[which]; u0 += g.ctas[which] * teams) {
        const Unit u(p, g, which, sg.heads, u0 + team);
        const uint4* in = static_cast<const uint4*>(sg.in.p) + u.at(sg.in) + ln.va;
        uint4* out = static_cast<uint4*>(sg.out.p) + u.at(sg.out) + ln.va;
        float* rstd = norm && sg.rstd && ln.l == 0 ? sg.rstd + (u.token * sg.heads + u.h) : nullptr;
        uint32_t put = 0, take = 0;
        int ahead = 0;
        auto fetch = [&]() {
            if (ahead < u.n) {
                if (ln.has_a) copy16(slot0 + put, in);
                if (ln.has_b) copy16(slot0 + put + 4096, in + vd);
                in += sg.in.sh;
            }
            ++ahead;
            copies_commit();
            put = put == (S - 1) * 8192 ? 0 : put + 8192;
        };
#pragma unroll
        for (int k = 0; k < S; ++k) fetch();
        if (u.n) ln.template angles<1, AXES>(p, g, u.b, u.s);
        for (int h = 0; h < per; ++h) {
            const bool live = h < u.n;
            copies_wait<S - 1>();
            f2 x[H], z[H];
            unpack2<DT>(*reinterpret_cast<const uint4*>(slots + take), x);
            unpack2<DT>(*reinterpret_cast<const uint4*>(slots + take + 4096), z);
            take = take == (S - 1) * 8192 ? 0 : take + 8192;
            fetch();
            if (norm) {
                f2 sq = 0;
#pragma unroll
                for (int e = 0; e < H; ++e) sq = f2_fma(z[e], z[e], f2_fma(x[e], x[e], sq));
                const float r = rsqrtf(fmaf(lanes_sum(f2_sum(sq), g.L), g.inv_d, p.eps));
                if (live && rstd) rstd[h] = r;
                const f2 r2 = f2_dup(r);
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    x[e] = f2_mul(f2_mul(x[e], r2), wa[e]);
                    z[e] = f2_mul(f2_mul(z[e], r2), wb[e]);
                }
            }
            ln.template turned<1>(p, g, x, z, row);
            if (live) {
                if (ln.has_a) st_stream(out, pack2<DT>(x));
                if (ln.has_b) st_stream(out + vd, pack2<DT>(z));
            }
            out += sg.out.sh;
        }
    }
    copies_wait<0>();
}

// Backward: turned back, then the norm's backward, with the weights' gradients of
// a lane's columns summed in registers over all the heads it sees, and over the
// CTA's teams (in order) into one partial row.
template <int DT, int LAYOUT, bool NORM, bool AXES>
__global__ void __launch_bounds__(256) rope_bwd_kernel(const RopeP p, const RopeUnits g) {
    using Ln = Lane<DT, LAYOUT>;
    constexpr int E = Ln::E, H = Ln::H, NV = NORM ? 4 : 2, S = kAhead;
    extern __shared__ __align__(16) float rows[];
    const int which = blockIdx.x >= g.ctas[0];
    const RopeSeg sg = p.seg[which];
    Ln ln(g);
    const int team = threadIdx.x >> g.log2L, teams = 256 >> g.log2L;
    float* row = rows + team * p.D;
    const uint4 zero4 = make_uint4(0u, 0u, 0u, 0u);
    const bool norm = NORM && sg.w;
    const int vd = ln.vb - ln.va, per = g.per[which];
    const unsigned char* slots = reinterpret_cast<const unsigned char*>(rows) + g.slots_at + threadIdx.x * 16;
    const uint32_t slot0 = static_cast<uint32_t>(__cvta_generic_to_shared(slots));
    for (int k = 0; k < S * NV; ++k)  // lanes past the head's end read zeros
        *reinterpret_cast<uint4*>(const_cast<unsigned char*>(slots) + k * 4096) = zero4;
    pdl_wait();
    f2 wa[H], wb[H], da[H], db[H];
#pragma unroll
    for (int e = 0; e < H; ++e) da[e] = db[e] = 0;
    if (norm) {
        const uint4* w = static_cast<const uint4*>(sg.w);
        weights2<DT>(ln.has_a ? __ldg(w + ln.va) : zero4, p.offset, wa);
        weights2<DT>(ln.has_b ? __ldg(w + ln.vb) : zero4, p.offset, wb);
    }
    const int64_t cta = blockIdx.x - (which ? g.ctas[0] : 0);
    for (int64_t u0 = cta * teams; u0 < g.units[which]; u0 += g.ctas[which] * teams) {
        const Unit u(p, g, which, sg.heads, u0 + team);
        const uint4* in = static_cast<const uint4*>(sg.in.p) + u.at(sg.in) + ln.va;
        const uint4* xin = static_cast<const uint4*>(sg.x.p) + (norm ? u.at(sg.x) + ln.va : 0);
        uint4* out = static_cast<uint4*>(sg.out.p) + u.at(sg.out) + ln.va;
        const float* rstd = norm ? sg.rstd + (u.token * sg.heads + u.h) : nullptr;
        uint32_t put = 0, take = 0;
        int ahead = 0;
        auto fetch = [&]() {
            if (ahead < u.n) {
                if (ln.has_a) copy16(slot0 + put, in);
                if (ln.has_b) copy16(slot0 + put + 4096, in + vd);
                if (norm) {
                    if (ln.has_a) copy16(slot0 + put + 8192, xin);
                    if (ln.has_b) copy16(slot0 + put + 12288, xin + vd);
                }
                in += sg.in.sh;
                xin += sg.x.sh;
            }
            ++ahead;
            copies_commit();
            put = put == (S - 1) * NV * 4096 ? 0 : put + NV * 4096;
        };
#pragma unroll
        for (int k = 0; k < S; ++k) fetch();
        float r_next = norm && u.n > 0 ? __ldg(rstd) : 0.f;
        if (u.n) ln.template angles<-1, AXES>(p, g, u.b, u.s);
        for (int h = 0; h < per; ++h) {
            const bool live = h < u.n;
            const float r = r_next;
            r_next = norm && h + 1 < u.n ? __ldg(rstd + h + 1) : 0.f;
            copies_wait<S - 1>();
            uint4 ga = zero4, gb = zero4, xa = zero4, xb = zero4;
            if (live) {
                ga = *reinterpret_cast<const uint4*>(slots + take);
                gb = *reinterpret_cast<const uint4*>(slots + take + 4096);
                if (norm) {
                    xa = *reinterpret_cast<const uint4*>(slots + take + 8192);
                    xb = *reinterpret_cast<const uint4*>(slots + take + 12288);
                }
            }
            take = take == (S - 1) * NV * 4096 ? 0 : take + NV * 4096;
            fetch();
            f2 ta[H], tb[H];
            unpack2<DT>(ga, ta);
            unpack2<DT>(gb, tb);
            ln.template turned<-1>(p, g, ta, tb, row);
            if (norm) {
                f2 x[H], z[H], c2 = 0;
                unpack2<DT>(xa, x);
                unpack2<DT>(xb, z);
                const f2 r2 = f2_dup(r);
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    const f2 gx = f2_mul(ta[e], x[e]), gz = f2_mul(tb[e], z[e]);
                    da[e] = f2_fma(gx, r2, da[e]);
                    db[e] = f2_fma(gz, r2, db[e]);
                    c2 = f2_fma(gz, wb[e], f2_fma(gx, wa[e], c2));
                }
                const float c = lanes_sum(f2_sum(c2), g.L);
                // r^3 c / D, the small factor first: r^3 alone leaves fp32's range for
                // heads of an RMS below 1e-13
                const f2 mf = f2_dup(-(r * (r * (r * (c * g.inv_d)))));
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    ta[e] = f2_fma(f2_mul(ta[e], r2), wa[e], f2_mul(x[e], mf));
                    tb[e] = f2_fma(f2_mul(tb[e], r2), wb[e], f2_mul(z[e], mf));
                }
            }
            if (live) {
                if (ln.has_a) st_stream(out, pack2<DT>(ta));
                if (ln.has_b) st_stream(out + vd, pack2<DT>(tb));
            }
            out += sg.out.sh;
        }
    }
    copies_wait<0>();
    pdl_launch_dependents();
    if (!norm) return;
    // A warp's teams meet by shuffles, the warps in order in shared memory:
    // [8 warps][L lanes][2E].
    __syncthreads();
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
            float2* part = reinterpret_cast<float2*>(rows) + (w * g.L + lane) * E;
            part[e] = a;
            part[H + e] = b;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < g.L * 2 * E; i += 256) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) t += rows[k * g.L * 2 * E + i];
        const int li = i / (2 * E), e = i % (2 * E);
        int a, b;
        lane_vectors<LAYOUT>(g, li, a, b);
        const int j = e < E ? a * E + e : b * E + e - E;
        if (j < p.D) p.ws[(which ? g.ctas[0] + cta : cta) * p.D + j] = t;
    }
}

// Element-wise kernels: any head size, alignment and stride; one warp per head
// of a token (head index over q's and then k's heads). A lane owns the pairs
// lane, lane + 32, ... and the values behind rotary_dim in the same way, reads
// both values of a pair before it writes them, and no lane reads another's, so
// the outputs may lie on the inputs.
struct Place {
    int seg;
    int64_t b, s, h, token;
};

__device__ __forceinline__ Place unit_of(const RopeP& p, int64_t u) {
    const int H = p.seg[0].heads + p.seg[1].heads;
    Place o;
    o.token = u / H;
    o.h = u - o.token * H;
    o.seg = o.h >= p.seg[0].heads;
    if (o.seg) o.h -= p.seg[0].heads;
    o.b = o.token / p.seq;
    o.s = o.token - o.b * p.seq;
    return o;
}

__device__ __forceinline__ int64_t at(const HeadsP& h, const Place& u) {
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
        const Place u = unit_of(p, i);
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
        __syncwarp();  // every lane's reads for the sum before the first write
        for (int j = lane; j < half; j += 32) {
            const float2 cs = turn(position_of(p, u.b, u.s, j), p.steps[j], p.magnitude);
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
        const Place u = unit_of(p, i);
        const RopeSeg& g = p.seg[u.seg];
        const int64_t d0 = at(g.in, u), o0 = at(g.out, u), x0 = at(g.x, u);
        // The gradient of the normed head at pair j (as its two values) and
        // behind rotary_dim.
        auto back = [&](int j) {
            const float2 cs = turn(position_of(p, u.b, u.s, j), p.steps[j], p.magnitude);
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
            f = r * (r * (warp_sum(c) / static_cast<float>(p.D)));
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
__global__ void __launch_bounds__(1024) rope_dw_kernel(const RopeP p, RopeRows rows, int paired) {
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, half = p.R / 2;
    const int slot = static_cast<int>(blockIdx.x) * 32 + lane;
    pdl_wait();
    if (!p.seg[blockIdx.y].w) return;
    float t = 0.f;
    if (slot < p.D) {
        const float* q = p.ws + (blockIdx.y ? rows.n[0] : 0) * p.D + slot;
        const int64_t n = rows.n[blockIdx.y];
        int64_t i = w;
        for (; i + 7 * 32 < n; i += 8 * 32) {  // eight loads, then the additions in order
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = q[(i + 32 * k) * p.D];
#pragma unroll
            for (int k = 0; k < 8; ++k) t += v[k];
        }
        for (; i < n; i += 32) t += q[i * p.D];
    }
    part[w][lane] = t;
    __syncthreads();
    if (w == 0 && slot < p.D) {
        t = 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) t += part[k][lane];
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

// Whether every head is whole 16-byte vectors, of at most 64.
bool vectors(const RopeP& p, bool bwd) {
    const int E = vec_elems(p.dtype);
    if (p.D % E != 0 || p.D > 64 * E) return false;
    if (!p.interleaved && p.R % 4 != 0) return false;  // kExchange takes values in twos
    for (const RopeSeg& s : p.seg) {
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
    return true;
}

int layout_of(const RopeP& p) {
    return p.interleaved ? kInterleaved : p.R % (2 * vec_elems(p.dtype)) == 0 ? kHalves : kExchange;
}

// Opts a kernel into `smem` bytes on the current device, once; the CTAs per SM.
int opt_in_occupancy(const void* fn, int threads, int smem) {
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
    return occupancy(fn, threads, smem);
}

// Lays out the units: lanes per head, heads per unit, CTAs; strides in vectors.
RopeUnits units_of(RopeP* p, const OpCfg& c, int threads, int ctas_per_sm) {
    const int E = vec_elems(p->dtype);
    for (RopeSeg& s : p->seg)
        for (HeadsP* h : {&s.in, &s.out, &s.x}) h->sb /= E, h->st /= E, h->sh /= E;
    RopeUnits g;
    g.slots_at = 0;
    g.nv = p->D / E;
    g.inv_d = 1.f / static_cast<float>(p->D);
    g.pairs = layout_of(*p) == kHalves ? p->R / (2 * E) : 0;
    g.L = 1;
    g.log2L = 0;
    while (g.L * 2 < g.nv) {
        g.L <<= 1;
        ++g.log2L;
    }
    const int64_t teams = threads / g.L, tokens = p->batch * p->seq;
    int64_t cap = static_cast<int64_t>(c.dev.sm_count) * ctas_per_sm;
    if (c.max_ctas > 0) cap = std::min<int64_t>(cap, std::max(c.max_ctas, 2));
    // Units of as many heads as leave every team one, and of eight at most, so that the
    // teams of long calls end together; a unit of many heads costs fewer angles (GB300,
    // us, at eight units per team and up to 16 heads / one and up to 16 / one and up to
    // 8: 8169 tokens of 25 heads of 128 bf16 with norms 31.6 / 22.8 / 23.6, 7391 of 24 of
    // 80 29.9 / 18.0 / 17.9, 16384 of 40 of 128 59.0 / 59.0 / 56.7, its backward 82.8 /
    // 84.2 / 82.9, each before the angles' series, which costs up to 2%).
    const int64_t heads = p->seg[0].heads + p->seg[1].heads;
    const int64_t share = std::max<int64_t>(1, std::min<int64_t>(8, tokens * heads / (cap * teams)));
    int64_t work[2] = {0, 0};
    for (int k = 0; k < 2; ++k) {
        const int64_t n = p->seg[k].heads;
        g.per[k] = g.chunks[k] = 0;
        g.units[k] = 0;
        if (n == 0) continue;
        g.chunks[k] = static_cast<int>((n + share - 1) / share);
        g.per[k] = static_cast<int>((n + g.chunks[k] - 1) / g.chunks[k]);
        g.chunks[k] = static_cast<int>((n + g.per[k] - 1) / g.per[k]);
        g.units[k] = tokens * g.chunks[k];
        work[k] = n;
    }
    // CTAs in proportion to the heads.
    int64_t need[2] = {(g.units[0] + teams - 1) / teams, (g.units[1] + teams - 1) / teams};
    if (need[0] + need[1] <= cap) {
        g.ctas[0] = need[0];
        g.ctas[1] = need[1];
    } else {
        g.ctas[0] = std::min(need[0], std::max<int64_t>(1, (cap * work[0] + heads / 2) / heads));
        g.ctas[1] = work[1] ? std::min(need[1], std::max<int64_t>(1, cap - g.ctas[0])) : 0;
    }
    return g;
}

template <int DT, int LAYOUT, bool NORM, bool AXES>
cudaError_t fwd_units(RopeP p, const OpCfg& c) {
    auto fn = rope_fwd_kernel<DT, LAYOUT, NORM, AXES>;
    // Heads to exchange, behind them the copies.
    const int at = LAYOUT == kExchange ? 256 * 2 * VecElems<DT>::value * 4 : 0;
    const int smem = at + 2 * kAhead * 4096;
    const int occ = opt_in_occupancy(reinterpret_cast<const void*>(fn), 256, smem);
    if (occ < 1) return cudaErrorInvalidConfiguration;
    RopeUnits g = units_of(&p, c, 256, occ);
    g.slots_at = at;
    return op_launch(c, fn, g.ctas[0] + g.ctas[1], 256, smem, p, g);
}

cudaError_t launch_dw(const RopeP& p, const OpCfg& c, int64_t rows_q, int64_t rows_k, int paired) {
    Launch l;
    l.grid = (p.D + 31) / 32;
    l.threads = 1024;
    LaunchCfg cfg(l, c.stream, c.pdl);
    cfg.cfg.gridDim.y = 2;
    return cudaLaunchKernelEx(&cfg.cfg, rope_dw_kernel, p, RopeRows{{rows_q, rows_k}}, paired);
}

template <int DT, int LAYOUT, bool NORM, bool AXES>
cudaError_t bwd_units(RopeP p, const OpCfg& c) {
    constexpr int E = VecElems<DT>::value;
    auto fn = rope_bwd_kernel<DT, LAYOUT, NORM, AXES>;
    // Heads to exchange, then the sums over the warps; behind them the copies.
    const int at = LAYOUT == kExchange || NORM ? 256 * 2 * E * 4 : 0;
    const int smem = at + (NORM ? 4 : 2) * kAhead * 4096;
    const int occ = std::min(8, opt_in_occupancy(reinterpret_cast<const void*>(fn), 256, smem));
    if (occ < 1) return cudaErrorInvalidConfiguration;
    RopeUnits g = units_of(&p, c, 256, occ);
    g.slots_at = at;
    const cudaError_t e = op_launch(c, fn, g.ctas[0] + g.ctas[1], 256, smem, p, g);
    return e != cudaSuccess || !NORM ? e : launch_dw(p, c, g.ctas[0], g.ctas[1], 0);
}

template <int DT, int LAYOUT, bool AXES>
cudaError_t run_units(const RopeP& p, const OpCfg& c, bool bwd) {
    if (p.seg[0].w || p.seg[1].w)
        return bwd ? bwd_units<DT, LAYOUT, true, AXES>(p, c) : fwd_units<DT, LAYOUT, true, AXES>(p, c);
    return bwd ? bwd_units<DT, LAYOUT, false, AXES>(p, c) : fwd_units<DT, LAYOUT, false, AXES>(p, c);
}

template <int DT, int LAYOUT>
cudaError_t run_axes(const RopeP& p, const OpCfg& c, bool bwd) {
    return p.axes > 1 ? run_units<DT, LAYOUT, true>(p, c, bwd) : run_units<DT, LAYOUT, false>(p, c, bwd);
}

template <int DT>
cudaError_t run(const RopeP& p, const OpCfg& c, bool bwd) {
    if (c.variant != RMSNORM_VARIANT_GENERIC && vectors(p, bwd)) {
        switch (layout_of(p)) {
            case kHalves: return run_axes<DT, kHalves>(p, c, bwd);
            case kInterleaved: return run_axes<DT, kInterleaved>(p, c, bwd);
            default: return run_axes<DT, kExchange>(p, c, bwd);
        }
    }
    if (c.variant == RMSNORM_VARIANT_CTA) return cudaErrorNotSupported;
    const int64_t G = generic_grid(p, c);
    if (!bwd) return op_launch(c, rope_fwd_generic_kernel<DT>, G, 256, 0, p);
    const cudaError_t e = op_launch(c, rope_bwd_generic_kernel<DT>, G, 256, 0, p);
    return e != cudaSuccess || !(p.seg[0].w || p.seg[1].w) ? e : launch_dw(p, c, G * 8, G * 8, 1);
}

cudaError_t run(const RopeP& p, const OpCfg& c, bool bwd) {
    switch (p.dtype) {
        case kBF16: return run<kBF16>(p, c, bwd);
        case kFP16: return run<kFP16>(p, c, bwd);
        default: return run<kFP32>(p, c, bwd);
    }
}

}  // namespace

int64_t rope_bwd_partial_rows(int sm_count) {
    return 2LL * sm_count * kGenericCtasPerSM * 8;
}

cudaError_t rope_fwd_run(const RopeP& p, const OpCfg& c) { return run(p, c, false); }

cudaError_t rope_bwd_run(const RopeP& p, const OpCfg& c) { return run(p, c, true); }

}  // namespace rmsn
