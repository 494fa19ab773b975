// Attention over the quantised cache by matrix instructions, for blocks of 8 * NT rows of a key
// head: single tokens of the query heads that share a key head, a few drafted tokens, and
// prompts.
//
// The mathematics. With K = 2^a * c (a scale a token and group, c the codes), a score is
//   s[t, r] = sum over groups of 2^a[t, g] * (c[t, g, :] . q[r, g, :])
// so the codes themselves are an operand (exact in fp16, whatever the scale), q the other (a row
// brought near 2^15 by a power of two, so that fp16 holds bf16 and fp16 values exactly but for those
// 2^-28 below the row's largest; fp32 in two pieces of 11 bits), and the scale is a factor on
// fp32 sums: 16 tokens x 8 rows of a group in four instructions per lane instead of one per
// value. For V the scale goes to the probabilities, o[d, r] += c[t, d] * (2^b[t, g] p[t, r]), per
// group, relative to the group's largest scale so far and times 2^8: 22 powers of two below the
// largest are full fp16 values, 32 are kept in part.
// Both products take the codes as the first operand (16 tokens x 16 values of K; 16 values
// x 16 tokens of V) and 8 rows as the second, so a row costs an eighth of an instruction and no
// lane idles for 8 rows. A token's probabilities for the second product come from the first one's
// sums by an 8x8 transposition in registers.
// Order of values: the sum over d, the sum over t and the place of d in the result may be permuted
// at will, as long as both operands agree. A lane takes 8 neighbouring values of K (its k
// indices 2t, 2t+1, 2t+8, 2t+9 of two instructions) and 4 of V, so that codes are read by words,
// bytes of two tokens are paired by one permutation for two pairs, and a conversion instruction takes a
// pair. Row g of the first product is token g ^ (g >> 2 & 1): with that the four tokens of a
// V read lie on different banks too.
//
// Each warp runs on its own: a ring of two tiles, filled by asynchronous copies of 16 bytes (a token's
// row of codes at a time), no barrier in the loop; page numbers are looked up two tiles ahead,
// scale bytes travel through registers one tile ahead. Softmax with a running maximum, which moves
// only where a score exceeds it by more than 2^4 (the sums then carry factors up to 2^4).
// Bound: for 8 rows, reading the cache (HBM); for 32, the matrix and conversion instructions.
#pragma once

#include "attn_common.cuh"
#include "attn_rows.h"

namespace rmsn {
namespace {

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 half2_values(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint32_t pair_e4m3(uint32_t c) {
    const __half2 h = static_cast<__half2>(
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c & 0xffffu), __NV_E4M3));
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pair_e2m1(uint32_t c) {
    const __half2 h = static_cast<__half2>(
        __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(c & 0xffu), __NV_E2M1));
    return *reinterpret_cast<const uint32_t*>(&h);
}

// d += a b: a 16x16 (rows lane / 4 and that + 8), b 16x8, fp16 in, fp32 sums.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint2& b) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}
// An 8x8 matrix of 16-bit values (row lane / 4, columns 2 (lane % 4) and the next) transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, bool some) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(some ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_async4(uint32_t dst, const void* src, bool some) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(some ? 4 : 0) : "memory");
}
__device__ __forceinline__ uint32_t smem_at(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 2^e as fp32, 0 below 2^-126 (e <= 127).
__device__ __forceinline__ float power(int e) { return __uint_as_float(e < -126 ? 0u : static_cast<uint32_t>(e + 127) << 23); }

// A block of rows of a sequence, and the tiles of tokens that it sees.
struct Slot {
    int64_t b;
    Sequence s;
    int64_t r0;        // first row of the block among the sequence's (queries times G)
    int rows;          // 0: no such slot
    int64_t low, high; // tokens that any of its rows sees
    int64_t tile0;     // the first tile
    int64_t tiles;     // at least one where there are rows
};

__device__ __forceinline__ int64_t slot_start(const AttnP& p, int64_t b, int R) {
    return first_row(p, b) * p.G / R + b;
}

__device__ __forceinline__ Slot slot_of(const AttnP& p, int64_t slot, int R, int tile) {
    int64_t lo = 0, hi = p.sequences - 1;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (slot_start(p, mid, R) <= slot) lo = mid;
        else hi = mid - 1;
    }
    Slot r;
    r.b = lo;
    r.s = sequence(p, lo);
    const int64_t start = slot_start(p, lo, R), all = r.s.n * p.G;
    r.r0 = (slot - start) * R;
    r.rows = 0;
    r.low = r.high = r.tile0 = r.tiles = 0;
    if (slot < start || r.r0 >= all) return r;
    r.rows = static_cast<int>(all - r.r0 < R ? all - r.r0 : R);
    r.low = seen(p, r.s, r.r0 / p.G).low;
    r.high = seen(p, r.s, (r.r0 + r.rows - 1) / p.G).high;
    if (r.high > r.s.len) r.high = r.s.len;
    r.tile0 = r.low / tile;
    r.tiles = r.high > r.low ? (r.high + tile - 1) / tile - r.tile0 : 1;
    return r;
}

// F: format; GD: groups of a head; NT: blocks of 8 NT rows; NP: pieces of q and of the
// probabilities (2 for fp32).
template <int F, int GD, int NT, int NP>
struct Rows {
    static constexpr bool E4 = F == RMSNORM_CACHE_E4M3;
    static constexpr int DP = GD * 32, RB = E4 ? DP : DP / 2, PITCH = rows_pitch(E4, GD);
    static constexpr int TM = !E4 && GD <= 4 ? 2 : 1, TOK = 16 * TM, STAGE = 2 * TOK * PITCH;
    static constexpr int FP = rows_factors(GD), R = 8 * NT, KS = 2 * GD;
    static constexpr bool QREG = NT == 1 && NP == 1;
    // Two CTAs of eight warps an SM where the sums leave the registers for it.
    static constexpr int CTAS = GD * NT <= 4 && NP == 1 ? 2 : 1;
    static constexpr int LIFT = 8;  // the probabilities' factor 2^8 (see above)

    static __host__ __device__ constexpr int ring_bytes() {
        const int results = (R * (DP + 4) + 2 * R) * 4;
        return 2 * STAGE > results ? 2 * STAGE : results;
    }
    static __host__ __device__ constexpr int q_bytes() { return QREG ? 0 : NP * KS * NT * 32 * 8; }
    static __host__ __device__ constexpr int factor_bytes() { return 2 * TOK * FP * 4; }
};

// A 16-bit pair of the call's type.
__device__ __forceinline__ float2 unpack16(uint32_t v, bool bf16) {
    return bf16 ? Codec<kBF16>::unpack2(v) : Codec<kFP16>::unpack2(v);
}
template <int NP>
__device__ __forceinline__ float load_value(const void* p, int64_t i, int dtype) {
    if (NP == 2) return load1<kFP32>(p, i);
    return dtype == kBF16 ? load1<kBF16>(p, i) : load1<kFP16>(p, i);
}
template <int NP>
__device__ __forceinline__ void store_value(void* p, int64_t i, float v, int dtype) {
    if (NP == 2) store1<kFP32>(p, i, v);
    else if (dtype == kBF16) store1<kBF16>(p, i, v);
    else store1<kFP16>(p, i, v);
}

template <int F, int GD, int NT, int NP>
__global__ void __launch_bounds__(256, Rows<F, GD, NT, NP>::CTAS) attn_rows_kernel(const AttnP p, const RowsPlan r) {
    using C = Rows<F, GD, NT, NP>;
    constexpr bool E4 = C::E4;
    constexpr int DP = C::DP, RB = C::RB, PITCH = C::PITCH, TM = C::TM, TOK = C::TOK, FP = C::FP, R = C::R, KS = C::KS;
    constexpr float kNegInf = -INFINITY;
    extern __shared__ __align__(128) unsigned char sm[];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    const int head_local = w % r.hb, slice = w / r.hb, threads = blockDim.x;
    const int x = static_cast<int>(blockIdx.x) / r.head_blocks, hblock = static_cast<int>(blockIdx.x) - x * r.head_blocks;
    const int head = hblock * r.hb + head_local;
    const int tile_tokens = TOK * r.wph;
    unsigned char* ring = sm + r.at_ring + w * r.ring;
    float* factors = reinterpret_cast<float*>(sm + r.at_factors + w * C::factor_bytes());
    uint2* qs = reinterpret_cast<uint2*>(sm + r.at_q + head_local * C::q_bytes());
    int64_t* before = reinterpret_cast<int64_t*>(sm + r.at_plan);  // tiles before each slot
    if (r.narrow) {  // what lies behind a token's codes stays zero
        for (int i = lane; i < 2 * C::STAGE / 16; i += 32) reinterpret_cast<uint4*>(ring)[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    pdl_wait();
    pdl_launch_dependents();

    // Which tiles are this CTA's.
    int64_t begin = 0, end = 0, share = 1;
    int64_t slot = x;
    if (r.split) {
        __shared__ int64_t warp_tiles[8];
        const int run = (r.slots + threads - 1) / threads;
        int64_t own = 0;
        for (int i = threadIdx.x * run; i < min(r.slots, static_cast<int>(threadIdx.x + 1) * run); ++i) {
            const int64_t n = slot_of(p, i, R, tile_tokens).tiles;
            before[i + 1] = n;
            own += n;
        }
        int64_t sum = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += o;
        }
        if (lane == 31) warp_tiles[w] = sum;
        __syncthreads();
        sum -= own;
        int64_t total = 0;
        for (int i = 0; i < threads / 32; ++i) {
            if (i < w) sum += warp_tiles[i];
            total += warp_tiles[i];
        }
        if (threadIdx.x == 0) before[0] = 0;
        for (int i = threadIdx.x * run; i < min(r.slots, static_cast<int>(threadIdx.x + 1) * run); ++i) {
            sum += before[i + 1];
            before[i + 1] = sum;
        }
        __syncthreads();
        share = (total + r.gx - 1) / r.gx;
        begin = share * x;
        end = begin + share < total ? begin + share : total;
        if (begin >= end) return;
        int lo = 0, hi = r.slots - 1;  // the last slot that begins at or before the first tile
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (before[mid] <= begin) lo = mid;
            else hi = mid - 1;
        }
        slot = lo;
    }

    const uint8_t* kcodes = p.codes[0];
    const uint8_t* vcodes = p.codes[1];
    const int64_t head_off = head * head_step(p);
    const int gtok = g ^ ((g >> 2) & 1);              // the token of row g of a product
    const int vt0 = (2 * t4) ^ (t4 >> 1), vt1 = vt0 ^ 1;  // the tokens of its columns 2 t4 and 2 t4 + 1

    for (; slot < r.slots; slot += r.split ? 1 : r.gx) {
        if (r.split && before[slot] >= end) break;
        const Slot sl = slot_of(p, slot, R, tile_tokens);
        int64_t first = 0, last = sl.tiles;  // tiles of the slot, from its first
        int64_t slot_begin = 0;
        if (r.split) {
            slot_begin = before[slot];
            first = begin > slot_begin ? begin - slot_begin : 0;
            last = before[slot + 1] < end ? sl.tiles : end - slot_begin;
        }
        if (sl.rows == 0) continue;
        first += sl.tile0;
        last += sl.tile0;

        // ---- q: a row's largest magnitude, its power of two, and its values as fp16 operands
        uint2 qreg[C::QREG ? KS : 1];
        float col_scale[NT][2];
        int lim[NT][2], low[NT][2];  // tokens that a column's row sees, relative to the slot's first tile
        const int64_t base_token = sl.tile0 * tile_tokens;
        int min_lim = INT32_MAX, max_low = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int rr = nt * 8 + g;
            const bool live = rr < sl.rows;
            const int64_t i = live ? (sl.r0 + rr) / p.G : 0;
            const int64_t row = sl.s.row0 + i;
            const int qh = head * p.G + (live ? static_cast<int>(sl.r0 + rr - i * p.G) : 0);
            const int64_t at = row * p.q.st + qh * p.q.sh;
            float v[GD][8];
            float top = 0.f;
#pragma unroll
            for (int grp = 0; grp < GD; ++grp) {
                const int d = grp * 32 + t4 * 8;
                if (live && r.vec_q && d + 8 <= p.D) {
                    const unsigned char* src = static_cast<const unsigned char*>(p.q.p) + (at + d) * (NP == 2 ? 4 : 2);
#pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        const uint4 u = __ldg(reinterpret_cast<const uint4*>(src) + k);
                        const uint32_t word[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (NP == 2) {
                                v[grp][(k * 4 + e) & 7] = __uint_as_float(word[e]);
                            } else {
                                const float2 f = unpack16(word[e], p.dtype == kBF16);
                                v[grp][2 * e] = f.x;
                                v[grp][2 * e + 1] = f.y;
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[grp][e] = live && d + e < p.D ? load_value<NP>(p.q.p, at + d + e, p.dtype) : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[grp][e]));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            int ex = static_cast<int>(__float_as_uint(top) >> 23);
            ex = top == 0.f ? 141 : ex < 15 ? 15 : ex;  // both powers stay normal
            const float up = __uint_as_float(static_cast<uint32_t>(268 - ex) << 23);
            const float down = __uint_as_float(static_cast<uint32_t>(ex - 14) << 23) * (p.scale * 1.4426950408889634f);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const float* f = &v[ks >> 1][(ks & 1) * 4];
                const float a0 = f[0] * up, a1 = f[1] * up, a2 = f[2] * up, a3 = f[3] * up;
                const uint2 hi = make_uint2(half2_bits(a0, a1), half2_bits(a2, a3));
                if (C::QREG) {
                    qreg[C::QREG ? ks : 0] = hi;
                } else if (slice == 0) {
                    qs[(ks * NT + nt) * 32 + lane] = hi;
                    if (NP == 2) {
                        const float2 h0 = half2_values(hi.x), h1 = half2_values(hi.y);
                        qs[(KS * NT + ks * NT + nt) * 32 + lane] =
                            make_uint2(half2_bits(a0 - h0.x, a1 - h0.y), half2_bits(a2 - h1.x, a3 - h1.y));
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = 2 * t4 + e;
                col_scale[nt][e] = __shfl_sync(0xffffffffu, down, col * 4);
                const int cr = nt * 8 + col;
                lim[nt][e] = INT32_MAX;
                low[nt][e] = 0;
                if (cr < sl.rows) {
                    const Seen see = seen(p, sl.s, (sl.r0 + cr) / p.G);
                    const int64_t h = (see.high < sl.s.len ? see.high : sl.s.len) - base_token;
                    lim[nt][e] = static_cast<int>(h < 0 ? 0 : h);
                    low[nt][e] = static_cast<int>(see.low > base_token ? see.low - base_token : 0);
                    min_lim = min(min_lim, lim[nt][e]);
                    max_low = max(max_low, low[nt][e]);
                }
            }
        }
        min_lim = __reduce_min_sync(0xffffffffu, min_lim);
        max_low = __reduce_max_sync(0xffffffffu, max_low);
        if (!C::QREG) __syncthreads();

        float acc[GD][2][NT][4], m[NT][2], l[NT][2];
        int ref[GD];  // the group's largest scale byte of v so far
#pragma unroll
        for (int grp = 0; grp < GD; ++grp) {
            ref[grp] = -300;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[grp][k][nt][e] = 0.f;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) m[nt][e] = kNegInf, l[nt][e] = 0.f;

        // ---- tiles: a token a lane is looked up, copied, and its scale bytes fetched
        auto lookup = [&](int64_t tile) -> int64_t {
            const int64_t t = tile * tile_tokens + slice * TOK + lane;
            if (tile >= last || lane >= TOK || t < sl.low || t >= sl.high) return -1;
            const int64_t at = token_at(p, sl.b, t);
            if (at < 0) {
                atomicOr(p.status, 1u);
                return -1;
            }
            return at + head_off;
        };
        auto copy = [&](int stage, int64_t at) {
            const uint32_t to = smem_at(ring + stage * C::STAGE);
            if (!r.narrow) {
                constexpr int CH = RB / 16;
#pragma unroll
                for (int k = 0; k < TOK * CH / 32; ++k) {
                    const int i = lane + 32 * k, row = i / CH, c = i - row * CH;
                    const int64_t h = __shfl_sync(0xffffffffu, at, row);
                    const int64_t off = (h < 0 ? 0 : h) * RB + c * 16;
                    copy_async16(to + row * PITCH + c * 16, kcodes + off, h >= 0);
                    copy_async16(to + TOK * PITCH + row * PITCH + c * 16, vcodes + off, h >= 0);
                }
            } else {
                const int words = p.code_bytes / 4;
                for (int row0 = 0; row0 < TOK; row0 += 4) {
                    const int row = row0 + (lane >> 3);
                    const int64_t h = __shfl_sync(0xffffffffu, at, row);
                    const int64_t off = (h < 0 ? 0 : h) * p.code_bytes;
                    for (int c = lane & 7; c < words; c += 8) {
                        copy_async4(to + row * PITCH + c * 4, kcodes + off + c * 4, h >= 0);
                        copy_async4(to + TOK * PITCH + row * PITCH + c * 4, vcodes + off + c * 4, h >= 0);
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // the scale bytes of a token, low byte first
        auto scales = [&](int which, int64_t at, uint32_t (&s)[2]) {
            s[0] = s[1] = 0;
            if (at < 0) return;
            const uint8_t* b = p.scales[which] + at * p.groups;
            if (r.vec_scales && GD == 4) {
                s[0] = __ldg(reinterpret_cast<const uint32_t*>(b));
            } else if (r.vec_scales && GD == 8) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(b));
                s[0] = v.x;
                s[1] = v.y;
            } else if (r.vec_scales && GD == 2) {
                s[0] = __ldg(reinterpret_cast<const uint16_t*>(b));
            } else {
#pragma unroll
                for (int k = 0; k < GD; ++k)
                    if (k < p.groups) s[k >> 2] |= static_cast<uint32_t>(__ldg(b + k)) << (8 * (k & 3));
            }
        };

        int64_t at = lookup(first), at_next = lookup(first + 1);
        uint32_t sk[2], sv[2];
        copy(0, at);
        scales(0, at, sk);
        scales(1, at, sv);
        int stage = 0;
        for (int64_t tile = first; tile < last; ++tile) {
            const uint32_t there = __ballot_sync(0xffffffffu, at >= 0);
            // factors of the tile's tokens: 2^a for k; for v 2^(b - ref + LIFT)
            uint32_t bad = 0;  // groups of this lane's token whose v is not a number
            {
                float kf[FP], vf[FP];
#pragma unroll
                for (int grp = 0; grp < GD; ++grp) {
                    const uint32_t kb = (sk[grp >> 2] >> (8 * (grp & 3))) & 0xffu;
                    uint32_t vb = (sv[grp >> 2] >> (8 * (grp & 3))) & 0xffu;
                    if (vb == 255u) {
                        bad |= 1u << grp;
                        vb = 0;
                    }
                    kf[grp] = scale_of(kb);
                    const int most = static_cast<int>(__reduce_max_sync(0xffffffffu, vb));
                    if (most > ref[grp] + 3) {  // the sums move to the new largest scale
                        const float f = power(ref[grp] - most);
                        ref[grp] = most;
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[grp][k][nt][e] *= f;
                    }
                    vf[grp] = at >= 0 ? power(static_cast<int>(vb) - ref[grp] + C::LIFT) : 0.f;
                }
#pragma unroll
                for (int grp = GD; grp < FP; ++grp) kf[grp] = vf[grp] = 0.f;
                if (lane < TOK) {
#pragma unroll
                    for (int k = 0; k < FP; k += 2) {
                        *reinterpret_cast<float2*>(factors + lane * FP + k) = make_float2(kf[k], kf[k + 1]);
                        *reinterpret_cast<float2*>(factors + (TOK + lane) * FP + k) = make_float2(vf[k], vf[k + 1]);
                    }
                }
            }
            if (tile + 1 < last) {
                copy(stage ^ 1, at_next);
                scales(0, at_next, sk);
                scales(1, at_next, sv);
                at = at_next;
                at_next = lookup(tile + 2);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            __syncwarp();  // the tile's codes and factors are there for all lanes
            const unsigned char* kt = ring + stage * C::STAGE;
            const unsigned char* vt = kt + TOK * PITCH;

            // ---- scores, in powers of two
            float s[TM][NT][4];
#pragma unroll
            for (int mt = 0; mt < TM; ++mt) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
                const unsigned char* row = kt + (mt * 16 + gtok) * PITCH;
                const float* f0 = factors + (mt * 16 + gtok) * FP;
#pragma unroll
                for (int grp = 0; grp < GD; ++grp) {
                    uint32_t a[2][4];  // two instructions' codes
                    if (E4) {
                        const uint2 c0 = *reinterpret_cast<const uint2*>(row + grp * 32 + t4 * 8);
                        const uint2 c1 = *reinterpret_cast<const uint2*>(row + 8 * PITCH + grp * 32 + t4 * 8);
                        a[0][0] = pair_e4m3(c0.x), a[0][1] = pair_e4m3(c1.x);
                        a[0][2] = pair_e4m3(c0.x >> 16), a[0][3] = pair_e4m3(c1.x >> 16);
                        a[1][0] = pair_e4m3(c0.y), a[1][1] = pair_e4m3(c1.y);
                        a[1][2] = pair_e4m3(c0.y >> 16), a[1][3] = pair_e4m3(c1.y >> 16);
                    } else {
                        const uint32_t c0 = *reinterpret_cast<const uint32_t*>(row + grp * 16 + t4 * 4);
                        const uint32_t c1 = *reinterpret_cast<const uint32_t*>(row + 8 * PITCH + grp * 16 + t4 * 4);
                        a[0][0] = pair_e2m1(c0), a[0][1] = pair_e2m1(c1);
                        a[0][2] = pair_e2m1(c0 >> 8), a[0][3] = pair_e2m1(c1 >> 8);
                        a[1][0] = pair_e2m1(c0 >> 16), a[1][1] = pair_e2m1(c1 >> 16);
                        a[1][2] = pair_e2m1(c0 >> 24), a[1][3] = pair_e2m1(c1 >> 24);
                    }
                    const float fa = f0[grp], fb = f0[8 * FP + grp];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int ks = grp * 2 + k;
                            mma(d, a[k], C::QREG ? qreg[C::QREG ? ks : 0] : qs[(ks * NT + nt) * 32 + lane]);
                            if (NP == 2) mma(d, a[k], qs[(KS * NT + ks * NT + nt) * 32 + lane]);
                        }
                        s[mt][nt][0] = fmaf(d[0], fa, s[mt][nt][0]);
                        s[mt][nt][1] = fmaf(d[1], fa, s[mt][nt][1]);
                        s[mt][nt][2] = fmaf(d[2], fb, s[mt][nt][2]);
                        s[mt][nt][3] = fmaf(d[3], fb, s[mt][nt][3]);
                    }
                }
            }
            // ---- what is seen, and the running maximum
            const int t0 = static_cast<int>(tile - sl.tile0) * tile_tokens + slice * TOK;
            const bool masked = there != (TOK == 32 ? 0xffffffffu : 0xffffu) || t0 + TOK > min_lim || t0 < max_low;
            auto sees = [&](int mt, int half, int nt, int e) {
                const int tok = mt * 16 + half * 8 + gtok;
                return ((there >> tok) & 1u) && t0 + tok < lim[nt][e] && t0 + tok >= low[nt][e];
            };
            bool grow = false;
            float top[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float best = kNegInf;
#pragma unroll
                    for (int mt = 0; mt < TM; ++mt) {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float& v = s[mt][nt][half * 2 + e];
                            v *= col_scale[nt][e];
                            if (masked && !sees(mt, half, nt, e)) v = kNegInf;
                            best = fmaxf(best, v);
                        }
                    }
                    best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 4));
                    best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 8));
                    best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 16));
                    top[nt][e] = best;
                    grow |= best > m[nt][e] + 4.f;
                }
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float next = fmaxf(m[nt][e], top[nt][e]);
                        const float f = m[nt][e] == next ? 1.f : exp2_fast(m[nt][e] - next);
                        m[nt][e] = next;
                        l[nt][e] *= f;
#pragma unroll
                        for (int grp = 0; grp < GD; ++grp)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                acc[grp][k][nt][e] *= f;
                                acc[grp][k][nt][2 + e] *= f;
                            }
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float at0 = m[nt][e] == kNegInf ? 0.f : m[nt][e];
#pragma unroll
                    for (int mt = 0; mt < TM; ++mt) {
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float& v = s[mt][nt][half * 2 + e];
                            v = exp2_fast(v - at0);
                            l[nt][e] += v;
                        }
                    }
                }
            }
            // ---- groups of v that are not numbers reach the rows that see them (rare)
            if (__any_sync(0xffffffffu, bad != 0)) {
#pragma unroll
                for (int grp = 0; grp < GD; ++grp) {
                    const uint32_t which = __ballot_sync(0xffffffffu, (bad >> grp) & 1u);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            bool hit = false;
#pragma unroll
                            for (int mt = 0; mt < TM; ++mt)
#pragma unroll
                                for (int half = 0; half < 2; ++half)
                                    hit |= ((which >> (mt * 16 + half * 8 + gtok)) & 1u) && sees(mt, half, nt, e);
                            const uint32_t hits = __ballot_sync(0xffffffffu, hit);
                            if (hits & (0x11111111u << t4)) {
                                const float nan = __uint_as_float(0x7fc00000u);
#pragma unroll
                                for (int k = 0; k < 2; ++k) acc[grp][k][nt][e] = acc[grp][k][nt][2 + e] = nan;
                            }
                        }
                    }
                }
            }
            // ---- sums of v
#pragma unroll
            for (int mt = 0; mt < TM; ++mt) {
                const float* f0 = factors + (TOK + mt * 16 + gtok) * FP;
                const unsigned char* v0 = vt + (mt * 16 + vt0) * PITCH;
                const unsigned char* v1 = vt + (mt * 16 + vt1) * PITCH;
#pragma unroll
                for (int grp = 0; grp < GD; ++grp) {
                    uint32_t a[2][4];
                    if (E4) {
                        const int c = grp * 32 + g * 4;
                        const uint32_t wa = *reinterpret_cast<const uint32_t*>(v0 + c);
                        const uint32_t wb = *reinterpret_cast<const uint32_t*>(v1 + c);
                        const uint32_t wc = *reinterpret_cast<const uint32_t*>(v0 + 8 * PITCH + c);
                        const uint32_t wd = *reinterpret_cast<const uint32_t*>(v1 + 8 * PITCH + c);
                        const uint32_t p0 = __byte_perm(wa, wb, 0x5140), p1 = __byte_perm(wa, wb, 0x7362);
                        const uint32_t p2 = __byte_perm(wc, wd, 0x5140), p3 = __byte_perm(wc, wd, 0x7362);
                        a[0][0] = pair_e4m3(p0), a[0][1] = pair_e4m3(p0 >> 16);
                        a[0][2] = pair_e4m3(p2), a[0][3] = pair_e4m3(p2 >> 16);
                        a[1][0] = pair_e4m3(p1), a[1][1] = pair_e4m3(p1 >> 16);
                        a[1][2] = pair_e4m3(p3), a[1][3] = pair_e4m3(p3 >> 16);
                    } else {
                        const int c = grp * 16 + g * 2;
                        const uint32_t wa = *reinterpret_cast<const uint16_t*>(v0 + c);
                        const uint32_t wb = *reinterpret_cast<const uint16_t*>(v1 + c);
                        const uint32_t wc = *reinterpret_cast<const uint16_t*>(v0 + 8 * PITCH + c);
                        const uint32_t wd = *reinterpret_cast<const uint16_t*>(v1 + 8 * PITCH + c);
                        const uint32_t y0 = __byte_perm(wa, wc, 0x5410), y1 = __byte_perm(wb, wd, 0x5410);
                        const uint32_t even = (y0 & 0x0f0f0f0fu) | ((y1 << 4) & 0xf0f0f0f0u);
                        const uint32_t odd = ((y0 >> 4) & 0x0f0f0f0fu) | (y1 & 0xf0f0f0f0u);
                        a[0][0] = pair_e2m1(even), a[0][1] = pair_e2m1(odd);
                        a[0][2] = pair_e2m1(even >> 16), a[0][3] = pair_e2m1(odd >> 16);
                        a[1][0] = pair_e2m1(even >> 8), a[1][1] = pair_e2m1(odd >> 8);
                        a[1][2] = pair_e2m1(even >> 24), a[1][3] = pair_e2m1(odd >> 24);
                    }
                    const float fa = f0[grp], fb = f0[8 * FP + grp];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float x0 = s[mt][nt][0] * fa, x1 = s[mt][nt][1] * fa;
                        const float x2 = s[mt][nt][2] * fb, x3 = s[mt][nt][3] * fb;
                        const uint32_t h0 = half2_bits(x0, x1), h1 = half2_bits(x2, x3);
                        const uint2 b = make_uint2(transposed(h0), transposed(h1));
                        mma(acc[grp][0][nt], a[0], b);
                        mma(acc[grp][1][nt], a[1], b);
                        if (NP == 2) {
                            const float2 y0 = half2_values(h0), y1 = half2_values(h1);
                            const uint2 b2 = make_uint2(transposed(half2_bits(x0 - y0.x, x1 - y0.y)),
                                                        transposed(half2_bits(x2 - y1.x, x3 - y1.y)));
                            mma(acc[grp][0][nt], a[0], b2);
                            mma(acc[grp][1][nt], a[1], b2);
                        }
                    }
                }
            }
            __syncwarp();  // the stage and the factors are free again
            if (tile + 1 >= last) at = -1;
            stage ^= 1;
        }

        // ---- the warps of a head are joined, and the result or the part of it is written
        float* mine = reinterpret_cast<float*>(ring);  // [R][DP + 4], then maxima and sums
        float* ml = mine + R * (DP + 4);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[nt][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int row = nt * 8 + 2 * t4 + e;
                if (g == 0) {
                    ml[row] = m[nt][e];
                    ml[R + row] = sum;
                }
#pragma unroll
                for (int grp = 0; grp < GD; ++grp) {
                    // 2^(ref - 127 - LIFT) in two factors, which stay normal
                    const int ex = ref[grp] < 0 ? 0 : ref[grp] - 127 - C::LIFT;
                    const float f1 = power(ex / 2), f2_ = power(ex - ex / 2);
                    *reinterpret_cast<float4*>(mine + row * (DP + 4) + grp * 32 + g * 4) =
                        make_float4(acc[grp][0][nt][e] * f1 * f2_, acc[grp][0][nt][2 + e] * f1 * f2_,
                                    acc[grp][1][nt][e] * f1 * f2_, acc[grp][1][nt][2 + e] * f1 * f2_);
                }
            }
        }
        __syncthreads();
        const bool whole = !r.split || (begin <= slot_begin && before[slot + 1] <= end);
        // begun before this CTA: its part 2x; begun here and unfinished: 2x + 1
        const int part = 2 * x + (r.split && begin <= slot_begin ? 1 : 0);
        if (r.split && begin <= slot_begin && hblock == 0 && threadIdx.x == 0)
            r.entries[slot] = make_int2(x, static_cast<int>((before[slot + 1] - 1) / share));
        for (int u = w; u < r.hb * sl.rows; u += threads / 32) {
            const int hl = u % r.hb, row = u / r.hb;
            const float* from = reinterpret_cast<const float*>(sm + r.at_ring + hl * r.ring);
            const int stride = r.hb * r.ring / 4;  // to the next slice's warp of the head
            float M = kNegInf, L = 0.f;
            for (int k = 0; k < r.wph; ++k) M = fmaxf(M, from[k * stride + R * (DP + 4) + row]);
            float4 o[DP <= 128 ? 1 : 2];
#pragma unroll
            for (int k = 0; k < (DP <= 128 ? 1 : 2); ++k) o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < r.wph; ++k) {
                const float* f = from + k * stride;
                const float mk = f[R * (DP + 4) + row];
                const float wk = mk == kNegInf ? 1.f : exp2_fast(mk - M);  // no token: zeros
                L += wk * f[R * (DP + 4) + R + row];
#pragma unroll
                for (int c = 0; c < (DP <= 128 ? 1 : 2); ++c) {
                    const int d = lane * 4 + c * 128;
                    if (d >= DP) continue;
                    const float4 v = *reinterpret_cast<const float4*>(f + row * (DP + 4) + d);
                    o[c].x = fmaf(wk, v.x, o[c].x), o[c].y = fmaf(wk, v.y, o[c].y);
                    o[c].z = fmaf(wk, v.z, o[c].z), o[c].w = fmaf(wk, v.w, o[c].w);
                }
            }
            const int hk = hblock * r.hb + hl;
            if (!whole) {
                const int64_t at_part = (static_cast<int64_t>(part) * p.heads + hk) * R + row;
                if (lane == 0) r.ml[at_part] = make_float2(M, L);
#pragma unroll
                for (int c = 0; c < (DP <= 128 ? 1 : 2); ++c) {
                    const int d = lane * 4 + c * 128;
                    if (d < DP) *reinterpret_cast<float4*>(r.o + at_part * DP + d) = o[c];
                }
                continue;
            }
            const int64_t i = (sl.r0 + row) / p.G;
            const int qh = hk * p.G + static_cast<int>(sl.r0 + row - i * p.G);
            const int64_t out_row = sl.s.row0 + i;
            const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
            for (int c = 0; c < (DP <= 128 ? 1 : 2); ++c) {
                const int d = lane * 4 + c * 128;
                const float v[4] = {o[c].x, o[c].y, o[c].z, o[c].w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (d + e < p.D)
                        store_value<NP>(p.out.p, out_row * p.out.st + qh * p.out.sh + d + e, L == 0.f ? 0.f : v[e] * inv,
                                        p.dtype);
            }
            if (p.lse && lane == 0)
                p.lse[out_row * p.heads_q + qh] = L == 0.f ? kNegInf : (M + log2f(L)) * 0.6931471805599453f;
        }
        __syncthreads();  // the rings are free again
        if (r.narrow) {   // and what lies behind a token's codes is zero again
            for (int i = lane; i < 2 * C::STAGE / 16; i += 32)
                reinterpret_cast<uint4*>(ring)[i] = make_uint4(0u, 0u, 0u, 0u);
            __syncwarp();
        }
    }
}

template <int F, int GD, int NT, int NP>
cudaError_t launch_rows(const AttnP& p, RowsPlan r, const OpCfg& c) {
    using C = Rows<F, GD, NT, NP>;
    auto fn = attn_rows_kernel<F, GD, NT, NP>;
    const int warps = r.hb * r.wph;
    r.ring = C::ring_bytes();
    r.at_q = 0;
    r.at_factors = r.at_q + r.hb * C::q_bytes();
    r.at_ring = r.at_factors + warps * C::factor_bytes();
    r.at_plan = r.at_ring + warps * r.ring;
    r.smem = r.at_plan + (r.split ? (r.slots + 1) * 8 : 0);
    if (r.smem + 1024 > c.dev.max_smem_optin) return cudaErrorInvalidConfiguration;
    const cudaError_t e =
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, c.dev.max_smem_optin - 1024);
    if (e != cudaSuccess) return e;
    return op_launch(c, fn, static_cast<int64_t>(r.gx) * r.head_blocks, warps * 32, r.smem, p, r);
}

template <int F, int NP, int GD>
cudaError_t pick_rows(const AttnP& p, const RowsPlan& r, const OpCfg& c) {
    if (r.nt == 1) return launch_rows<F, GD, 1, NP>(p, r, c);
    if constexpr (GD <= 4) {
        if (r.nt == 4) return launch_rows<F, GD, 4, NP>(p, r, c);
    }
    return launch_rows<F, GD, 2, NP>(p, r, c);
}

template <int F, int NP>
cudaError_t pick_groups(const AttnP& p, const RowsPlan& r, const OpCfg& c) {
    switch (r.gd) {
        case 2: return pick_rows<F, NP, 2>(p, r, c);
        case 3: return pick_rows<F, NP, 3>(p, r, c);
        case 4: return pick_rows<F, NP, 4>(p, r, c);
        case 6: return pick_rows<F, NP, 6>(p, r, c);
        default: return pick_rows<F, NP, 8>(p, r, c);
    }
}

}  // namespace
}  // namespace rmsn
