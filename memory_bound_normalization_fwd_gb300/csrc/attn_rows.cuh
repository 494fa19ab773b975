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
// value. For V the token's largest scale goes to the probabilities,
//   o[d, r] += (c[t, d] 2^(b[t, g] - b[t] + C)) * (2^(b[t] - B + 8) p[t, r])
// relative to the largest scale B so far, where 22 powers of two below the largest are full fp16
// values and 32 are kept in part; what the groups of a token differ by goes to the codes, by
// packed fp16 products (exact down to 2^-(C + 15) of the token's largest scale, kept in part
// to 2^-(C + 24); C is 6 for 8-bit codes, 12 for 4-bit ones). (A scale per group on the
// probabilities took a conversion and a transposition for every group and block of 8 rows: one
// key head of 256 values in 8 bits, 16 rows, 52.6 us.)
// Both products take the codes as the first operand (16 tokens x 16 values of K; 16 values
// x 16 tokens of V) and 8 rows as the second, so a row costs an eighth of an instruction and no
// lane idles for 8 rows. A token's probabilities for the second product come from the first one's
// sums by an 8x8 transposition in registers.
// Order of values: the sum over d, the sum over t and the place of d in the result may be permuted
// at will, as long as both operands agree. So codes come by ldmatrix, which hands a lane the bytes of
// a token (K) or, transposed, the bytes of two neighbouring tokens at one place (V); the
// bytes of two tokens are paired by permutations of words, and one conversion instruction
// makes a pair of fp16 values. Tokens lie an odd number of 16 bytes apart, on different banks.
//
// Each warp runs on its own: a ring of two tiles, filled by asynchronous copies of 16 bytes (a token's
// row of codes at a time), no barrier in the loop; page numbers are looked up two tiles ahead,
// scale bytes travel through registers one tile ahead. Softmax with a running maximum, which moves
// only where a score exceeds it by more than 2^4 (the sums then carry factors up to 2^4).
// Bound (GB300): the latency of a warp's instructions; no unit is full. 32 sequences of up to 8192 tokens, 32
// query heads on 8 of 128 values in 4 bits, 144 MB, 48 us, 45% of the rate of a copy: issue slots 57%,
// integer and conversion units 47% (each of their instructions takes two cycles), matrix units 18%, four
// warps a scheduler; about 650 instructions a tile of 32 tokens and 1800 a slot. With q and the
// probabilities in two pieces, as fp32 calls have them, 55 us: 16-bit outputs take one of 11 bits, whose
// error bf16's own rounding hides (relative to 64 bits 0.0017 with either) and fp16's nearly (0.00024 for
// 0.00021). Two sequences of up to 131072 tokens, 16 query heads on one of 256 values
// in 8 bits, 131 MB, 46 us: 2 warps a scheduler, which the sums in registers allow, issue 33% of the time.
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
// Pairs of fp16 values from the codes of a word, low bytes first.
__device__ __forceinline__ void pairs_e4m3(uint32_t c, uint32_t& d0, uint32_t& d1) {
    asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
        : "=r"(d0), "=r"(d1)
        : "r"(c));
}
__device__ __forceinline__ void pairs_e2m1(uint32_t c, uint32_t& d0, uint32_t& d1, uint32_t& d2, uint32_t& d3) {
    asm("{ .reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4; cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b; "
        "cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d; }"
        : "=r"(d0), "=r"(d1), "=r"(d2), "=r"(d3)
        : "r"(c));
}
// The low four bits of a's bytes, the high four of b's.
__device__ __forceinline__ uint32_t low_nibbles(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, 0x0f0f0f0f, 0xe4;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ const uint8_t* plus(const uint8_t* p, uint32_t n, uint32_t times) {
    uint64_t r;
    asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(r) : "r"(n), "r"(times), "l"(reinterpret_cast<uint64_t>(p)));
    return reinterpret_cast<const uint8_t*>(r);
}
// 8x8 matrices of 16-bit units; lane l gives row l % 8 of matrix l / 8.
template <bool TRANS>
__device__ __forceinline__ void load4(uint32_t (&r)[4], uint32_t at) {
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
template <bool TRANS>
__device__ __forceinline__ void load2(uint32_t (&r)[4], uint32_t at) {
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at) : "memory");
}

// d += a b: a 16x16 (rows lane / 4 and that + 8), b 16x8, fp16 in, fp32 sums.
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint2& b) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y));
}
// d = a b.
__device__ __forceinline__ void mma_new(float (&d)[4], const uint32_t (&a)[4], const uint2& b) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y), "f"(0.f));
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
template <int FP>
__device__ __forceinline__ void load_factors(float (&f)[FP], const float* from) {
    if constexpr (FP == 2) {
        const float2 v = *reinterpret_cast<const float2*>(from);
        f[0] = v.x, f[1] = v.y;
    } else {
#pragma unroll
        for (int k = 0; k < FP; k += 4) {
            const float4 v = *reinterpret_cast<const float4*>(from + k);
            f[k] = v.x, f[k + 1] = v.y, f[k + 2] = v.z, f[k + 3] = v.w;
        }
    }
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ bool at_there(uint32_t there, int lane) { return (there >> lane) & 1u; }
// 2^e as fp32, 0 below 2^-126 (e <= 127).
__device__ __forceinline__ float power(int e) { return __uint_as_float(e < -126 ? 0u : static_cast<uint32_t>(e + 127) << 23); }

// A block of rows of a sequence, and the tiles of tokens that it sees. (Numbers of rows, tokens
// and tiles are below 2^31.)
struct Slot {
    int b, row0, n, len;  // the sequence, its first row, its rows and tokens
    int held;             // tokens that the row of the table has room for
    int r0;               // first row of the block among the sequence's (queries times G)
    int rows;             // 0: no such slot
    int low, high;        // tokens that any of its rows sees
    int tile0;            // the first tile
    int tiles;            // at least one where there are rows
};

__device__ __forceinline__ int divide(int a, uint32_t mul, int shift) {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(a)) * mul >> shift);
}

// First rows and lengths of the sequences: in shared memory where the slots are split.
struct Sequences {
    const int* row0;  // null: read from the call's arrays
    const int* len;
    __device__ __forceinline__ int row(const AttnP& p, int b) const {
        return row0 ? row0[b] : static_cast<int>(first_row(p, b));
    }
    __device__ __forceinline__ int length(const AttnP& p, int b) const {
        return row0 ? len[b] : static_cast<int>(sequence(p, b).len);
    }
};

// Tokens that query i sees.
__device__ __forceinline__ void seen32(const AttnP& p, const RowsPlan& r, int n, int len, int i, int& low, int& high) {
    const int pos = len - n + i;
    high = p.causal ? max(pos + 1, 0) : len;
    low = r.window && pos + 1 > r.window ? pos + 1 - r.window : 0;
}

template <int R>
__device__ __forceinline__ Slot slot_of(const AttnP& p, const RowsPlan& r, const Sequences& q, int slot) {
    auto start = [&](int b) { return q.row(p, b) * p.G / R + b; };  // rows * G is below 2^31
    int lo = 0, hi = static_cast<int>(p.sequences) - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start(mid) <= slot) lo = mid;
        else hi = mid - 1;
    }
    Slot s;
    s.b = lo;
    s.row0 = q.row(p, lo);
    s.n = max(q.row(p, lo + 1) - s.row0, 0);
    s.len = q.length(p, lo);
    s.held = min(s.len, r.most_tokens);
    const int first = s.row0 * p.G / R + lo, all = s.n * p.G;
    s.r0 = (slot - first) * R;
    s.rows = s.low = s.high = s.tile0 = s.tiles = 0;
    if (slot < first || s.r0 >= all) return s;
    s.rows = min(all - s.r0, R);
    int unused;
    seen32(p, r, s.n, s.len, divide(s.r0, r.g_mul, r.g_shift), s.low, unused);
    seen32(p, r, s.n, s.len, divide(s.r0 + s.rows - 1, r.g_mul, r.g_shift), unused, s.high);
    s.high = min(s.high, s.held);
    s.tile0 = s.low >> r.tile_shift;
    s.tiles = s.high > s.low ? ((s.high - 1) >> r.tile_shift) + 1 - s.tile0 : 1;
    return s;
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
    static constexpr int CODE = E4 ? 6 : 12;  // C above
    static __host__ __device__ constexpr int factor_bytes() { return TOK * FP * 4 + TOK * 4 + (GD + 1) / 2 * 2 * TOK * 2; }
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
// Values d and d + 1 of a row at `at` (of D; `vec`: rows start on vectors' borders).
template <int NP>
__device__ __forceinline__ void store_two(void* p, int64_t at, int d, float a, float b, int D, bool vec, int dtype) {
    if (d >= D) return;
    if (vec && d + 2 <= D) {
        if (NP == 2) *reinterpret_cast<float2*>(static_cast<float*>(p) + at + d) = make_float2(a, b);
        else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p) + at + d) =
            dtype == kBF16 ? Codec<kBF16>::pack2(a, b) : Codec<kFP16>::pack2(a, b);
        return;
    }
    for (int k = 0; k < 2; ++k) {
        if (d + k >= D) return;
        const float v = k ? b : a;
        if (NP == 2) store1<kFP32>(p, at + d + k, v);
        else if (dtype == kBF16) store1<kBF16>(p, at + d + k, v);
        else store1<kFP16>(p, at + d + k, v);
    }
}

template <int F, int GD, int NT, int NP>
__global__ void __launch_bounds__(256, Rows<F, GD, NT, NP>::CTAS) attn_rows_kernel(const AttnP p, const RowsPlan r) {
    using C = Rows<F, GD, NT, NP>;
    constexpr bool E4 = C::E4;
    constexpr int DP = C::DP, RB = C::RB, PITCH = C::PITCH, TM = C::TM, TOK = C::TOK, FP = C::FP, R = C::R, KS = C::KS;
    constexpr float kNegInf = -INFINITY;
    constexpr uint32_t kNone = 0xffffffffu;  // no token
    constexpr uint32_t kAll = TOK == 32 ? 0xffffffffu : 0xffffu;
    constexpr int W = (GD + 3) / 4;
    extern __shared__ __align__(128) unsigned char sm[];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t4 = lane & 3;
    const int head_local = w % r.hb, slice = w / r.hb, threads = blockDim.x;
    const int x = static_cast<int>(blockIdx.x) / r.head_blocks, hblock = static_cast<int>(blockIdx.x) - x * r.head_blocks;
    const int head = hblock * r.hb + head_local;
    unsigned char* ring = sm + r.at_ring + w * r.ring;
    float* factors = reinterpret_cast<float*>(sm + r.at_factors + w * C::factor_bytes());
    uint2* qs = reinterpret_cast<uint2*>(sm + r.at_q + head_local * C::q_bytes());
    int* before = reinterpret_cast<int*>(sm + r.at_plan);  // tiles before each slot
    Sequences seq{nullptr, nullptr};
    if (r.narrow) {  // what lies behind a token's codes stays zero
        for (int i = lane; i < 2 * C::STAGE / 16; i += 32) reinterpret_cast<uint4*>(ring)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncwarp();  // before other lanes' copies go there
    }
    pdl_wait();
    pdl_launch_dependents();

    // Which tiles are this CTA's.
    int begin = 0, end = 0, share = 1, slot = x;
    if (r.split) {
        __shared__ int warp_tiles[8];
        int* rows = before + r.slots + 1;
        int* lens = rows + p.sequences + 1;
        for (int b = threadIdx.x; b <= p.sequences; b += threads) {
            rows[b] = static_cast<int>(first_row(p, b));
            if (b < p.sequences) lens[b] = max(__ldg(p.lengths + b), 0);
        }
        seq = Sequences{rows, lens};
        __syncthreads();
        const int run = (r.slots + threads - 1) / threads;
        const int run0 = min(static_cast<int>(threadIdx.x) * run, r.slots), run1 = min(run0 + run, r.slots);
        int own = 0;
        for (int i = run0; i < run1; ++i) {
            // a slot's start counts as some tiles: what a CTA spends on another slot beside its tiles
            const int tiles = slot_of<R>(p, r, seq, i).tiles, n = tiles ? tiles + r.start_tiles : 0;
            before[i + 1] = n;
            own += n;
        }
        int sum = own;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += o;
        }
        if (lane == 31) warp_tiles[w] = sum;
        __syncthreads();
        sum -= own;
        int total = 0;
        for (int i = 0; i < threads / 32; ++i) {
            if (i < w) sum += warp_tiles[i];
            total += warp_tiles[i];
        }
        if (threadIdx.x == 0) before[0] = 0;
        for (int i = run0; i < run1; ++i) {
            sum += before[i + 1];
            before[i + 1] = sum;
        }
        __syncthreads();
        share = static_cast<int>((static_cast<uint32_t>(total) + r.gx - 1) / r.gx);
        const int64_t from = static_cast<int64_t>(share) * x;
        if (x == 0 && hblock == 0)  // slots without rows have no parts to join
            for (int i = run0; i < run1; ++i)
                if (before[i + 1] == before[i]) r.entries[i] = make_int4(-1, 0, 0, 0);
        if (from >= total) return;
        begin = static_cast<int>(from);
        end = share < total - begin ? begin + share : total;
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
    const uint32_t head_off = static_cast<uint32_t>(head * head_step(p));
    // a lane's row of the matrices that ldmatrix takes from 16 tokens: two of 8 tokens of a 16-byte
    // piece, two of the next piece
    const uint32_t mat = (lane & 15) * PITCH + (lane >> 4) * 16;

    for (; slot < r.slots; slot += r.split ? 1 : r.gx) {
        if (r.split && before[slot] >= end) break;
        const Slot sl = slot_of<R>(p, r, seq, slot);
        if (sl.rows == 0) continue;
        if (sl.len > sl.held && threadIdx.x == 0) atomicOr(p.status, 1u);  // tokens past the table's row
        int first = 0, last = sl.tiles, slot_begin = 0;
        if (r.split) {
            slot_begin = before[slot] + r.start_tiles;
            first = max(begin - slot_begin, 0);
            last = min(before[slot + 1], end) - slot_begin;
            if (first >= last) continue;  // only a part of its start
        }
        first += sl.tile0;
        last += sl.tile0;
        const int32_t* table = p.table + sl.b * p.width;

        // ---- tiles: a token a lane is looked up, copied, and its scale bytes fetched
        // (in two steps, a tile apart: the page's number is on its way in between)
        auto token = [&](int tile) { return (tile << r.tile_shift) + slice * TOK + lane; };
        auto page_of = [&](int tile) -> uint32_t {
            const int t = token(tile);
            if (tile >= last || lane >= TOK || t < sl.low || t >= sl.high) return kNone;
            return static_cast<uint32_t>(__ldg(table + divide(t, r.page_mul, r.page_shift)));
        };
        auto place = [&](int tile, uint32_t page) -> uint32_t {
            if (page >= r.pages) {
                const int t = token(tile);  // a token that is seen, on a page that is not there
                if (tile < last && lane < TOK && t >= sl.low && t < sl.high) atomicOr(p.status, 1u);
                return kNone;
            }
            const uint32_t t = token(tile), off = t - divide(t, r.page_mul, r.page_shift) * p.page_size;
            return (p.heads_first ? page * p.heads * p.page_size + off : (page * p.page_size + off) * p.heads) + head_off;
        };
        auto copy = [&](int stage, uint32_t at, uint32_t there) {
            const uint32_t to = smem_at(ring + stage * C::STAGE);
            if (!r.narrow) {
                constexpr int CH = RB / 16;
                const uint32_t own = at == kNone ? 0 : at;  // nothing is read for a token that is not there
#pragma unroll
                for (int k = 0; k < TOK * CH / 32; ++k) {
                    const int i = lane + 32 * k, row = i / CH, c = i - row * CH;
                    const uint32_t h = __shfl_sync(0xffffffffu, own, row);
                    const uint32_t dst = to + row * PITCH + c * 16;
                    const uint8_t *kfrom = plus(kcodes + c * 16, h, RB), *vfrom = plus(vcodes + c * 16, h, RB);
                    if (there == kAll) {
                        copy_async16(dst, kfrom, true);
                        copy_async16(dst + TOK * PITCH, vfrom, true);
                    } else {
                        const bool some = (there >> row) & 1u;
                        copy_async16(dst, kfrom, some);
                        copy_async16(dst + TOK * PITCH, vfrom, some);
                    }
                }
            } else {
                for (int row0 = 0; row0 < TOK; row0 += 4) {
                    const int row = row0 + (lane >> 3);
                    const uint32_t h = __shfl_sync(0xffffffffu, at, row);
                    const bool some = h != kNone;
                    const uint64_t off = some ? static_cast<uint64_t>(h) * p.code_bytes : 0;
                    const uint8_t *kfrom = kcodes + off, *vfrom = vcodes + off;
                    const uint32_t dst = to + row * PITCH;
                    for (int c = (lane & 7) * r.narrow; c < p.code_bytes; c += 8 * r.narrow) {
                        if (r.narrow == 16) {
                            copy_async16(dst + c, kfrom + c, some);
                            copy_async16(dst + TOK * PITCH + c, vfrom + c, some);
                        } else {
                            copy_async4(dst + c, kfrom + c, some);
                            copy_async4(dst + TOK * PITCH + c, vfrom + c, some);
                        }
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // Bits before a token's scale bytes in the words that are read for them.
        auto scale_place = [&](uint32_t at) -> uint32_t { return at * static_cast<uint32_t>(p.groups) % 4 * 8; };
        auto shifted = [&](uint32_t (&s)[2], uint32_t shift) {
            s[0] = __funnelshift_r(s[0], s[1], shift);
            if (GD == 3) s[0] &= 0xffffffu, s[1] = 0;
            else s[1] = s[1] >> shift & 0xffffu;
        };
        // the scale bytes of a token, low byte first
        auto scales = [&](int which, uint32_t at, uint32_t (&s)[2]) {
            s[0] = s[1] = 0;
            if (at == kNone) return;
            const uint8_t* b = p.scales[which] + static_cast<uint64_t>(at) * p.groups;
            if (r.vec_scales && GD == 4) {
                s[0] = __ldg(reinterpret_cast<const uint32_t*>(b));
            } else if (r.vec_scales && GD == 8) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(b));
                s[0] = v.x;
                s[1] = v.y;
            } else if (r.vec_scales && GD == 2) {
                s[0] = __ldg(reinterpret_cast<const uint16_t*>(b));
            } else if (r.vec_scales && (GD == 3 || GD == 6)) {
                // the words that hold them (the array is whole words), shifted where they are used: there
                // the loads have arrived (GB300, us, 32 sequences of 8192 tokens, 8 heads in 4 bits, shifted
                // here / there: 96 values 97 / 72, 192 values 281 / 163)
                const uint32_t* words = reinterpret_cast<const uint32_t*>(b - scale_place(at) / 8);
                s[0] = __ldg(words);
                if (GD == 6 || scale_place(at) > 8) s[1] = __ldg(words + 1);
            } else {
#pragma unroll
                for (int k = 0; k < GD; ++k)
                    if (k < p.groups) s[k >> 2] |= static_cast<uint32_t>(__ldg(b + k)) << (8 * (k & 3));
            }
        };

        const uint32_t page0 = page_of(first);
        uint32_t page = page_of(first + 1);
        const uint32_t at = place(first, page0);
        uint32_t there_next = __ballot_sync(0xffffffffu, at != kNone);
        uint32_t sk[2], sv[2];
        copy(0, at, there_next);
        scales(0, at, sk);
        scales(1, at, sv);
        uint32_t shift = scale_place(at);

        // ---- q: a row's largest magnitude, its power of two, and its values as fp16 operands
        uint2 qreg[C::QREG ? KS : 1];
        float col_scale[NT][2];
        int lim[NT][2], low[NT][2];  // tokens that a column's row sees, relative to the slot's first tile
        const int base_token = sl.tile0 << r.tile_shift;
        int min_lim = INT32_MAX, max_low = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int rr = nt * 8 + g;
            const bool live = rr < sl.rows;
            const int i = live ? divide(sl.r0 + rr, r.g_mul, r.g_shift) : 0;
            const int qh = head * p.G + (live ? sl.r0 + rr - i * p.G : 0);
            const int64_t at = (sl.row0 + i) * p.q.st + qh * p.q.sh;
            // the values of K that the lane gets in two instructions of a group, four each
            float v[GD][8];
            float top = 0.f;
            if (r.vec_q && p.D == DP) {  // no branch: a row past the block's takes the first one's values, times 0
                const unsigned char* src = static_cast<const unsigned char*>(p.q.p) + at * (NP == 2 ? 4 : 2);
                if (NP == 2) {
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        const int d = (k >> 1) * 32 + (E4 ? (k & 1) * 16 + t4 * 4 : t4 * 8 + (k & 1) * 4);
                        const float4 f = __ldg(reinterpret_cast<const float4*>(src + d * 4));
                        float* to = &v[k >> 1][(k & 1) * 4];
                        to[0] = f.x, to[1] = f.y, to[2] = f.z, to[3] = f.w;
                    }
                } else {
                    uint2 u[KS];
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        const int d = (k >> 1) * 32 + (E4 ? (k & 1) * 16 + t4 * 4 : t4 * 8 + (k & 1) * 4);
                        u[k] = __ldg(reinterpret_cast<const uint2*>(src + d * 2));
                    }
                    const bool bf16 = p.dtype == kBF16;
                    if (bf16) {
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            const float2 a = unpack16(u[k].x, true), b = unpack16(u[k].y, true);
                            float* to = &v[k >> 1][(k & 1) * 4];
                            to[0] = a.x, to[1] = a.y, to[2] = b.x, to[3] = b.y;
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            const float2 a = unpack16(u[k].x, false), b = unpack16(u[k].y, false);
                            float* to = &v[k >> 1][(k & 1) * 4];
                            to[0] = a.x, to[1] = a.y, to[2] = b.x, to[3] = b.y;
                        }
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const int d = (k >> 1) * 32 + (E4 ? (k & 1) * 16 + t4 * 4 : t4 * 8 + (k & 1) * 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[k >> 1][(k & 1) * 4 + e] = live && d + e < p.D ? load_value<NP>(p.q.p, at + d + e, p.dtype) : 0.f;
                }
            }
#pragma unroll
            for (int grp = 0; grp < GD; ++grp)
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[grp][e]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            int ex = static_cast<int>(__float_as_uint(top) >> 23);
            ex = top == 0.f ? 141 : ex < 15 ? 15 : ex;  // both powers stay normal
            const float up = live ? __uint_as_float(static_cast<uint32_t>(268 - ex) << 23) : 0.f;
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
                    int from, to;
                    seen32(p, r, sl.n, sl.len, divide(sl.r0 + cr, r.g_mul, r.g_shift), from, to);
                    lim[nt][e] = max(min(to, sl.held) - base_token, 0);
                    low[nt][e] = max(from - base_token, 0);
                    min_lim = min(min_lim, lim[nt][e]);
                    max_low = max(max_low, low[nt][e]);
                }
            }
        }
        min_lim = __reduce_min_sync(0xffffffffu, min_lim);
        max_low = __reduce_max_sync(0xffffffffu, max_low);
        if (!C::QREG) {
            if (r.wph == 1) __syncwarp();
            else __syncthreads();
        }

        // base: what scores are taken relative to (0 before a row has seen a token); limit: where
        // above it a score moves it (2^4; -infinity before)
        float acc[GD][2][NT][4], base[NT][2], limit[NT][2], l[NT][2];
        uint32_t ref = 0, most = 3;  // v's largest scale byte so far, and the most that it serves for
#pragma unroll
        for (int grp = 0; grp < GD; ++grp)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[grp][k][nt][e] = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) base[nt][e] = l[nt][e] = 0.f, limit[nt][e] = kNegInf;

        int stage = 0;
        for (int tile = first; tile < last; ++tile) {
            const uint32_t there = there_next;
            // factors of the tile's tokens: 2^a for k; for v 2^(b - ref + LIFT), b the token's largest
            // byte, and 2^(the group's byte - b + CODE) in fp16. Two groups at a time, in halves of 16 bits.
            uint32_t bad = 0;  // groups of this lane's token whose v is not a number
            if ((GD == 3 || GD == 6) && r.vec_scales) {
                shifted(sk, shift);
                shifted(sv, shift);
            }
            {
                constexpr uint32_t kBoth = 0x00010001u;
                uint32_t x[W][2], y[W][2], e[W][2];  // bytes 0 and 2, and 1 and 3, of k's and v's scales
                uint32_t kmax = 0, vmax = 0;
#pragma unroll
                for (int i = 0; i < W; ++i) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        x[i][h] = (sk[i] >> (8 * h)) & 0x00ff00ffu;
                        y[i][h] = (sv[i] >> (8 * h)) & 0x00ff00ffu;
                        kmax = __vmaxu2(kmax, x[i][h]);
                        vmax = __vmaxu2(vmax, y[i][h]);
                    }
                }
                uint32_t b = max(vmax & 0xffffu, vmax >> 16);
                // a byte - b + CODE + 15 as fp16's exponent, at least 0 (a bias of 256 keeps the
                // halves apart)
                uint32_t least = 0xffffffffu;
                auto exponents = [&]() {
                    least = 0xffffffffu;
#pragma unroll
                    for (int i = 0; i < W; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            e[i][h] = __vmaxu2(y[i][h] + kBoth * (256 + C::CODE + 15) - kBoth * b, kBoth * 256) - kBoth * 256;
                            // (groups that are not there do not count)
                            const int g0 = i * 4 + h;
                            least = __vminu2(least, e[i][h] | (g0 < GD ? 0u : 0xffffu) | (g0 + 2 < GD ? 0u : 0xffff0000u));
                        }
                };
                exponents();
                uint32_t odd = 0;  // groups whose k is not a number
                const bool rare = b > most || (least & 0xffffu) == 0 || least < 0x10000u || (kmax & 0xffffu) == 255u ||
                                  kmax >= 0xff0000u;
                const bool slow = __any_sync(0xffffffffu, rare && at_there(there, lane));
                if (slow) {
                    b = 0;
#pragma unroll
                    for (int grp = 0; grp < GD; ++grp) {
                        const int i = grp >> 2, h = grp & 1, sh = (grp & 2) * 8;
                        if (((x[i][h] >> sh) & 0xffffu) == 255u) odd |= 1u << grp;
                        if (((y[i][h] >> sh) & 0xffffu) == 255u) {
                            bad |= 1u << grp;
                            y[i][h] &= ~(0xffffu << sh);
                        }
                        b = max(b, (y[i][h] >> sh) & 0xffffu);
                    }
                    exponents();
                    const uint32_t top = __reduce_max_sync(0xffffffffu, b);
                    if (top > ref + 3) {  // the sums move to the new largest scale
                        const float f = power(static_cast<int>(ref) - static_cast<int>(top));
                        ref = top;
                        most = min(top + 3, 254u);
#pragma unroll
                        for (int grp = 0; grp < GD; ++grp)
#pragma unroll
                            for (int k = 0; k < 2; ++k)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int q = 0; q < 4; ++q) acc[grp][k][nt][q] *= f;
                    }
                }
                if (lane < TOK) {
                    float kf[FP];
                    uint16_t* hf = reinterpret_cast<uint16_t*>(factors + TOK * FP + TOK) + lane;
#pragma unroll
                    for (int grp = 0; grp < FP; ++grp) {
                        const int i = grp >> 2, h = grp & 1;
                        kf[grp] = 0.f;
                        if (i >= W || grp >= GD) continue;
                        // (byte 0: 2^-127, below the normal values)
                        kf[grp] = __uint_as_float(max(grp & 2 ? (x[i][h] & 0xffff0000u) << 7 : x[i][h] << 23, 0x400000u));
                        uint32_t half = (grp & 2 ? e[i][h] >> 16 : e[i][h] & 0xffffu) << 10;
                        if (slow) {
                            if (odd >> grp & 1u) kf[grp] = __uint_as_float(0x7fc00000u);
                            // below fp16's normal values
                            const int low = static_cast<int>(y[i][h] >> (grp & 2) * 8 & 0xffffu) - static_cast<int>(b) + C::CODE;
                            if (low < -14) half = low >= -24 ? 1u << (low + 24) : 0u;
                        }
                        hf[grp * TOK] = static_cast<uint16_t>(half);
                    }
#pragma unroll
                    for (int k = 0; k < FP; k += 2)
                        *reinterpret_cast<float2*>(factors + lane * FP + k) = make_float2(kf[k], kf[k + 1]);
                    const int ex = static_cast<int>(b) - static_cast<int>(ref) + C::LIFT + 127;
                    factors[TOK * FP + lane] = __uint_as_float(static_cast<uint32_t>(max(ex, 0)) << 23);
                }
            }
            if (tile + 1 < last) {
                const uint32_t next = place(tile + 1, page);
                there_next = __ballot_sync(0xffffffffu, next != kNone);
                copy(stage ^ 1, next, there_next);
                scales(0, next, sk);
                scales(1, next, sv);
                shift = scale_place(next);
                page = page_of(tile + 2);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
            } else {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
            }
            __syncwarp();  // the tile's codes and factors are there for all lanes

            // ---- scores, in powers of two, relative to the rows' bases
            float s[TM][NT][4];
            const uint32_t kt = smem_at(ring + stage * C::STAGE) + mat, vt = kt + TOK * PITCH;
#pragma unroll
            for (int mt = 0; mt < TM; ++mt) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
                float fa[FP], fb[FP];
                load_factors<FP>(fa, factors + (mt * 16 + g) * FP);
                load_factors<FP>(fb, factors + (mt * 16 + 8 + g) * FP);
                uint32_t c[4];
#pragma unroll
                for (int grp = 0; grp < GD; ++grp) {
                    uint32_t a[2][4];  // two instructions' codes
                    const uint32_t from = kt + mt * 16 * PITCH + grp * (E4 ? 32 : 16);
                    if (E4) {
                        load4<false>(c, from);
                        pairs_e4m3(c[0], a[0][0], a[0][2]);
                        pairs_e4m3(c[1], a[0][1], a[0][3]);
                        pairs_e4m3(c[2], a[1][0], a[1][2]);
                        pairs_e4m3(c[3], a[1][1], a[1][3]);
                    } else {
                        if (grp % 2 == 0 && grp + 1 < GD) load4<false>(c, from);
                        else if (grp % 2 == 0) load2<false>(c, from);
                        const int k = grp % 2 * 2;
                        pairs_e2m1(c[k], a[0][0], a[0][2], a[1][0], a[1][2]);
                        pairs_e2m1(c[k + 1], a[0][1], a[0][3], a[1][1], a[1][3]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float d[4];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int ks = grp * 2 + k;
                            const uint2 b = C::QREG ? qreg[C::QREG ? ks : 0] : qs[(ks * NT + nt) * 32 + lane];
                            if (k == 0) mma_new(d, a[k], b);
                            else mma(d, a[k], b);
                            if (NP == 2) mma(d, a[k], qs[(KS * NT + ks * NT + nt) * 32 + lane]);
                        }
                        // (not in pairs: a factor for two would have to be copied)
                        s[mt][nt][0] = fmaf(d[0], fa[grp], s[mt][nt][0]);
                        s[mt][nt][1] = fmaf(d[1], fa[grp], s[mt][nt][1]);
                        s[mt][nt][2] = fmaf(d[2], fb[grp], s[mt][nt][2]);
                        s[mt][nt][3] = fmaf(d[3], fb[grp], s[mt][nt][3]);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[mt][nt][e] = fmaf(s[mt][nt][e], col_scale[nt][e & 1], -base[nt][e & 1]);
                }
            }
            // ---- what is seen, and the running maximum
            const int t0 = ((tile - sl.tile0) << r.tile_shift) + slice * TOK;
            const bool masked = there != kAll || t0 + TOK > min_lim || t0 < max_low;
            auto sees = [&](int mt, int half, int nt, int e) {
                const int tok = mt * 16 + half * 8 + g;
                return ((there >> tok) & 1u) && t0 + tok < lim[nt][e] && t0 + tok >= low[nt][e];
            };
            if (masked) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int mt = 0; mt < TM; ++mt)
#pragma unroll
                            for (int half = 0; half < 2; ++half)
                                if (!sees(mt, half, nt, e)) s[mt][nt][half * 2 + e] = kNegInf;
            }
            bool grow = false;
            float top[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[nt][e] = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
                    if (TM == 2) top[nt][e] = fmaxf(top[nt][e], fmaxf(s[TM - 1][nt][e], s[TM - 1][nt][2 + e]));
                    grow |= top[nt][e] > limit[nt][e];
                }
            }
            if (__any_sync(0xffffffffu, grow)) {  // the rows' maxima over all lanes, and all sums to them
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float up = top[nt][e];
                        up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 4));
                        up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 8));
                        up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 16));
                        if (limit[nt][e] == kNegInf ? up == kNegInf : up <= 0.f) continue;  // nothing seen, or no larger
                        const float f = limit[nt][e] == kNegInf ? 0.f : exp2_fast(-up);
                        base[nt][e] += up;
                        limit[nt][e] = 4.f;
                        l[nt][e] *= f;
#pragma unroll
                        for (int grp = 0; grp < GD; ++grp)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                acc[grp][k][nt][e] *= f;
                                acc[grp][k][nt][2 + e] *= f;
                            }
#pragma unroll
                        for (int mt = 0; mt < TM; ++mt) {
                            s[mt][nt][e] -= up;
                            s[mt][nt][2 + e] -= up;
                        }
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int mt = 0; mt < TM; ++mt)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            float& v = s[mt][nt][half * 2 + e];
                            v = exp2_fast(v);
                            l[nt][e] += v;
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
                                    hit |= ((which >> (mt * 16 + half * 8 + g)) & 1u) && sees(mt, half, nt, e);
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
                const float fa = factors[TOK * FP + mt * 16 + g], fb = factors[TOK * FP + mt * 16 + 8 + g];
                uint2 b[NT], b2[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float2 x = make_float2(s[mt][nt][0] * fa, s[mt][nt][1] * fa);
                    const float2 y = make_float2(s[mt][nt][2] * fb, s[mt][nt][3] * fb);
                    const uint32_t h0 = half2_bits(x.x, x.y), h1 = half2_bits(y.x, y.y);
                    b[nt] = make_uint2(transposed(h0), transposed(h1));
                    if (NP == 2) {
                        const float2 hx = half2_values(h0), hy = half2_values(h1);
                        b2[nt] = make_uint2(transposed(half2_bits(x.x - hx.x, x.y - hx.y)),
                                            transposed(half2_bits(y.x - hy.x, y.y - hy.y)));
                    }
                }
                const uint16_t* hf = reinterpret_cast<const uint16_t*>(factors + TOK * FP + TOK) + mt * 16 + 2 * t4;
                uint32_t c[4];
#pragma unroll
                for (int grp = 0; grp < GD; ++grp) {
                    uint32_t a[2][4];
                    const uint32_t from = vt + mt * 16 * PITCH + grp * (E4 ? 32 : 16);
                    if (E4) {  // a word: two values of a token, and of the next
                        load4<true>(c, from);
                        pairs_e4m3(__byte_perm(c[0], 0, 0x3120), a[0][0], a[0][1]);
                        pairs_e4m3(__byte_perm(c[1], 0, 0x3120), a[0][2], a[0][3]);
                        pairs_e4m3(__byte_perm(c[2], 0, 0x3120), a[1][0], a[1][1]);
                        pairs_e4m3(__byte_perm(c[3], 0, 0x3120), a[1][2], a[1][3]);
                    } else {   // a word: four values of a token, and of the next
                        if (grp % 2 == 0 && grp + 1 < GD) load4<true>(c, from);
                        else if (grp % 2 == 0) load2<true>(c, from);
                        const int k = grp % 2 * 2;
                        const uint32_t y0 = __byte_perm(c[k], c[k + 1], 0x5410), y1 = __byte_perm(c[k], c[k + 1], 0x7632);
                        const uint32_t even = low_nibbles(y0, y1 << 4), odd = low_nibbles(y0 >> 4, y1);
                        pairs_e2m1(even, a[0][0], a[1][0], a[0][2], a[1][2]);
                        pairs_e2m1(odd, a[0][1], a[1][1], a[0][3], a[1][3]);
                    }
                    // the group's scale beside the token's, of tokens 2 t4 and the next, and 8 on
                    const uint32_t f0 = *reinterpret_cast<const uint32_t*>(hf + grp * TOK);
                    const uint32_t f1 = *reinterpret_cast<const uint32_t*>(hf + grp * TOK + 8);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        a[k][0] = mul2(a[k][0], f0), a[k][1] = mul2(a[k][1], f0);
                        a[k][2] = mul2(a[k][2], f1), a[k][3] = mul2(a[k][3], f1);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma(acc[grp][0][nt], a[0], b[nt]);
                        mma(acc[grp][1][nt], a[1], b[nt]);
                        if (NP == 2) {
                            mma(acc[grp][0][nt], a[0], b2[nt]);
                            mma(acc[grp][1][nt], a[1], b2[nt]);
                        }
                    }
                }
            }
            __syncwarp();  // the stage and the factors are free again
            stage ^= 1;
        }

        const bool whole = !r.split || (begin <= slot_begin && before[slot + 1] <= end);
        // begun before this CTA: its part 2x; begun here and unfinished: 2x + 1
        const int part = 2 * x + (r.split && begin <= slot_begin ? 1 : 0);
        if (r.split && begin <= slot_begin && hblock == 0 && threadIdx.x == 0)
            r.entries[slot] = make_int4(whole ? -1 : x | (before[slot + 1] - 1) / share << 16, sl.row0, sl.r0, sl.rows);
        // the sums in v's own scale: times 2^(ref - 127 - LIFT - CODE), in two factors, which stay normal
        const int ex = static_cast<int>(ref) - 127 - C::LIFT - C::CODE;
        const float f1 = power(ex >> 1), f2_ = power(ex - (ex >> 1));
#pragma unroll
        for (int grp = 0; grp < GD; ++grp)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[grp][k][nt][e] = acc[grp][k][nt][e] * f1 * f2_;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
                l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
                l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
            }
        }
        // ---- a warp that has its head to itself writes from its registers: lanes of a row lie side
        // by side, four values each (two and two with 8-bit codes)
        if (r.wph == 1) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = nt * 8 + 2 * t4 + e;
                    if (row >= sl.rows) continue;
                    const float L = l[nt][e], M = limit[nt][e] == kNegInf ? kNegInf : base[nt][e];
                    if (!whole) {
                        const int64_t at_part = (static_cast<int64_t>(part) * p.heads + head) * R + row;
                        if (g == 0) r.ml[at_part] = make_float2(M, L);
                        float* to = r.o + at_part * DP + (E4 ? 2 : 4) * g;
#pragma unroll
                        for (int grp = 0; grp < GD; ++grp) {
                            const float(&a)[4] = acc[grp][0][nt], (&b)[4] = acc[grp][1][nt];
                            if (E4) {
                                *reinterpret_cast<float2*>(to + grp * 32) = make_float2(a[e], a[2 + e]);
                                *reinterpret_cast<float2*>(to + grp * 32 + 16) = make_float2(b[e], b[2 + e]);
                            } else {
                                *reinterpret_cast<float4*>(to + grp * 32) = make_float4(a[e], a[2 + e], b[e], b[2 + e]);
                            }
                        }
                        continue;
                    }
                    const int i = divide(sl.r0 + row, r.g_mul, r.g_shift), qh = head * p.G + sl.r0 + row - i * p.G;
                    const int64_t out_row = sl.row0 + i, at = out_row * p.out.st + qh * p.out.sh;
                    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
                    for (int grp = 0; grp < GD; ++grp) {
                        const float v0 = acc[grp][0][nt][e] * inv, v1 = acc[grp][0][nt][2 + e] * inv;
                        const float v2 = acc[grp][1][nt][e] * inv, v3 = acc[grp][1][nt][2 + e] * inv;
                        const int d = grp * 32 + (E4 ? 2 : 4) * g;
                        store_two<NP>(p.out.p, at, d, v0, v1, p.D, r.vec_out, p.dtype);
                        store_two<NP>(p.out.p, at, d + (E4 ? 16 : 2), v2, v3, p.D, r.vec_out, p.dtype);
                    }
                    if (p.lse && g == 0)
                        p.lse[out_row * p.heads_q + qh] = L == 0.f ? kNegInf : (M + log2f(L)) * 0.6931471805599453f;
                }
            }
            continue;
        }
        // ---- the warps of a head are joined, and the result or the part of it is written
        float* mine = reinterpret_cast<float*>(ring);  // [R][DP + 4], then maxima and sums
        float* ml = mine + R * (DP + 4);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = nt * 8 + 2 * t4 + e;
                if (g == 0) {
                    ml[row] = limit[nt][e] == kNegInf ? kNegInf : base[nt][e];
                    ml[R + row] = l[nt][e];
                }
#pragma unroll
                for (int grp = 0; grp < GD; ++grp) {
                    float* to = mine + row * (DP + 4) + grp * 32;
                    const float2 lo = make_float2(acc[grp][0][nt][e], acc[grp][0][nt][2 + e]);
                    const float2 hi = make_float2(acc[grp][1][nt][e], acc[grp][1][nt][2 + e]);
                    if (E4) {
                        *reinterpret_cast<float2*>(to + g * 2) = lo;
                        *reinterpret_cast<float2*>(to + 16 + g * 2) = hi;
                    } else {
                        *reinterpret_cast<float4*>(to + g * 4) = make_float4(lo.x, lo.y, hi.x, hi.y);
                    }
                }
            }
        }
        __syncthreads();
        // a head's warps take its rows in turn
        const float* from = reinterpret_cast<const float*>(sm + r.at_ring + head_local * r.ring);
        const int stride = r.hb * r.ring / 4;  // to the next warp of the head
        for (int row = slice; row < sl.rows; row += r.wph) {
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
            if (!whole) {
                const int64_t at_part = (static_cast<int64_t>(part) * p.heads + head) * R + row;
                if (lane == 0) r.ml[at_part] = make_float2(M, L);
#pragma unroll
                for (int c = 0; c < (DP <= 128 ? 1 : 2); ++c) {
                    const int d = lane * 4 + c * 128;
                    if (d < DP) *reinterpret_cast<float4*>(r.o + at_part * DP + d) = o[c];
                }
                continue;
            }
            const int i = divide(sl.r0 + row, r.g_mul, r.g_shift), qh = head * p.G + sl.r0 + row - i * p.G;
            const int64_t out_row = sl.row0 + i;
            const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
            for (int c = 0; c < (DP <= 128 ? 1 : 2); ++c) {
                const int d = lane * 4 + c * 128;
                const int64_t at = out_row * p.out.st + qh * p.out.sh;
                store_two<NP>(p.out.p, at, d, o[c].x * inv, o[c].y * inv, p.D, r.vec_out, p.dtype);
                store_two<NP>(p.out.p, at, d + 2, o[c].z * inv, o[c].w * inv, p.D, r.vec_out, p.dtype);
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
    r.tile_shift = C::TOK == 32 ? 5 : 4;
    while ((C::TOK * r.wph) >> (r.tile_shift + 1)) ++r.tile_shift;  // wph is a power of two
    r.smem = r.at_plan + (r.split ? (r.slots + 1 + 2 * static_cast<int>(p.sequences) + 1) * 4 : 0);
    if (r.smem + 1024 > c.dev.max_smem_optin) return cudaErrorInvalidConfiguration;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), c.dev.max_smem_optin - 1024);
    if (e != cudaSuccess) return e;
    return op_launch(c, fn, static_cast<int64_t>(r.gx) * r.head_blocks, warps * 32, r.smem, p, r);
}

template <int F, int NP, int GD>
cudaError_t pick_rows(const AttnP& p, const RowsPlan& r, const OpCfg& c) {
    if (r.nt == 1) return launch_rows<F, GD, 1, NP>(p, r, c);
    if constexpr (GD <= 3) {
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
