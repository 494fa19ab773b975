// Attention over the quantised cache for prompts, on the tensor cores (tcgen05): blocks of 256
// rows of a key head against tiles of 128 tokens.
//
// The mathematics. Each tile's codes become fp16 in shared memory, c * 2^(a - A + C): a the scale
// byte of a token's group, A the tile's largest, C such that the largest code comes near 2^15 (6 for
// 8-bit codes, 12 for 4-bit ones). That is exact while the codes' last bit (2^-9; 2^-1) stays at
// 2^-24 or above: for groups within 2^21 (2^35) of the tile's largest. Below, values are off by less
// than 2^-22 (2^-34) of 2^(A - 127), and groups beyond 2^30 (2^36) are left out. A goes into the
// scores' factor, a number for the tile. q is brought near 2^15 by a power of two per row, as
// in attn_rows.cuh. So S = Q K^T has exact products and fp32 sums; o += P V has P in fp16 (11
// bits) and V in the same form as K, with the tile's B relative to a reference R that moves only where
// B exceeds it by more than 2^1: p * 2^(B - R + 8), which keeps p to 2^-33 of R. Softmax with a running
// maximum that moves by more than 2^6 at a time, so that the sums in tensor memory are rarely read
// and scaled.
//
// Who does what, in a CTA of 16 warps: two warpgroups of softmax (a thread a row, each with 128
// rows of its own), one warpgroup that looks up, loads and converts the tiles (into two stages of
// K and of V), and two warps that issue the matrix instructions, one for either half (one for both
// took longer over them than they run: prompts' chunks 361 us). The softmax takes a tile in two
// steps of 64 tokens. S takes 128 columns of tensor memory for either half, and P goes over it as the
// second product's first operand; o takes head_dim columns. While one half is in its softmax the
// other half's products run.
// Bound (GB300): the chain of softmax and products within a half. Three chunks of 2048 queries of 32
// heads of 128 values behind up to 8192 tokens of 8 heads in 4 bits, bf16, 351 us, 46% of the rate of
// a large product: matrix units active 39%, issue slots 45%, exponentials 20%; a half waits for S about as
// long as its softmax takes, as both halves' products go through the same matrix unit, which reads
// their operands at the rate of shared memory. (S in steps of 64 tokens, so that softmax starts
// earlier: 346 to 354 us, the same.)
//
// Every wait is bounded; a role whose wait ran out leaves its loop, which makes the others' run out too, and the
// tensor memory is freed when the matrix instructions are done.
#include "rmsnorm.h"

#include "async_copy.cuh"
#include "attn_rows.cuh"
#include "give_up.h"
#include "tensor_core.cuh"

namespace rmsn {
namespace {

constexpr int kTile = 128;      // tokens of a tile
constexpr int kHalf = 128;      // rows of a half
constexpr int kThreads = 512;
constexpr int kStep = 64;       // tokens of a step
constexpr int kInfos = 4;       // tiles whose facts are kept
// P = p * 2^(B - R + kLift) in fp16: below 2^-14 of it rounding is no longer relative, so that p * 2^(B - R)
// is kept to 2^-33. The maximum may lag by 2^kGrow, R by 2^kFar: together at most 2^15. (GB300, prompts' chunks
// as above, us, grow / far: 4 / 3 372, 5 / 2 358, 6 / 1 351, 7 / 0 352; without the lift, 8 / 6, 355.)
constexpr int kLift = 8, kGrow = 6, kFar = 1;

// What the softmax needs to know of a tile.
struct TileInfo {
    float k;                   // 2^(a - 127 - C), a k's largest scale byte
    int b;                     // v's largest scale byte
    uint32_t there[4];         // tokens whose page is there and that a row sees
    uint32_t bad;              // some group of v is not a number
    uint32_t pad;
};

template <int GD>
struct Tiles {
    static constexpr int D = GD * 32, BLOCKS = (GD + 1) / 2;  // 64 values (128 bytes) of a row
    static constexpr int MATRIX = BLOCKS * 128 * 128;         // 128 rows
    static constexpr int Q = 0, K = 2 * MATRIX, V = K + 2 * MATRIX, END = V + 2 * MATRIX;
    static constexpr int SMEM = END + 1024;  // to a boundary of 1024 bytes
};

// Byte of piece `c` (16 bytes) of a row in a matrix of 128 rows.
__device__ __forceinline__ uint32_t piece_at(int row, int c) {
    return (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}
__device__ __forceinline__ void store_piece(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// 2^e as a pair of fp16, 0 below 2^-24 (e <= 15).
__device__ __forceinline__ uint32_t power_half2(int e) {
    const uint32_t h = e >= -14 ? static_cast<uint32_t>(e + 15) << 10 : e >= -24 ? 1u << (e + 24) : 0u;
    return h | h << 16;
}
// 2^e as fp32, also below 2^-126 (-149 <= e <= 127).
__device__ __forceinline__ float tiny_power(int e) {
    return __uint_as_float(e < -126 ? 1u << (e + 149) : static_cast<uint32_t>(e + 127) << 23);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// The lowest n bits (n below 0: none, above 32: all).
__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }
// True for one lane of the warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(yes));
    return yes != 0;
}
// The loading warpgroup's own barrier.
__device__ __forceinline__ void loaders_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

struct TilesP {
    int slots;
    int window, most_tokens;
    uint32_t g_mul, page_mul, pages;
    int g_shift, page_shift;
    long long limit;  // of a wait, in cycles
};

template <int F, int GD>
__global__ void __launch_bounds__(kThreads, 1) attn_tiles_kernel(const AttnP p, const TilesP tp) {
    using C = Tiles<GD>;
    constexpr bool E4 = F == RMSNORM_CACHE_E4M3;
    constexpr int CODE = E4 ? 6 : 12;               // C above
    constexpr int CH = E4 ? 2 * GD : GD;            // 16 code bytes: pieces of a token, and of a thread in a tile
    constexpr uint32_t kNone = 0xffffffffu;
    extern __shared__ unsigned char raw[];
    __shared__ __align__(8) uint64_t bars[19];
    __shared__ TileInfo infos[kInfos];
    __shared__ uint32_t bads[kInfos][kTile];        // groups of a token's v that are not numbers
    __shared__ uint32_t tokens[2][kTile];           // where the tile's tokens lie
    __shared__ int tops[2][2][4];
    __shared__ uint32_t tmem_at;
    __shared__ GiveUp late;
    const uint32_t smem = (smem_u32(raw) + 1023u) & ~1023u;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int head = static_cast<int>(blockIdx.x) % p.heads;
    const int slot = tp.slots - 1 - static_cast<int>(blockIdx.x) / p.heads;  // the longest first
    // barriers: K and V ready (loaders), K and V read (products), S ready, P ready, o summed, all done
    auto bar = [&](int i) { return smem_u32(bars + i); };
    constexpr int kKFull = 0, kVFull = 2, kKFree = 4, kVFree = 6, kSFull = 8, kPFull = 12, kOFree = 16, kDone = 18;
    if (w == 0) tmem_alloc(smem_u32(&tmem_at));
    pdl_wait();
    pdl_launch_dependents();

    RowsPlan plan;  // what the slots' arithmetic takes of it
    plan.window = tp.window;
    plan.g_mul = tp.g_mul;
    plan.g_shift = tp.g_shift;
    plan.tile_shift = 7;
    plan.most_tokens = tp.most_tokens;
    const Slot sl = slot_of<2 * kHalf>(p, plan, Sequences{nullptr, nullptr}, slot);
    const int halves = sl.rows > kHalf ? 2 : 1, tiles = sl.tiles;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(kKFull + i), 128);
            mbar_init(bar(kVFull + i), 128);
            mbar_init(bar(kKFree + i), halves);
            mbar_init(bar(kVFree + i), halves);
            mbar_init(bar(kOFree + i), 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(bar(kSFull + i), 1);
        for (int i = 0; i < 4; ++i) mbar_init(bar(kPFull + i), 128);  // half * 2 + step
        mbar_init(bar(kDone), halves);
        late.clear();
        fence_mbar_init();
    }

    if (sl.rows && sl.len > sl.held && threadIdx.x == 0) atomicOr(p.status, 1u);  // tokens past the table's row

    // ---- q, by the softmax threads: a row each
    float row_scale = 0.f;
    int lim = 0, low = 0;  // tokens that the row sees
    const int half = w >> 2, rr = threadIdx.x;
    const bool live = w < 8 && rr < sl.rows;
    int64_t out_row = 0;
    int qh = 0;
    if (w < 8 && half < halves) {
        uint32_t v[C::D / 2];
        float top = 0.f;
        if (live) {
            const int i = divide(sl.r0 + rr, tp.g_mul, tp.g_shift);
            out_row = sl.row0 + i;
            qh = head * p.G + sl.r0 + rr - i * p.G;
            int to;
            seen32(p, plan, sl.n, sl.len, i, low, to);
            lim = min(to, sl.held);
            const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q.p) + out_row * p.q.st + qh * p.q.sh);
#pragma unroll
            for (int k = 0; k < C::D / 8; ++k) {
                const uint4 u = __ldg(q + k);
                v[4 * k] = u.x, v[4 * k + 1] = u.y, v[4 * k + 2] = u.z, v[4 * k + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < C::D / 2; ++k) v[k] = 0;
        }
#pragma unroll
        for (int k = 0; k < C::D / 2; ++k) {
            const float2 f = unpack16(v[k], p.dtype == kBF16);
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        int ex = static_cast<int>(__float_as_uint(top) >> 23);
        ex = top == 0.f ? 141 : ex < 15 ? 15 : ex;  // both powers stay normal
        const float up = __uint_as_float(static_cast<uint32_t>(268 - ex) << 23);
        row_scale = __uint_as_float(static_cast<uint32_t>(ex - 14) << 23) * (p.scale * 1.4426950408889634f);
        const uint32_t to = smem + C::Q + half * C::MATRIX;
#pragma unroll
        for (int k = 0; k < C::D / 8; ++k) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = unpack16(v[4 * k + e], p.dtype == kBF16);
                h[e] = half2_bits(f.x * up, f.y * up);
            }
            store_piece(to + piece_at(rr & 127, k), h[0], h[1], h[2], h[3]);
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_at;

    // Registers go from the others to the softmax: 2 * 168 + 120 + 56 = 4 * 128 of each warpgroup.
    if (w < 8) {
        // ---- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        if (sl.rows && half < halves) {
            const uint32_t lanes = tmem + (static_cast<uint32_t>((w & 3) * 32) << 16);
            const uint32_t o_at = lanes + 256 + half * 128;
            float m = 0.f, l = 0.f;
            bool started = false;
            int ref = 0;
            uint32_t nan_groups = 0;
            bool ok = true;
            for (int u = 0; u < 2 * tiles; ++u) {
                const int t = u >> 1, step = u & 1;
                if (step == 0) {
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kSFull + half), t & 1, tp.limit));
                    if (!ok) break;
                }
                tc_fence_after();
                const uint32_t s_at = lanes + half * 128 + step * 64;
                uint32_t v[64];
                tmem_load_async(v, s_at);
                tmem_load_async(v + 32, s_at + 32);
                const TileInfo& info = infos[t % kInfos];
                const int b = info.b, t0 = (sl.tile0 + t) * kTile + step * kStep;
                const uint32_t there0 = info.there[2 * step], there1 = info.there[2 * step + 1];
                const float factor = row_scale * info.k;
                // Sums of the tiles before, scaled by f (all lanes of the warp).
                auto scale_sums = [&](float f) {
#pragma unroll 1
                    for (int c = 0; c < GD * 32; c += 16) {
                        uint32_t o[16];
                        tmem_load16(o, o_at + c);
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_store16(o_at + c, o);
                    }
                    tmem_stored();
                };
                if (u == 0) ref = b;
                // The same for all threads. Where v lies far below the reference (a tile of zeros: byte 0),
                // no lower than -40: P is at most 2^(14 - 40) there, nothing in fp16, and l, which is
                // summed from the shifted values, keeps the tile's weight.
                const int far = max(b - ref, -40), moved = far > kFar ? kLift : far + kLift;
                const float shift = static_cast<float>(moved);
                const bool masked = __any_sync(0xffffffffu, (there0 & there1) != 0xffffffffu || t0 + kStep > lim || t0 < low);
                if (info.bad) {  // rare: which groups of v are not numbers for this row
                    for (int k = 0; k < kStep; ++k)
                        if (t0 + k < lim && t0 + k >= low) nan_groups |= bads[t % kInfos][step * kStep + k];
                }
                // in powers of two, above the row's maximum so far; -infinity where the row does
                // not see the token
                const float less = shift - m;
                float most = -INFINITY;
                tmem_loaded(v);
                const f2 factor2 = f2_dup(factor), less2 = f2_dup(less);
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    const float2 x = f2_get(f2_fma(f2_make(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), factor2, less2));
                    v[e] = __float_as_uint(x.x);
                    v[e + 1] = __float_as_uint(x.y);
                }
                if (masked) {
                    const uint32_t s0 = there0 & bits_below(lim - t0) & ~bits_below(low - t0);
                    const uint32_t s1 = there1 & bits_below(lim - t0 - 32) & ~bits_below(low - t0 - 32);
#pragma unroll
                    for (int e = 0; e < 64; ++e)
                        if (!(((e < 32 ? s0 : s1) >> (e & 31)) & 1u)) v[e] = 0xff800000u;
                }
                float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                for (int e = 0; e < 64; e += 4) {
                    m0 = max3(m0, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                    m1 = max3(m1, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
                }
                most = fmaxf(m0, m1);
                const float above = most - shift;
                const bool grow = started ? above > static_cast<float>(kGrow) : most > -INFINITY;
                if (__any_sync(0xffffffffu, grow || far > kFar)) {
                    // the sums so far are complete: the products that this S waited behind
                    float f = far > kFar ? power(-far) : 1.f;
                    if (far > kFar) ref = b;
                    if (grow) {
                        const float g = started ? exp2_fast(-above) : 0.f;
                        m += above;
                        started = true;
                        l *= g;
                        f *= g;
#pragma unroll
                        for (int e = 0; e < 64; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) - above);
                    }
                    if (u > 0) {
                        // (S came behind the last tile's products; step 0's may be on its way)
                        ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(kOFree + half), (u - 1) & 1, tp.limit));
                        if (!ok) break;
                        tc_fence_after();
                        scale_sums(f);
                    }
                }
                f2 s0 = 0, s1 = 0;
#pragma unroll
                for (int e = 0; e < 64; e += 2) {
                    const float px = exp2_fast(__uint_as_float(v[e])), py = exp2_fast(__uint_as_float(v[e + 1]));
                    if (e & 2) s1 = f2_add(s1, f2_make(px, py));
                    else s0 = f2_add(s0, f2_make(px, py));
                    v[e / 2] = half2_bits(px, py);
                }
                tmem_store32(s_at, v);
                l = fmaf(f2_sum(f2_add(s0, s1)), power(-moved), l);
                tmem_stored();
                tc_fence_before();
                mbar_arrive(bar(kPFull + half * 2 + step));
            }
            ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar(kDone), 0, tp.limit));
            if (!ok) {
                if (lane == 0) atomicOr(p.late, 1u);
            } else {
                tc_fence_after();
                const float inv = l == 0.f ? 0.f : 1.f / l;
                // 2^(ref - 127 - CODE - kLift) in two factors, which stay normal
                const int e = ref - 127 - CODE - kLift;
                const float f1 = power(e / 2) * inv, f2_ = power(e - e / 2);
                uint16_t* out = static_cast<uint16_t*>(p.out.p) + out_row * p.out.st + qh * p.out.sh;
                const bool vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
#pragma unroll
                for (int c = 0; c < GD; ++c) {
                    uint32_t v[32], h[16];
                    tmem_load_async(v, o_at + c * 32);
                    tmem_loaded(v);
                    const bool nan = (nan_groups >> c) & 1u;
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float x = __uint_as_float(v[2 * k]) * f1 * f2_, y = __uint_as_float(v[2 * k + 1]) * f1 * f2_;
                        if (l == 0.f) x = y = 0.f;
                        if (nan) x = y = __uint_as_float(0x7fc00000u);
                        h[k] = p.dtype == kBF16 ? Codec<kBF16>::pack2(x, y) : Codec<kFP16>::pack2(x, y);
                    }
                    if (!live) continue;
                    if (vec) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *reinterpret_cast<uint4*>(out + c * 32 + k * 8) = make_uint4(h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            out[c * 32 + 2 * k] = static_cast<uint16_t>(h[k]);
                            out[c * 32 + 2 * k + 1] = static_cast<uint16_t>(h[k] >> 16);
                        }
                    }
                }
                if (p.lse && live)
                    p.lse[out_row * p.heads_q + qh] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            }
        }
    } else if (w < 12) {
        // ---- tiles: thread i looks up token i; pieces of 16 code bytes go round the threads
        asm volatile("setmaxnreg.dec.sync.aligned.u32 120;");
        if (sl.rows) {
            const int tid = threadIdx.x - 256, lw = w - 8;
            const int32_t* table = p.table + static_cast<int64_t>(sl.b) * p.width;
            const uint32_t head_off = static_cast<uint32_t>(head * head_step(p));
            // (in two steps, a tile apart: the page's number is on its way in between)
            auto page_of = [&](int t) -> uint32_t {
                const int tok = (sl.tile0 + t) * kTile + tid;
                if (t >= tiles || tok < sl.low || tok >= sl.high) return kNone;
                return static_cast<uint32_t>(__ldg(table + divide(tok, tp.page_mul, tp.page_shift)));
            };
            auto lookup = [&](int t, uint32_t page) {
                const int tok = (sl.tile0 + t) * kTile + tid;
                uint32_t at = kNone;
                if (t < tiles && tok >= sl.low && tok < sl.high) {
                    const uint32_t off = tok - divide(tok, tp.page_mul, tp.page_shift) * p.page_size;
                    if (page < tp.pages)
                        at = (p.heads_first ? page * p.heads * p.page_size + off : (page * p.page_size + off) * p.heads) + head_off;
                    else
                        atomicOr(p.status, 1u);
                }
                tokens[t & 1][tid] = at;
                bads[t % kInfos][tid] = 0;
                const uint32_t some = __ballot_sync(0xffffffffu, at != kNone);
                if (lane == 0) infos[t % kInfos].there[lw] = some;
                if (tid == 0) infos[t % kInfos].bad = 0;
            };
            uint4 kc[CH], vc[CH];
            uint32_t ks[CH], vs[CH];
            auto load_codes = [&](int t, int which, uint4 (&c)[CH]) {
#pragma unroll
                for (int k = 0; k < CH; ++k) {
                    const int i = tid + 128 * k, tok = i / CH, part = i - tok * CH;
                    const uint32_t at = tokens[t & 1][tok];
                    c[k] = at == kNone ? make_uint4(0u, 0u, 0u, 0u)
                                       : __ldg(reinterpret_cast<const uint4*>(plus(p.codes[which] + part * 16, at, CH * 16)));
                }
            };
            auto load_scales = [&](int t, int which, uint32_t (&s)[CH]) {
#pragma unroll
                for (int k = 0; k < CH; ++k) {
                    const int i = tid + 128 * k, tok = i / CH, part = i - tok * CH;
                    const uint32_t at = tokens[t & 1][tok];
                    s[k] = at == kNone ? 0u : __ldg(plus(p.scales[which] + (E4 ? part >> 1 : part), at, GD));
                }
            };
            // A piece of codes as fp16 into the matrix at `to`.
            auto convert = [&](uint32_t to, int k, const uint4& c, uint32_t f) {
                const int i = tid + 128 * k, tok = i / CH, part = i - tok * CH;
                // Lanes of the upper half of a row's pieces write theirs in another order: eight lanes
                // write to eight different columns of 16 bytes.
                const bool upper = part >= CH / 2 && C::BLOCKS == 2 && GD == 4;
                const uint32_t word[4] = {upper ? c.z : c.x, upper ? c.w : c.y, upper ? c.x : c.z, upper ? c.y : c.w};
                if (E4) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        uint32_t h[4];
                        pairs_e4m3(word[2 * j], h[0], h[1]);
                        pairs_e4m3(word[2 * j + 1], h[2], h[3]);
                        store_piece(to + piece_at(tok, part * 2 + (j ^ (upper ? 1 : 0))), mul2(h[0], f), mul2(h[1], f), mul2(h[2], f), mul2(h[3], f));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t h[4];
                        pairs_e2m1(word[j], h[0], h[1], h[2], h[3]);
                        store_piece(to + piece_at(tok, part * 4 + (j ^ (upper ? 2 : 0))), mul2(h[0], f), mul2(h[1], f), mul2(h[2], f), mul2(h[3], f));
                    }
                }
            };
            lookup(0, page_of(0));
            uint32_t page = page_of(1);
            loaders_sync();
            load_codes(0, 0, kc);
            load_scales(0, 0, ks);
            load_scales(0, 1, vs);
            for (int t = 0; t < tiles; ++t) {
                const int stage = t & 1;
                load_codes(t, 1, vc);
                // the largest scale bytes that are numbers
                int a = 0, b = 0;
#pragma unroll
                for (int k = 0; k < CH; ++k) {
                    a = max(a, static_cast<int>(ks[k] == 255u ? 0u : ks[k]));
                    b = max(b, static_cast<int>(vs[k] == 255u ? 0u : vs[k]));
                }
                a = __reduce_max_sync(0xffffffffu, a);
                b = __reduce_max_sync(0xffffffffu, b);
                if (lane == 0) tops[stage][0][lw] = a, tops[stage][1][lw] = b;
                if (t >= 2 && !mbar_wait_bounded(bar(kKFree + stage), ((t >> 1) + 1) & 1, tp.limit)) late.mark(2 * t);
                loaders_sync();
                if (late.at(2 * t)) break;
#pragma unroll
                for (int k = 0; k < 4; ++k) a = max(a, tops[stage][0][k]), b = max(b, tops[stage][1][k]);
                if (tid == 0) infos[t % kInfos].k = tiny_power(a - 127 - CODE), infos[t % kInfos].b = b;
#pragma unroll
                for (int k = 0; k < CH; ++k) {
                    if (vs[k] == 255u) {
                        const int i = tid + 128 * k, tok = i / CH, part = i - tok * CH;
                        atomicOr(&bads[t % kInfos][tok], 1u << (E4 ? part >> 1 : part));
                        infos[t % kInfos].bad = 1;
                    }
                    const uint32_t f = ks[k] == 255u ? 0x7e007e00u : power_half2(static_cast<int>(ks[k]) - a + CODE);
                    convert(smem + C::K + stage * C::MATRIX, k, kc[k], f);
                }
                fence_proxy_async_smem();
                mbar_arrive(bar(kKFull + stage));
                lookup(t + 1, page);
                page = page_of(t + 2);
                uint32_t vf[CH];
#pragma unroll
                for (int k = 0; k < CH; ++k) vf[k] = vs[k] == 255u ? 0u : power_half2(static_cast<int>(vs[k]) - b + CODE);
                if (t >= 2 && !mbar_wait_bounded(bar(kVFree + stage), ((t >> 1) + 1) & 1, tp.limit)) late.mark(2 * t + 1);
                loaders_sync();
                if (late.at(2 * t + 1)) break;
                if (t + 1 < tiles) {
                    load_codes(t + 1, 0, kc);
                    load_scales(t + 1, 0, ks);
                    load_scales(t + 1, 1, vs);
                }
#pragma unroll
                for (int k = 0; k < CH; ++k) convert(smem + C::V + stage * C::MATRIX, k, vc[k], vf[k]);
                fence_proxy_async_smem();
                mbar_arrive(bar(kVFull + stage));
            }
        }
    } else {
        // ---- matrix instructions
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        const int q = w - 12;  // the half
        if (q < halves && sl.rows) {  // all lanes go through it together, one issues
        constexpr uint32_t s_shape = mma_shape(128, kTile, false), o_shape = mma_shape(128, C::D, true);
        const bool leader = elect_one();
        bool ok = true;
        // Matrices by their first piece; others are a number of 16 bytes on.
        const uint64_t q_at = smem_matrix(smem + C::Q, 16, 1024), k_at = smem_matrix(smem + C::K, 16, 1024);
        const uint64_t v_at = smem_matrix(smem + C::V, 16384, 1024);
        auto commit = [&](int i) {
            if (leader) tc_commit(bar(i));
        };
        auto wait = [&](int i, int parity) { return __all_sync(0xffffffffu, mbar_wait_bounded(bar(i), parity, tp.limit)); };
        auto scores = [&](int stage) {
            const uint64_t a = q_at + q * (C::MATRIX / 16), b = k_at + stage * (C::MATRIX / 16);
            if (leader) {
#pragma unroll
                for (int k = 0; k < C::D / 16; ++k) {
                    const uint32_t off = (k >> 2) * 1024 + (k & 3) * 2;
                    tc_mma(tmem + q * 128, a + off, b + off, s_shape, k > 0);
                }
                tc_commit(bar(kSFull + q));
                tc_commit(bar(kKFree + stage));
            }
        };
        ok = wait(kKFull, 0);
        if (ok) {
            tc_fence_after();
            scores(0);
        }
        for (int u = 0; ok && u < 2 * tiles; ++u) {
            const int t = u >> 1, step = u & 1, stage = t & 1;
            if (step == 0) ok = wait(kVFull + stage, (t >> 1) & 1);
            ok = ok && wait(kPFull + q * 2 + step, t & 1);
            if (!ok) break;
            tc_fence_after();
            // V: 64 values of head_dim a row of 128 bytes; 16 tokens are 2048 bytes on
            const uint64_t v = v_at + stage * (C::MATRIX / 16) + step * (kStep * 128 / 16);
            const uint32_t from = tmem + q * 128 + step * 64, d = tmem + 256 + q * 128;
            if (leader) {
#pragma unroll
                for (int k = 0; k < kStep / 16; ++k) tc_mma_tmem(d, from + k * 8, v + k * 128, o_shape, u > 0 || k > 0);
                tc_commit(bar(kOFree + q));
            }
            if (step == 1) commit(kVFree + stage);
            if (step == 1 && t + 1 < tiles) {
                ok = wait(kKFull + (stage ^ 1), ((t + 1) >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                scores(stage ^ 1);
            }
        }
        if (!ok && leader) atomicOr(p.late, 1u);
        commit(kDone);
        // nothing of it is on its way when the memory is freed (two seconds, whatever the call's limit)
        mbar_wait_bounded(bar(kDone), 0, 4000000000LL);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (w == 0) {
        tc_fence_after();
        tmem_free(tmem);
    }
}

template <int F, int GD>
cudaError_t launch_tiles(const AttnP& p, const TilesP& tp, const OpCfg& c) {
    auto fn = attn_tiles_kernel<F, GD>;
    const int smem = Tiles<GD>::SMEM;
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn), smem);
    if (e != cudaSuccess) return e;
    return op_launch(c, fn, static_cast<int64_t>(tp.slots) * p.heads, kThreads, smem, p, tp);
}

template <int F>
cudaError_t pick_tiles(const AttnP& p, const TilesP& tp, const OpCfg& c) {
    switch (p.groups) {
        case 2: return launch_tiles<F, 2>(p, tp, c);
        case 3: return launch_tiles<F, 3>(p, tp, c);
        default: return launch_tiles<F, 4>(p, tp, c);
    }
}

}  // namespace

cudaError_t attn_tiles(const AttnP& p, const RowsPlan& r, const OpCfg& c) {
    TilesP tp;
    tp.slots = static_cast<int>(p.rows * p.G / (2 * kHalf) + p.sequences);
    tp.window = r.window;
    tp.most_tokens = r.most_tokens;
    tp.g_mul = r.g_mul;
    tp.g_shift = r.g_shift;
    tp.page_mul = r.page_mul;
    tp.page_shift = r.page_shift;
    tp.pages = r.pages;
    // SM cycles, at about two a nanosecond
    tp.limit = 2 * (c.wait_limit_ns > 0 ? c.wait_limit_ns : 1000000000LL);
    return p.format == RMSNORM_CACHE_E4M3 ? pick_tiles<RMSNORM_CACHE_E4M3>(p, tp, c) : pick_tiles<RMSNORM_CACHE_E2M1>(p, tp, c);
}

}  // namespace rmsn
