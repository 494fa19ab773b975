// Row teams with a ring of rows in shared memory, for the block operator's
// vector kernels.
//
// A team of T threads (whole warps) walks a contiguous range of rows. Its
// leader brings each row's arrays into the team's ring of S stages by bulk
// asynchronous copies, counted on the stage's mbarrier, S rows ahead, so the
// bytes in flight do not depend on registers. A CTA holds up to kMaxTeams
// teams; they share nothing but the SM.
//
// Waits are bounded: a thread whose stage does not land in time marks the row,
// which all threads of the team see behind the row's reduction barrier (give_up.h);
// the team then writes nothing more, waits (bounded) for its copies in flight and ends.
#pragma once

#include "async_copy.cuh"
#include "give_up.h"
#include "ops_common.cuh"

namespace rmsn {

constexpr int kMaxTeams = 8;
constexpr int kMaxRing = 8;      // stages
constexpr int kMaxTeamWarps = 16;

// How rows, teams and stages are laid out; filled by the host.
struct RingShape {
    int T;            // threads of a team, a multiple of 32
    int teams;        // of a CTA
    int stages;
    int nvec;         // 16-byte vectors of a row
    int cluster;      // CTAs of a cluster that share a row (1: none)
    int slice;        // vectors of a row in each of them but the last
    int arrays;       // rows per stage
    int rem;          // the first `rem` teams walk q + 1 rows, the others q
    int64_t q;
    int64_t slots;    // partial rows per workspace area (backward)
    int sums_at;      // byte offset behind the rings (backward)
    long long limit;  // bound of a wait in SM cycles
    long long drain;  // of the wait for copies in flight before a team that gave up ends
};

// A 16-byte vector of shared memory by its 32-bit shared address. (The address
// arithmetic of generic pointers was a third of the kernels' instructions.)
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}

struct RingShared {
    uint64_t bars[kMaxTeams][kMaxRing];
    GiveUp give_up[kMaxTeams];
};

__device__ __forceinline__ void ring_barrier(int team, int T) {
    if (T == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(T) : "memory");
}

// Sums over a team in a fixed order, one team barrier. `part` is [4][kMaxTeamWarps]
// floats of this call's parity ([1][..] for one sum), zero behind the team's warps.
// One sum: a butterfly over the warp, then over the warps' sums, which every warp
// reads with one load.
__device__ __forceinline__ float team_sum(float v, float* part, int team, int t, int T) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (T > 32 && (t & 31) == 0) part[t >> 5] = v;
    ring_barrier(team, T);
    if (T > 32) {
        v = part[t & 15];
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    }
    return v;
}

// Three sums at once: the first two steps of the butterfly also hand out which
// sum a lane goes on with (lanes 0-7 the first, 8-15 the second, 16-23 the
// third), so six shuffles do what fifteen would; the same across the warps.
__device__ __forceinline__ void team_sums3(float (&v)[3], float* part, int team, int t, int T) {
    const int lane = t & 31;
    const bool up = lane & 16, up8 = lane & 8;
    float a = up ? v[2] : v[0], b = up ? 0.f : v[1];
    a += __shfl_xor_sync(0xffffffffu, up ? v[0] : v[2], 16);
    b += __shfl_xor_sync(0xffffffffu, up ? v[1] : 0.f, 16);
    float k = up8 ? b : a;
    k += __shfl_xor_sync(0xffffffffu, up8 ? a : b, 8);
    k += __shfl_xor_sync(0xffffffffu, k, 4);
    k += __shfl_xor_sync(0xffffffffu, k, 2);
    k += __shfl_xor_sync(0xffffffffu, k, 1);
    if (T > 32 && (lane & 7) == 0) part[(lane >> 3) * kMaxTeamWarps + (t >> 5)] = k;
    ring_barrier(team, T);
    if (T > 32) {
        const float* q = part + (lane >> 3) * kMaxTeamWarps + (lane & 7);
        k = q[0] + q[8];
        k += __shfl_xor_sync(0xffffffffu, k, 4);
        k += __shfl_xor_sync(0xffffffffu, k, 2);
        k += __shfl_xor_sync(0xffffffffu, k, 1);
    }
    v[0] = __shfl_sync(0xffffffffu, k, 0);
    v[1] = __shfl_sync(0xffffffffu, k, 8);
    v[2] = __shfl_sync(0xffffffffu, k, 16);
}

// A team's ring: the leader's issue side and the place of each stage.
struct Ring {
    uint32_t bars;       // shared address of the team's barriers
    uint32_t base;       // shared address of the team's stages
    uint32_t row_bytes;  // of one array
    uint32_t stage_bytes;

    __device__ __forceinline__ uint32_t stage(int st) const { return base + st * stage_bytes; }
    __device__ __forceinline__ uint32_t bar(int st) const { return bars + 8 * st; }
    __device__ __forceinline__ void expect(int st) const { mbar_arrive_expect_tx(bar(st), stage_bytes); }
    __device__ __forceinline__ void copy(int st, int array, const void* src) const {
        bulk_g2s(stage(st) + array * row_bytes, src, row_bytes, bar(st));
    }
};

}  // namespace rmsn
