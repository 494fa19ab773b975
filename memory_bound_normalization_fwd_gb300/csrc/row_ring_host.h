// Host side of the row-team kernels: how many teams, stages and CTAs.
#pragma once

#include "ops.h"
#include "row_ring.cuh"

#include <atomic>

namespace rmsn {

struct RingPlan {
    RingShape shape;
    int64_t grid;  // CTAs
    int threads;
    int smem;
};

// Lays out `arrays` rows of `nvec` vectors per stage for teams of T threads in
// CTAs of up to `max_threads`, with `extra` more bytes of shared memory per
// CTA thread and about `in_flight` bytes of stages per SM. False where a row
// does not fit two stages of shared memory. cluster > 1: the CTAs of a cluster
// take a row's slices, `nvec` vectors each (one team per CTA). At most `max_teams`
// teams (clusters) in all.
bool ring_plan(const void* fn, const OpCfg& c, int64_t M, int nvec, int T, int max_threads, int arrays,
               int extra, int in_flight, int cluster, int64_t max_teams, RingPlan* out);

// Reads a status word of the current device and clears it. `launched`: whether a kernel
// that writes it ever was; a word that none did is not read (9 us each).
template <typename S>
cudaError_t symbol_read_and_clear(const S& symbol, const std::atomic<bool>& launched, unsigned int* value) {
    *value = 0;
    if (!launched.load()) return cudaSuccess;
    cudaError_t e = cudaMemcpyFromSymbol(value, symbol, sizeof(*value));
    if (e == cudaSuccess && *value != 0) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(symbol, &zero, sizeof(zero));
    }
    return e;
}

}  // namespace rmsn
