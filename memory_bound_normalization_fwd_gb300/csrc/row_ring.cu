// Layout of the row-team kernels' launches.
#include "row_ring_host.h"

#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>
#include <utility>

namespace rmsn {
namespace {

// What a kernel needs of the device, looked up once per device: its static
// shared memory and the CTAs of `threads` threads that registers allow per SM.
struct Facts {
    int static_smem = 0;
    int by_registers = 0;
};

Facts facts(const void* fn, int threads, int max_optin) {
    static std::mutex mu;
    static std::map<std::pair<int, std::pair<const void*, int>>, Facts> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return {};
    std::lock_guard<std::mutex> guard(mu);
    const auto key = std::make_pair(dev, std::make_pair(fn, threads));
    auto it = cache.find(key);
    if (it != cache.end()) return it->second;
    Facts f;
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, fn) == cudaSuccess &&
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             max_optin - static_cast<int>(attr.sharedSizeBytes)) == cudaSuccess &&
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&f.by_registers, fn, threads, 0) == cudaSuccess)
        f.static_smem = static_cast<int>(attr.sharedSizeBytes);
    else
        f.by_registers = 0;
    return cache[key] = f;
}

// Clusters of CTAs that the device holds at once, looked up once.
int max_clusters(const void* fn, int cluster, int threads, int smem) {
    static std::mutex mu;
    static std::map<std::tuple<int, const void*, int, int, int>, int> cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::lock_guard<std::mutex> guard(mu);
    const auto key = std::make_tuple(dev, fn, cluster, threads, smem);
    auto it = cache.find(key);
    if (it != cache.end()) return it->second;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(cluster);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) n = 0;
    return cache[key] = n;
}

}  // namespace

bool ring_plan(const void* fn, const OpCfg& c, int64_t M, int nvec, int T, int max_threads, int arrays,
               int extra, int in_flight, int cluster, int64_t max_teams, RingPlan* out) {
    if (T > max_threads) return false;
    int teams = cluster > 1 ? 1 : std::min(max_threads / T, kMaxTeams);
    // Few rows: one team per CTA spreads them over more SMs.
    while (teams > 1 && static_cast<int64_t>(teams) * c.dev.sm_count > M) --teams;
    const Facts f = facts(fn, teams * T, c.dev.max_smem_optin);
    if (f.by_registers < 1) return false;
    const int64_t stage = static_cast<int64_t>(nvec) * 16 * arrays * teams;
    // Shared memory of an SM is 1 KB per CTA more than a CTA may ask for.
    const int64_t per_sm = c.dev.max_smem_optin + 1024;
    int ctas = f.by_registers, stages = 0;
    for (; ctas >= 1; --ctas) {
        const int64_t room = per_sm / ctas - 1024 - f.static_smem - static_cast<int64_t>(extra) * teams * T;
        stages = static_cast<int>(std::min<int64_t>(room / stage, kMaxRing));
        if (stages >= 2) break;
    }
    if (ctas < 1) return false;
    // More stages than carry the bandwidth cost it (see the callers' figures).
    const int64_t enough = (in_flight + ctas * stage / 2) / (ctas * stage);
    stages = static_cast<int>(std::max<int64_t>(2, std::min<int64_t>(stages, enough)));
    const int64_t want = (M + teams - 1) / teams;
    int64_t cap = static_cast<int64_t>(c.dev.sm_count) * ctas;
    if (cluster > 1)
        cap = max_clusters(fn, cluster, teams * T,
                           static_cast<int>(stage * stages + static_cast<int64_t>(extra) * teams * T));
    if (c.max_ctas > 0) cap = std::min<int64_t>(cap, std::max(1, c.max_ctas / cluster));
    cap = std::min(cap, max_teams / teams);
    int64_t groups = std::min(want, cap);  // CTAs, or clusters
    // Every team walks at least one row.
    while (groups * teams > M) --groups;
    if (groups < 1) return false;
    const int64_t n = groups * teams;
    out->grid = groups * cluster;
    RingShape& s = out->shape;
    s.cluster = cluster;
    s.slice = nvec;
    s.T = T;
    s.teams = teams;
    s.q = M / n;
    s.rem = static_cast<int>(M % n);
    s.stages = static_cast<int>(std::min<int64_t>(stages, s.q + (s.rem ? 1 : 0)));
    s.nvec = nvec;
    s.arrays = arrays;
    s.slots = 0;
    s.sums_at = 0;
    s.drain = 2100000000LL;  // one second at the top SM clock
    s.limit = c.wait_limit_ns > 0 ? std::max<long long>(1, c.wait_limit_ns * 21 / 10) : s.drain;
    out->threads = teams * T;
    out->smem = static_cast<int>(stage * s.stages + static_cast<int64_t>(extra) * teams * T);
    return s.q < (int64_t(1) << 31);
}

}  // namespace rmsn
