// The row kernels of attention over a cache of 8-bit codes, fp32 queries (attn_rows.cuh).
#include "rmsnorm.h"

#include "attn_rows.cuh"

namespace rmsn {

cudaError_t attn_rows_e4m3_fp32(const AttnP& p, const RowsPlan& r, const OpCfg& c) {
    return pick_groups<RMSNORM_CACHE_E4M3, 2>(p, r, c);
}

}  // namespace rmsn
