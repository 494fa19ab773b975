// The row kernels of attention over a cache of 4-bit codes, 16-bit queries (attn_rows.cuh).
#include "rmsnorm.h"

#include "attn_rows.cuh"

namespace rmsn {

cudaError_t attn_rows_e2m1(const AttnP& p, const RowsPlan& r, const OpCfg& c) {
    return pick_groups<RMSNORM_CACHE_E2M1, 1>(p, r, c);
}

}  // namespace rmsn
