"""GB300 (sm_103a) RMSNorm forward: y = x * rsqrt(mean(x^2) + eps) * (offset + w),
with the per-row fp32 rstd kept for backward, and the operators a transformer block
runs next to it: block_fwd / block_bwd (norms around a block, gate, residual),
rope_fwd / rope_bwd (rotary positions with head norms, of one or several axes), Cache,
cache_write and cache_read (k and v in 8 or 4 bits), and what serves from that cache:
cache_attention, cache_copy_pages, cache_fork, cache_free and cache_compact.

The computation runs in hand-written CUDA kernels behind the C ABI of
``include/rmsnorm.h`` (``librmsnorm_gb300.so``); this package is the ctypes
binding (:mod:`.binding`), the in-tree build step (:mod:`.build`) and the
seeded input generator (:mod:`.workloads`).
"""
from .binding import (  # noqa: F401
    BF16, FP16, EXPORTS, VARIANTS, Cache, Options, RMSNormError, RopeAxes, block_bwd, block_fwd, bwd,
    cache_attention, cache_compact, cache_copy_pages, cache_fork, cache_free, cache_read, cache_write, fwd, lib, make_options, rope_bwd, rope_fwd, rope_steps,
    rmsnorm_bwd, rmsnorm_bwd_workspace_size,
    rmsnorm_check_device_status, rmsnorm_fwd, rmsnorm_fwd_ex, rmsnorm_fwd_strided, rmsnorm_last_error,
    rmsnorm_plan_info, rmsnorm_strerror, rmsnorm_version,
)
