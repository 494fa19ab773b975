/*
 * rmsnorm.h — C ABI of the GB300 (sm_103a) RMSNorm forward library
 * (librmsnorm_gb300.so).
 *
 * The operation. For a row-major activation x[M, N] and a weight w[N]:
 *
 *   rstd[i] = 1 / sqrt( (1/N) * sum_{j<N} x[i,j]^2 + eps )          (fp32)
 *   y[i,j]  = dtype( (x[i,j] * rstd[i]) * (offset + w[j]) )
 *
 * with offset 0 for Llama-style weights and 1 for Gemma-style weights.
 * Defined by the kernel listing of "Why cutile's rmsnorm required full
 * register" (TileGym issue #169): x is widened to fp32 before squaring, the
 * row sum of squares is divided by the true N, eps is added inside the rsqrt,
 * the fp32 rstd is stored "for backward", the normalised row is scaled by
 * (offset + w) in fp32 and cast once to x's dtype (the listing's cast to the
 * dtype of X, whatever that dtype is: bf16, fp16 or fp32). The same formula, with
 * offset 0, is the Overview and Verification formula of "RMSNorm Kernel
 * Optimization" (skillmd): out = x / sqrt(mean(x^2) + eps) * weight.
 * Arithmetic is fp32 throughout (sum of squares, mean, rsqrt, products); y is
 * rounded to nearest-even once (for fp32 y, the products are fp32 products).
 * Results are deterministic: the same inputs and
 * launch shape always give the same bits.
 *
 * Memory. Every pointer is a DEVICE pointer on the calling thread's current
 * CUDA device (cudaSetDevice), allocated by the caller, except the host
 * buffers of rmsnorm_fwd_host(). The library never allocates or frees caller
 * memory, copies it only in rmsnorm_fwd_host(), and never synchronises except
 * in rmsnorm_check_device_status().
 *   x     [M, N] bf16, fp16 or fp32, contiguous row-major (row i at x + i*N)
 *   w     [N]    same dtype as x
 *   y     [M, N] same dtype as x; may equal x exactly (in place), must not
 *                otherwise overlap x, w or rstd
 *   rstd  [M]    fp32; must not overlap x, w or y; may be NULL (inference:
 *                rstd is then not stored)
 * rmsnorm_fwd_strided() takes row strides instead (row i of x at x + i*ldx,
 * of y at y + i*ldy, in elements, each >= N), for rows that are slices of
 * wider tensors; the overlap rules then apply to the spans from the first to
 * the last element of each array.
 * x, w, y need only their element alignment (2 bytes; 4 for fp32) and rstd
 * 4 bytes. 16-byte-aligned x, w, y whose rows are whole 16-byte vectors (N a
 * multiple of 8; of 4 for fp32) take the vectorised kernels; anything else
 * takes the general kernel.
 *
 * Streams and errors. Work is enqueued on `stream` (a cudaStream_t; NULL is the
 * legacy default stream) and the call returns at once. Kernels are launched
 * with programmatic dependent launch allowed: a kernel may be scheduled while
 * the previous kernel on the stream finishes, but it touches no memory before
 * that kernel has completed, so stream order is kept. The return value
 * reports argument errors (checked on the host before any CUDA call) and launch
 * errors only. Kernels with bounded waits record a timeout in a per-device
 * status word instead of hanging; rmsnorm_check_device_status() reads it.
 * Calls are thread-safe. rmsnorm_last_error() gives a detail string for the
 * last failed call on the calling thread.
 */
#ifndef RMSNORM_GB300_H
#define RMSNORM_GB300_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define RMSNORM_GB300_VERSION 1

typedef enum rmsnorm_dtype {
    RMSNORM_DTYPE_BF16 = 0,
    RMSNORM_DTYPE_FP16 = 1,
    RMSNORM_DTYPE_FP32 = 2
} rmsnorm_dtype_t;

typedef enum rmsnorm_status {
    RMSNORM_OK = 0,
    RMSNORM_ERR_NULL = -1,           /* a required pointer is NULL */
    RMSNORM_ERR_SHAPE = -2,          /* M < 0, N <= 0, or x larger than 2^48 bytes */
    RMSNORM_ERR_DTYPE = -3,          /* dtype is not an rmsnorm_dtype_t value */
    RMSNORM_ERR_SCALAR = -4,         /* eps negative or not finite, or offset not finite */
    RMSNORM_ERR_EPS = -4,            /* the same code under the name of the eps check */
    RMSNORM_ERR_OVERLAP = -5,        /* buffers overlap other than y == x exactly */
    RMSNORM_ERR_CUDA = -6,           /* a CUDA runtime call or launch failed */
    RMSNORM_ERR_DEVICE_TIMEOUT = -7, /* a kernel's bounded wait ran out (see rmsnorm_check_device_status) */
    RMSNORM_ERR_UNSUPPORTED = -8,    /* the forced variant cannot take these arguments */
    RMSNORM_ERR_OPTIONS = -9,        /* malformed rmsnorm_options_t */
    RMSNORM_ERR_ALIGN = -10,         /* x, w or y not aligned to their element size, or rstd not
                                        4-byte aligned */
    RMSNORM_ERR_WORKSPACE = -11,     /* the backward's workspace is smaller than it needs */
    RMSNORM_ERR_DEVICE_INDEX = -12   /* a kernel met a slot, page or row index out of range and
                                        skipped it (see rmsnorm_check_device_status) */
} rmsnorm_status_t;

/* Kernel variants. RMSNORM_VARIANT_AUTO lets the planner choose. */
typedef enum rmsnorm_variant {
    RMSNORM_VARIANT_AUTO = 0,
    /* A team of 1..32 lanes of one warp per row, row held in registers,
     * several rows per warp when N is small (warp-per-row and
     * multi-row-per-warp). Needs 16-byte alignment and rows of whole 16-byte
     * vectors, at most 2 KB per row (N <= 1024 bf16/fp16, 512 fp32). */
    RMSNORM_VARIANT_WARP = 1,
    /* One CTA per row, row held in registers across the CTA, cross-warp sum
     * through shared memory. Needs 16-byte alignment and rows of whole 16-byte
     * vectors, at most 64 KB per row (N <= 32768 bf16/fp16, 16384 fp32). */
    RMSNORM_VARIANT_CTA = 2,
    /* Rows staged in shared memory by TMA bulk copies (cp.async.bulk with an
     * mbarrier), multi-stage pipeline, bounded waits. Needs 16-byte alignment
     * and rows of whole 16-byte vectors; rows up to the shared-memory limit. */
    RMSNORM_VARIANT_TMA = 3,
    /* Any alignment and any N: one CTA per row, two passes over the row. */
    RMSNORM_VARIANT_GENERIC = 4,
    /* Rows longer than one CTA's shared memory: a row split over a thread-block
     * cluster of 2..16 CTAs, each staging its column slice by TMA bulk copy; the
     * slice sums meet through distributed shared memory. Needs 16-byte alignment
     * and rows of whole 16-byte vectors; rows up to 16 slices of about 70 KB. */
    RMSNORM_VARIANT_CLUSTER = 5
} rmsnorm_variant_t;

/* Optional knobs for rmsnorm_fwd_ex(). Zero-initialise, then set fields. */
/* rmsnorm_options_t.flags bits. */
#define RMSNORM_FLAG_NO_PDL 1       /* launch without programmatic dependent launch */
#define RMSNORM_FLAG_BLOCKED_ROWS 2 /* each CTA takes one contiguous block of rows
                                       (default: CTAs stride over rows in passes) */
/* The caller promises that no kernel still running earlier on the stream
 * writes x or w. The kernel may then start reading them while the previous
 * kernel finishes (overlapping launches); its writes of y and rstd still wait
 * for that kernel to complete. Without the promise every read and write waits
 * (the kernel may still ask for its first rows of x to be brought into L2
 * before it waits: a hint that returns no values, see prewait_prefetch).
 * Ignored with RMSNORM_FLAG_NO_PDL and by the general kernel. */
#define RMSNORM_FLAG_EARLY_LOADS 4
/* The caller promises only that no kernel still running earlier on the stream
 * writes w (a weight that is not being updated, as in inference); x may be
 * the previous kernel's output. The kernel then reads w before the previous
 * kernel finishes and waits only before reading x, taking the weight load off
 * the critical path of a chain of dependent kernels. Ignored with
 * RMSNORM_FLAG_NO_PDL and by the general kernel; implied by EARLY_LOADS. */
#define RMSNORM_FLAG_EARLY_WEIGHTS 16
/* TMA variant with packed rows: y is written into the shared-memory stage and
 * leaves with one bulk copy (cp.async.bulk shared -> global) per stage instead
 * of per-thread stores. Ignored by the other variants and for strided rows. */
#define RMSNORM_FLAG_BULK_STORE 32
/* rmsnorm_fwd_host only: no ring and no copies; the kernel reads x and writes
 * y and rstd in page-locked host memory through their device addresses (the
 * GPU's own loads and stores cross the host link). Needs every host buffer to
 * be page-locked (cudaHostAlloc / cudaHostRegister), else
 * RMSNORM_ERR_UNSUPPORTED; takes no workspace; only the plain-load kernels
 * (WARP, CTA, GENERIC) run. Ignored by the device-memory calls. */
#define RMSNORM_FLAG_HOST_DIRECT 8

typedef struct rmsnorm_options {
    int32_t struct_size;     /* sizeof(rmsnorm_options_t) */
    int32_t variant;         /* rmsnorm_variant_t; 0 = automatic */
    int32_t max_ctas;        /* >0 caps the persistent grid; 0 = SMs x resident CTAs */
    int32_t lanes_per_row;   /* WARP: lanes per row (1..32, power of two); CTA: threads per
                                row (= per CTA); TMA: threads per row (16..1024);
                                GENERIC: threads per CTA; 0 = planner's choice */
    int32_t stages;          /* WARP: rows each team keeps in flight (1, 2 or 4); TMA: pipeline
                                depth (1..8); CLUSTER: 1..4; 0 = planner's choice */
    int32_t rows_per_stage;  /* TMA: rows per stage; 0 = planner's choice */
    int32_t flags;           /* RMSNORM_FLAG_* bits */
    int32_t cluster_size;    /* CLUSTER: CTAs per row (2..16); 0 = planner's choice */
    int64_t wait_limit_ns;   /* TMA: bound on each mbarrier wait in ns; 0 = 1 second */
    int32_t l2_prefetch;     /* WARP and TMA: L2 prefetch distance (a hint: cp.async.bulk.
                                prefetch.L2, no effect on results). WARP: each team asks
                                for its rows this many passes past the ones held in
                                registers to be brought into L2; TMA: each CTA, for this
                                many chunks past its ring's stages (packed rows; not in
                                the 512-thread plans nor fp16 plans of 128-thread teams
                                and up, where it reads 0). Ignored by the other variants
                                and by rmsnorm_bwd. 1..15; 0 = planner's choice; -1 = none */
    int32_t prewait_prefetch; /* WARP and TMA: before it waits for the previous kernel on
                                the stream, the kernel asks for its first rows to be brought
                                into L2 (cp.async.bulk.prefetch.L2, a hint: x is still read
                                after the wait, so the stream order is kept) and the WARP
                                kernel lets the next kernel be scheduled at once. WARP: this
                                many passes of each team's rows; TMA: this many chunks of
                                each CTA's. Under RMSNORM_FLAG_EARLY_LOADS a positive count
                                (or the planner, for the shapes where it measured faster)
                                replaces the loads before the wait with it; -1 keeps them.
                                rmsnorm_bwd: the warp and CTA row kernels prefetch this many
                                of their first rows of x and dy (default 1). Ignored by the
                                other variants. With RMSNORM_FLAG_NO_PDL the planner never
                                picks it and the forward TMA kernel ignores a count.
                                1..15; 0 = planner's choice; -1 = none */
} rmsnorm_options_t;

/* What the planner picked (rmsnorm_plan_info). */
typedef struct rmsnorm_plan {
    int32_t variant;         /* rmsnorm_variant_t actually launched */
    int32_t threads;         /* threads per CTA */
    int32_t grid;            /* CTAs launched (persistent grid) */
    int32_t lanes_per_row;   /* threads cooperating on one row */
    int32_t vecs_per_lane;   /* 16-byte vectors each thread holds per row (0: general kernel) */
    int32_t rows_per_stage;  /* TMA variant: rows per shared-memory stage (else 0) */
    int32_t stages;          /* TMA variant: pipeline depth (else 0) */
    int32_t smem_bytes;      /* dynamic shared memory per CTA */
    int32_t ctas_per_sm;     /* resident CTAs per SM (occupancy calculator) */
    int32_t sm_count;        /* SMs on the device */
    int32_t cluster_size;    /* CTAs per cluster (cluster variant; else 0) */
    int32_t l2_prefetch;     /* L2 prefetch distance in use (WARP, TMA; 0 = none) */
    int32_t prewait_prefetch; /* pre-wait L2 prefetch in use (WARP passes, TMA chunks; 0 =
                                none); when positive, x is read only after the wait */
} rmsnorm_plan_t;

/*
 * RMSNorm forward: y = x * rsqrt(mean(x^2) + eps) * (offset + w), rstd kept.
 *   x, w, y, rstd  device pointers as described above (x and y may be NULL
 *                  when M == 0, rstd may always be NULL; w must not be NULL)
 *   M              rows (>= 0; M == 0 launches nothing and returns RMSNORM_OK)
 *   N              columns (> 0)
 *   eps            >= 0 and finite; added to the mean of squares inside the root
 *   offset         finite; 0 = Llama, 1 = Gemma
 *   dtype          rmsnorm_dtype_t of x, w and y
 *   stream         cudaStream_t to enqueue on (NULL = legacy default stream)
 * Returns RMSNORM_OK or a negative rmsnorm_status_t; on error nothing is
 * launched and rmsnorm_last_error() says why.
 */
int rmsnorm_fwd(const void* x, const void* w, void* y, float* rstd, int64_t M, int64_t N,
                float eps, float offset, int dtype, void* stream);

/* rmsnorm_fwd with explicit options (variant choice, grid cap, pipeline depth,
 * wait bound). `opts` may be NULL (same as rmsnorm_fwd). */
int rmsnorm_fwd_ex(const void* x, const void* w, void* y, float* rstd, int64_t M, int64_t N,
                   float eps, float offset, int dtype, const rmsnorm_options_t* opts,
                   void* stream);

/* rmsnorm_fwd_ex over strided rows: row i of x starts at element i*ldx, row i
 * of y at element i*ldy (ldx, ldy >= N; in place needs y == x and ldy == ldx).
 * The vectorised kernels additionally need ldx and ldy to be multiples of 8;
 * other strides take the general kernel. Same operation and errors as
 * rmsnorm_fwd; RMSNORM_ERR_SHAPE if a stride is below N. */
int rmsnorm_fwd_strided(const void* x, int64_t ldx, const void* w, void* y, int64_t ldy,
                        float* rstd, int64_t M, int64_t N, float eps, float offset, int dtype,
                        const rmsnorm_options_t* opts, void* stream);

/*
 * The forward over activations in HOST memory. The pages' kernels take device
 * tensors and have no counterpart for this; it is the library's data path for
 * activations that live in host memory (offloaded or served from host RAM).
 * Same operation and arguments as rmsnorm_fwd_ex, except:
 *   x_host, y_host  [M, N] contiguous, in host memory (pinned with
 *                   cudaHostAlloc/cudaHostRegister for the copies to run
 *                   asynchronously and overlap; pageable memory is correct but
 *                   slower); y_host may equal x_host exactly
 *   rstd_host       [M] fp32 in host memory, or NULL
 *   w               [N] DEVICE pointer (weights stay resident)
 *   chunk_rows      rows moved per chunk (> 0), or 0 for about 4 MiB of x
 *   workspace       DEVICE memory, 16-byte aligned, of workspace_bytes >=
 *                   rmsnorm_fwd_host_workspace_size(M, N, dtype, chunk_rows);
 *                   owned by the caller, used by this call until it completes
 *                   on `stream`, and not to be shared with work running at the
 *                   same time
 * Unless RMSNORM_FLAG_HOST_DIRECT is set (see there; then the workspace may be
 * NULL), rows move in chunks through a ring of up to four slots of the workspace:
 * host->device copies of x on a copy-in stream, the forward kernel in place on
 * each slot on `stream`, device->host copies of y and rstd on a copy-out
 * stream, chained by events. The two copy streams are the library's, one pair
 * per device (made on first use, with that device current, and kept for the
 * life of the process). Both directions of the host link thus run at once.
 * The copy-in stream first waits for the work already on `stream`, and before
 * returning `stream` is made to wait for the last copy-out, so work enqueued
 * on `stream` after this call sees y and rstd in host memory; the host must
 * not read them before that work (or a stream synchronisation) completes.
 * RMSNORM_FLAG_EARLY_LOADS is ignored.
 * Errors: as rmsnorm_fwd_ex, plus RMSNORM_ERR_NULL (workspace), _ALIGN
 * (workspace), _WORKSPACE (too small), _OVERLAP (workspace against x, y, rstd
 * or w), _CUDA. Argument errors are found before anything is enqueued.
 */
int rmsnorm_fwd_host(const void* x_host, const void* w, void* y_host, float* rstd_host, int64_t M,
                     int64_t N, float eps, float offset, int dtype, int64_t chunk_rows,
                     void* workspace, int64_t workspace_bytes, const rmsnorm_options_t* opts,
                     void* stream);

/* Device workspace bytes rmsnorm_fwd_host needs for these sizes and chunk rows
 * (written to *bytes; 0 when M == 0). No CUDA call. */
int rmsnorm_fwd_host_workspace_size(int64_t M, int64_t N, int dtype, int64_t chunk_rows,
                                    int64_t* bytes);

/* Fills *out with the launch rmsnorm_fwd_ex would make for these arguments on
 * the current device (no launch). x, w, y are used only for their alignment
 * and may be any values with the alignment the real call will have. */
int rmsnorm_plan_info(int64_t M, int64_t N, int dtype, const void* x, const void* w,
                      const void* y, const rmsnorm_options_t* opts, rmsnorm_plan_t* out);

/*
 * Backward, consuming the rstd the forward kept. The pages state only that
 * rstd is kept "for backward"; the formulas are the chain rule of the forward
 * above (s_j = offset + w_j):
 *   c_i   = sum_j dy[i,j] * s_j * x[i,j]
 *   dx    = rstd[i] * (dy[i,j] * s_j - x[i,j] * rstd[i]^2 * c_i / N)   (x's dtype)
 *   dw[j] = sum_i dy[i,j] * x[i,j] * rstd[i]                              (fp32)
 * fp32 arithmetic; dx rounded once to nearest even; dw summed per CTA over its
 * rows, then over CTAs in a fixed order (deterministic for a fixed device).
 * The sum over CTAs is a second launch.
 *   x, dy, dx  [M, N] x's dtype (bf16, fp16 or fp32), contiguous; dx may equal
 *              x or dy exactly
 *   w          [N]    x's dtype
 *   rstd       [M]    fp32, as written by rmsnorm_fwd
 *   dw         [N]    fp32 output (overwritten; zero when M == 0)
 *   workspace  device scratch of at least rmsnorm_bwd_workspace_size() bytes,
 *              16-byte aligned, owned by the caller; its contents are
 *              overwritten. Calls sharing one workspace must not overlap on
 *              the GPU (one stream, or ordered streams).
 * With N % 8 == 0 and 16-byte aligned buffers, rows of up to 1024 columns take
 * a warp-per-row kernel and rows of up to 16384 columns a CTA-per-row kernel
 * (variant TMA: rows of up to 16 KB staged into shared memory by bulk copies,
 * bounded waits as in the forward, reported by rmsnorm_check_device_status);
 * others the general kernel, which keeps a CTA's dw partial row in shared memory
 * up to about 56K columns and, past that, in its own row of the workspace (any
 * N; the grid is then capped so that the partial rows stay within 64 MB).
 * Options: variant AUTO, WARP, CTA or GENERIC, lanes_per_row (CTA: threads per
 * CTA), max_ctas, RMSNORM_FLAG_NO_PDL, and
 * RMSNORM_FLAG_EARLY_LOADS, which here is the caller's promise that no kernel
 * still running earlier on the stream writes x, w or rstd (dy may be that
 * kernel's output, as in a chain of backward kernels): the warp and CTA
 * kernels then read the weights and their first row's x and rstd before that
 * kernel completes, and dy and every store only after it.
 */
int rmsnorm_bwd(const void* x, const void* w, const float* rstd, const void* dy, void* dx,
                float* dw, int64_t M, int64_t N, float offset, int dtype, void* workspace,
                int64_t workspace_bytes, const rmsnorm_options_t* opts, void* stream);

/*
 * rmsnorm_bwd without a workspace; allocates nothing. (The pages have no
 * counterpart: this entry point exists for callers, not for the method.)
 * Some callers cannot allocate device memory at the point of the call: a
 * plugin inside a host framework that owns every device allocation, or a
 * real-time path whose memory plan is fixed at start-up. Here the dw partials
 * go to a fixed 8 MiB fp32 array built into the library, which every GPU that
 * loads the library holds until the process exits. The grid is capped so that
 * grid * N fits in it; N above 2^21 is rejected with RMSNORM_ERR_WORKSPACE.
 * The first call on a device looks up the array's device address (a CUDA
 * runtime call, with that device current); make that first call before any
 * stream capture. All calls on a device share the array, and each call
 * overwrites the part it uses before reading it, so nothing carries over
 * between calls; calls that overlap on the GPU (concurrent streams) race on it.
 * Same arguments as rmsnorm_bwd otherwise; callers who can allocate should
 * prefer rmsnorm_bwd.
 */
int rmsnorm_bwd_noalloc(const void* x, const void* w, const float* rstd, const void* dy, void* dx,
                        float* dw, int64_t M, int64_t N, float offset, int dtype,
                        const rmsnorm_options_t* opts, void* stream);

/* Fills *out with the launch of the row kernel rmsnorm_bwd would make for
 * these sizes and options on the current device with 16-byte aligned buffers
 * (no launch); variant is RMSNORM_VARIANT_WARP, _CTA, _TMA or _GENERIC. */
int rmsnorm_bwd_plan_info(int64_t M, int64_t N, int dtype, const rmsnorm_options_t* opts,
                          rmsnorm_plan_t* out);

/* Bytes of workspace rmsnorm_bwd needs for these sizes and options on the
 * current device, for any buffer alignment (written to *bytes). */
int rmsnorm_bwd_workspace_size(int64_t M, int64_t N, int dtype, const rmsnorm_options_t* opts,
                               int64_t* bytes);

/* ---------------------------------------------------------------------------
 * The operators of a transformer block between its matrix products: the norms
 * around a block (rmsnorm_block_*), the rotation of the heads of q and k with
 * each head's norm (rmsnorm_rope_*), and the quantised cache that k and v go
 * into (rmsnorm_cache_*). Their arguments come in structs: zero-initialise,
 * set struct_size to the struct's size, then the fields.
 * Common to all of them: device pointers on the current device; tensors bf16,
 * fp16 or fp32 (one dtype per call) with elements aligned to their size; fp32
 * arithmetic, one rounding to nearest even per output; deterministic results;
 * work enqueued on `stream`, launched like the forward (programmatic dependent
 * launch, stream order kept); capturable into a CUDA graph. Strides are in
 * elements. Whole 16-byte vectors (row or head size, strides and pointers)
 * take the vector kernels: block rows of up to 2048 vectors, its backward's of
 * up to 32768 columns; heads of up to 64 vectors (halves of an even number of
 * values); cache heads of whole groups. Anything else takes the element-wise
 * ones, and so, without an explicit variant, does the block's backward of rows of
 * at most 128 columns where that is faster. `opts` may be
 * NULL; they read variant (AUTO, CTA: the vector kernels, GENERIC: the
 * element-wise kernels), max_ctas (a cap on persistent grids: not on the kernels of
 * rmsnorm_cache_attention that take prompts and that join parts, and of at least one CTA
 * a block of up to 8 key heads there), RMSNORM_FLAG_NO_PDL and wait_limit_ns (the block
 * operator's kernels that stage rows, attention's for prompts).
 * ------------------------------------------------------------------------- */

/*
 * The norm after a block, the block's gate, the scaled residual and the norm
 * before the next block, in one pass over the rows:
 *
 *   n    = h * rstd_post * (offset + w_post)     rstd_post = 1/sqrt(mean(h^2) + eps)
 *   s    = beta * r + alpha * gate * n
 *   y    = s * rstd_pre * (offset + w_pre)       rstd_pre = 1/sqrt(mean(s^2) + eps)
 *
 * s is the new residual stream; y is normed from s in fp32, before s is
 * rounded for its store.
 *   h, r   [M, N] the block's output and the residual stream (row strides ldh, ldr >= N)
 *   w_post [N]    NULL: no norm after the block (n = h)
 *   gate   [ceil(M / gate_rows), N] (row stride ldg >= N), row i of h takes gate row
 *                 i / gate_rows: gate_rows >= M is one gate per channel, the tokens per
 *                 sequence one gate per sequence, 1 a gate per element. NULL (and
 *                 gate_rows 0, which without rows is not looked at): no gate
 *   w_pre  [N]    NULL: no norm before the next block (y is then not written and NULL)
 *   s, y   [M, N] outputs (row strides lds, ldy >= N)
 *   rstd_post, rstd_pre  [M] fp32, kept for the backward; NULL: not stored
 * At least one of w_post and w_pre is given. s and y may each equal h or r
 * exactly (pointer and stride); no other overlap of an output with anything.
 */
typedef struct rmsnorm_block_args {
    int32_t struct_size; /* sizeof(rmsnorm_block_args_t) */
    int32_t dtype;       /* rmsnorm_dtype_t */
    int64_t M;           /* rows (>= 0) */
    int64_t N;           /* columns (> 0) */
    int64_t gate_rows;   /* rows of h per gate row; 0 without a gate */
    const void* h;
    const void* r;
    const void* w_post;
    const void* gate;
    const void* w_pre;
    void* s;
    void* y;
    float* rstd_post;
    float* rstd_pre;
    int64_t ldh;
    int64_t ldr;
    int64_t ldg;
    int64_t lds;
    int64_t ldy;
    float eps;    /* >= 0 and finite, both norms */
    float offset; /* finite, both norms: 0 or 1 as in rmsnorm_fwd */
    float alpha;  /* finite: scale of the block's branch */
    float beta;   /* finite: scale of the residual */
} rmsnorm_block_args_t;

int rmsnorm_block_fwd(const rmsnorm_block_args_t* args, const rmsnorm_options_t* opts,
                      void* stream);

/*
 * Its backward, from the gradients dy of y and ds of s, the saved s (as the
 * forward stored it), the kept rstd and h, w_post, gate, w_pre (args.r, args.y
 * and args.eps are not read):
 *
 *   t     = ds + rstd_pre * (u - s * rstd_pre^2 * sum(u s) / N)    u = dy * (offset + w_pre)
 *   dr    = beta * t
 *   dh    = rstd_post * (v - h * rstd_post^2 * sum(v h) / N)       v = alpha * gate * t * (offset + w_post)
 *   dgate = sum over the gate row's rows of alpha * t * n
 *   dw_post = sum over rows of alpha * gate * t * h * rstd_post
 *   dw_pre  = sum over rows of dy * s * rstd_pre
 *
 * (without w_post: dh = alpha * gate * t; without w_pre: t = ds).
 *   dy, ds  [M, N] dy is given exactly when w_pre is; ds may be NULL (zero) when dy is given
 *   dh, dr  [M, N] outputs; each may equal dy, ds, h or s exactly
 *   dgate   like gate (row stride lddg), given exactly when gate is
 *   dw_post, dw_pre  [N] fp32, given exactly when w_post, w_pre are (zero when M == 0)
 * Row sums are over fixed threads in a fixed order; the sums over rows are
 * taken per CTA and then over CTAs in a fixed order by a second launch.
 *   workspace  device scratch of rmsnorm_block_bwd_workspace_size() bytes, 16-byte
 *              aligned; calls sharing one must not overlap on the GPU
 */
typedef struct rmsnorm_block_grads {
    int32_t struct_size; /* sizeof(rmsnorm_block_grads_t) */
    int32_t reserved;    /* 0 */
    const void* dy;
    const void* ds;
    void* dh;
    void* dr;
    void* dgate;
    float* dw_post;
    float* dw_pre;
    int64_t lddy;
    int64_t ldds;
    int64_t lddh;
    int64_t lddr;
    int64_t lddg;
} rmsnorm_block_grads_t;

int rmsnorm_block_bwd(const rmsnorm_block_args_t* args, const rmsnorm_block_grads_t* grads,
                      void* workspace, int64_t workspace_bytes, const rmsnorm_options_t* opts,
                      void* stream);

/* Bytes of workspace rmsnorm_block_bwd needs for M rows of N columns on the
 * current device, whatever the other arguments, alignments and options (written
 * to *bytes; never less for a larger M). */
int rmsnorm_block_bwd_workspace_size(int64_t M, int64_t N, int dtype, int64_t* bytes);

/* Heads of a tensor: element d of head h of token s of batch b is at
 * ptr + b * batch_stride + s * token_stride + h * head_stride + d. */
typedef struct rmsnorm_heads {
    void* ptr;
    int64_t batch_stride;
    int64_t token_stride;
    int64_t head_stride;
} rmsnorm_heads_t;

/*
 * Rotary positions on the heads of q and k, after each head's RMSNorm where
 * weights are given:
 *
 *   x = head * rstd * (offset + w)      rstd = 1/sqrt(mean over head_dim of head^2 + eps)
 *                                       (x = head without weights)
 *   out[a] = magnitude * (x[a] cos t - x[b] sin t)
 *   out[b] = magnitude * (x[b] cos t + x[a] sin t)      t = position * frequency_i
 *
 * for the pairs i < rotary_dim / 2 of the first rotary_dim values: (a, b) =
 * (i, i + rotary_dim/2), or (2i, 2i + 1) when interleaved. The values behind
 * rotary_dim stay x. Angles are exact for every 64-bit position: frequencies
 * are given as steps, the fraction of a turn per position times 2^64
 * (rmsnorm_rope_steps), so position * step wraps modulo one turn.
 *   q [batch, seq, heads_q, head_dim], k likewise with heads_k (0: no k)
 *   out_q, out_k   outputs, may equal q and k exactly (pointer and strides)
 *   positions      [batch, seq] int64 (row stride positions_stride; 0: one row for all
 *                  batches); NULL: the index in the sequence
 *   w_q, w_k       [head_dim], each may be NULL
 *   rstd_q, rstd_k [batch, seq, heads] fp32, contiguous, kept for the backward; NULL: not
 *                  stored (and without weights not written)
 */
typedef struct rmsnorm_rope_args {
    int32_t struct_size; /* sizeof(rmsnorm_rope_args_t) */
    int32_t dtype;       /* rmsnorm_dtype_t */
    int64_t batch;
    int64_t seq;
    int32_t heads_q;     /* >= 1 */
    int32_t heads_k;     /* >= 0 */
    int32_t head_dim;    /* 2..65536 */
    int32_t rotary_dim;  /* even, 2..head_dim */
    int32_t interleaved; /* 0 or 1 */
    int32_t reserved;    /* 0 */
    const int64_t* positions;
    int64_t positions_stride;
    const uint64_t* steps; /* [rotary_dim / 2] on the device */
    const void* w_q;
    const void* w_k;
    float* rstd_q;
    float* rstd_k;
    float eps;
    float offset;
    float magnitude; /* finite; 1 for plain rotation */
    float reserved_f;
    rmsnorm_heads_t q;
    rmsnorm_heads_t k;
    rmsnorm_heads_t out_q;
    rmsnorm_heads_t out_k;
} rmsnorm_rope_args_t;

int rmsnorm_rope_fwd(const rmsnorm_rope_args_t* args, const rmsnorm_options_t* opts, void* stream);

/*
 * Its backward: gradients dout_q, dout_k of the outputs are turned back by the
 * same angles (times magnitude) and go through the norm's backward where
 * weights are given, which reads q, k and the kept rstd (args.out_q, args.out_k
 * and args.eps are not read; without weights q, k and rstd are not either).
 *   dout_q, dout_k   like the outputs; strides may be 0 (expanded)
 *   dq, dk           outputs; may equal dout_q and dout_k exactly
 *   dw_q, dw_k       [head_dim] fp32 sums over all tokens and heads, given exactly when the
 *                    weights are (zero without tokens)
 *   workspace        as in rmsnorm_block_bwd (may be NULL without weights)
 */
typedef struct rmsnorm_rope_grads {
    int32_t struct_size; /* sizeof(rmsnorm_rope_grads_t) */
    int32_t reserved;    /* 0 */
    rmsnorm_heads_t dout_q;
    rmsnorm_heads_t dout_k;
    rmsnorm_heads_t dq;
    rmsnorm_heads_t dk;
    float* dw_q;
    float* dw_k;
} rmsnorm_rope_grads_t;

int rmsnorm_rope_bwd(const rmsnorm_rope_args_t* args, const rmsnorm_rope_grads_t* grads,
                     void* workspace, int64_t workspace_bytes, const rmsnorm_options_t* opts,
                     void* stream);

/* Bytes of workspace rmsnorm_rope_bwd needs with weights on the current device
 * for heads of head_dim values, any number of tokens and heads. */
int rmsnorm_rope_bwd_workspace_size(int32_t head_dim, int64_t* bytes);

/* Scaling of rotary frequencies to longer contexts. */
typedef enum rmsnorm_rope_scaling_kind {
    RMSNORM_ROPE_PLAIN = 0,
    RMSNORM_ROPE_LINEAR = 1, /* every frequency / factor */
    RMSNORM_ROPE_NTK = 2,    /* base * factor^(rotary_dim / (rotary_dim - 2)); rotary_dim > 2 */
    RMSNORM_ROPE_YARN = 3,   /* pairs that turn more than beta_fast times within `length` stay,
                                those under beta_slow times are divided by factor, a ramp over
                                the pair index between; magnitude 0.1 ln(factor) + 1 */
    RMSNORM_ROPE_BANDS = 4   /* as YARN by the turns within `length` itself, ramp between
                                beta_slow and beta_fast turns; magnitude 1 */
} rmsnorm_rope_scaling_kind_t;

typedef struct rmsnorm_rope_scaling {
    int32_t struct_size; /* sizeof(rmsnorm_rope_scaling_t) */
    int32_t kind;        /* rmsnorm_rope_scaling_kind_t */
    double factor;       /* >= 1 */
    double length;       /* YARN, BANDS: the original context (> 0) */
    double beta_fast;    /* YARN, BANDS: > beta_slow > 0 */
    double beta_slow;
} rmsnorm_rope_scaling_t;

/* The steps of the frequencies base^(-2i / rotary_dim) (scaled; NULL: plain) into
 * the HOST array steps[rotary_dim / 2], and the magnitude that goes with them
 * (may be NULL). No CUDA call. */
int rmsnorm_rope_steps(int32_t rotary_dim, double base, const rmsnorm_rope_scaling_t* scaling,
                       uint64_t* steps, float* magnitude);

/* Formats of a cached value. Groups of 32 values of a head (the last group of a
 * head may be shorter) share a scale 2^(byte - 127): the smallest such power, not
 * below 2^-127, by which every value of the group is within the format. A group
 * that holds an infinity or a NaN has scale byte 255 and reads back as NaN. */
typedef enum rmsnorm_cache_format {
    RMSNORM_CACHE_E4M3 = 0, /* 8 bits: largest 448 */
    RMSNORM_CACHE_E2M1 = 1  /* 4 bits: 0, .5, 1, 1.5, 2, 3, 4, 6; even d in the low half of a byte */
} rmsnorm_cache_format_t;

/*
 * A paged cache: slot page * page_size + i is token i of a page. Codes are
 * [pages, page_size, heads, code bytes] and scales [pages, page_size, heads,
 * ceil(head_dim / 32)] bytes, contiguous; with heads_first the heads come before
 * the tokens of the page. Code bytes: head_dim (E4M3), ceil(head_dim / 2) (E2M1).
 * v_codes and v_scales are both NULL in a cache of one tensor.
 */
typedef struct rmsnorm_cache {
    int32_t struct_size; /* sizeof(rmsnorm_cache_t) */
    int32_t format;      /* rmsnorm_cache_format_t */
    int64_t pages;       /* >= 1 */
    int32_t page_size;   /* >= 1 */
    int32_t heads;       /* >= 1 */
    int32_t head_dim;    /* 1..65536 */
    int32_t heads_first; /* 0 or 1 */
    uint8_t* k_codes;
    uint8_t* k_scales;
    uint8_t* v_codes;
    uint8_t* v_scales;
} rmsnorm_cache_t;

/*
 * Quantises k and v (tokens [T, heads, head_dim] by their token and head
 * strides; batch_stride is not read; v may be NULL) into the cache: token t
 * goes to slot slots[t] (int64 on the device; negative: the token is padding
 * and not read). A slot past the cache is skipped and reported by
 * rmsnorm_check_device_status. Slots of a call must be distinct: a slot named
 * twice ends with bytes of either token.
 */
int rmsnorm_cache_write(const rmsnorm_cache_t* cache, const rmsnorm_heads_t* k,
                        const rmsnorm_heads_t* v, const int64_t* slots, int64_t T, int dtype,
                        const rmsnorm_options_t* opts, void* stream);

/*
 * Reads a ragged batch back: row i of the outputs, for cu_rows[b] <= i <
 * cu_rows[b + 1], is token p = starts[b] + i - cu_rows[b] of sequence b, from
 * slot table[b][p / page_size] * page_size + p % page_size.
 *   table    [sequences, table_width] int32 pages, contiguous
 *   cu_rows  [sequences + 1] int32, not decreasing, cu_rows[0] = 0
 *   starts   [sequences] int32 (NULL: 0)
 *   rows     rows of the outputs; rows from cu_rows[sequences] on are left as they are
 *   k_out, v_out  [rows, heads, head_dim] by their token and head strides; either may be
 *            NULL (not both)
 * A row whose page lies outside the cache or the table is set to zero and
 * reported by rmsnorm_check_device_status.
 */
int rmsnorm_cache_read(const rmsnorm_cache_t* cache, const int32_t* table, int64_t table_width,
                       const int32_t* cu_rows, const int32_t* starts, int64_t sequences,
                       int64_t rows, const rmsnorm_heads_t* k_out, const rmsnorm_heads_t* v_out,
                       int dtype, const rmsnorm_options_t* opts, void* stream);

/*
 * Rotary positions with several axes (frames, rows and columns of images and
 * video): as rmsnorm_rope_fwd and rmsnorm_rope_bwd, but pair i turns by the position
 * of its axis. args.positions (required) are those of axis 0, axis a's lie axis_stride
 * elements further each. The pairs are dealt to the axes in sections (the first
 * pairs[0] pairs to axis 0, the next pairs[1] to axis 1, ...), or in turn: pair i
 * belongs to axis i % axes while i / axes < pairs[i % axes], and to axis 0 otherwise.
 * The frequencies (args.steps) are one per pair as before: one table over all
 * pairs, or, for axes with frequencies of their own, the axes' tables one behind
 * the other.
 */
typedef struct rmsnorm_rope_axes {
    int32_t struct_size;  /* sizeof(rmsnorm_rope_axes_t) */
    int32_t axes;         /* 1..4 */
    int32_t pairs[4];     /* of each axis, >= 0, 0 past the last; together rotary_dim / 2 */
    int32_t in_turn;      /* 0 or 1; in turn, the pairs named for every axis must lie below
                             rotary_dim / 2: axes * (pairs[a] - 1) + a for a >= 1 */
    int32_t reserved;     /* 0 */
    int64_t axis_stride;  /* >= 0 */
} rmsnorm_rope_axes_t;

int rmsnorm_rope_axes_fwd(const rmsnorm_rope_args_t* args, const rmsnorm_rope_axes_t* axes,
                          const rmsnorm_options_t* opts, void* stream);
int rmsnorm_rope_axes_bwd(const rmsnorm_rope_args_t* args, const rmsnorm_rope_axes_t* axes,
                          const rmsnorm_rope_grads_t* grads, void* workspace, int64_t workspace_bytes,
                          const rmsnorm_options_t* opts, void* stream);

/*
 * Attention of ragged queries over the cache, which is read as it is held:
 *
 *   out[i, h] = sum_t p_t v[t, h / G]     p = softmax over t of scale * q[i, h] . k[t, h / G]
 *   lse[i, h] = log of the sum over t of exp(scale * q[i, h] . k[t, h / G])
 *
 * with G = heads_q / cache heads. Rows cu_rows[b] to cu_rows[b + 1] of q and out are
 * the n newest tokens of sequence b, which holds lengths[b] tokens (the new ones among
 * them, written before the call): row cu_rows[b] + i is at position
 * lengths[b] - n + i. It sees the tokens 0 <= t < lengths[b], with causal those up to its
 * own position, with a window those after its position - window. A row that sees
 * nothing gets zeros and an lse of -infinity. Token t of sequence b lies in slot
 * table[b][t / page_size] * page_size + t % page_size; a token whose page lies outside
 * the cache or the table is left out and reported by rmsnorm_check_device_status.
 * Tokens that no row sees may hold anything; a group stored with an infinity or a NaN
 * (scale byte 255) makes NaN of what sees it: of the rows by k, of the group's values by v.
 * A code that is itself a NaN (E4M3, which rmsnorm_cache_write never stores) may reach
 * further within its tile of tokens.
 *
 * Sums and softmax statistics are held in fp32. The matrix instructions take fp16: q is exact
 * within 2^28 of its row's largest value (fp32: 22 bits of it), codes within 2^21 (8 bits; 4
 * bits: 2^35) of the largest scale beside theirs, and what lies below is off by less than
 * 2^-22 (2^-34) of that scale. Beside it are, for v, the groups of its token and head; in calls
 * of enough rows for the tensor cores, for k and v, those of the head in a run of 128 tokens.
 * Probabilities are rounded to 11 bits for 16-bit outputs and to 22 bits for fp32, with a
 * floor: p * (largest scale beside the token's v) is kept to 2^-33 of the sequence's largest
 * scale. The element-wise kernel computes all of it in fp32.
 *   cu_rows  [sequences + 1] int32, not decreasing, from 0; NULL: one row a sequence
 *            (rows == sequences)
 *   rows     rows of q and out; rows from cu_rows[sequences] on are left as they are
 *   q, out   tokens [rows, heads_q, head_dim] (batch_stride is not read); out may not
 *            overlap q; the cache must hold v, with head_dim at most 512
 *   lse      [rows, heads_q] fp32, contiguous, or NULL
 *   workspace  device scratch of rmsnorm_cache_attention_workspace_size() bytes, 16-byte
 *            aligned; calls that share one must not overlap on the GPU
 */
typedef struct rmsnorm_cache_attention_args {
    int32_t struct_size;  /* sizeof(rmsnorm_cache_attention_args_t) */
    int32_t dtype;        /* rmsnorm_dtype_t of q and out */
    int32_t heads_q;      /* a multiple of the cache's heads */
    int32_t causal;       /* 0 or 1 */
    int64_t sequences;
    int64_t rows;
    int64_t table_width;
    int64_t window;       /* tokens a row sees, its own among them; 0: no window (needs causal) */
    const int32_t* table; /* [sequences, table_width], contiguous */
    const int32_t* lengths; /* [sequences], >= 0 (below: taken as 0) */
    const int32_t* cu_rows;
    float* lse;
    float scale;          /* finite */
    float reserved;       /* 0 */
    rmsnorm_heads_t q;
    rmsnorm_heads_t out;
} rmsnorm_cache_attention_args_t;

int rmsnorm_cache_attention(const rmsnorm_cache_t* cache, const rmsnorm_cache_attention_args_t* args,
                            void* workspace, int64_t workspace_bytes, const rmsnorm_options_t* opts,
                            void* stream);

/* Bytes of workspace rmsnorm_cache_attention needs on the current device for any
 * lengths, strides and options. */
int rmsnorm_cache_attention_workspace_size(int32_t cache_heads, int32_t heads_q, int32_t head_dim,
                                           int64_t sequences, int64_t rows, int64_t* bytes);

/*
 * Pages of a cache that sequences share. refs[p] is the number of table entries that name
 * page p (0: free); an entry below 0 names none; lengths[b] tokens of sequence b lie in
 * the pages of its row of the table, from the first on.
 */
typedef struct rmsnorm_cache_pages {
    int32_t struct_size;  /* sizeof(rmsnorm_cache_pages_t) */
    int32_t reserved;     /* 0 */
    int64_t pages;        /* of the cache: 1..2^25 */
    int64_t sequences;    /* 0..2^30 */
    int64_t table_width;  /* 0..2^30 */
    int32_t* refs;        /* [pages] */
    int32_t* table;       /* [sequences, table_width], contiguous */
    int32_t* lengths;     /* [sequences]; rmsnorm_cache_compact takes NULL */
} rmsnorm_cache_pages_t;

/* Copies page src[i] to page dst[i] for i < n (int32 on the device; either below 0: no
 * copy). A page past the cache is skipped and reported by rmsnorm_check_device_status.
 * Pages in dst must be distinct and must not be in src (else they end with bytes of
 * either). */
int rmsnorm_cache_copy_pages(const rmsnorm_cache_t* cache, const int32_t* src, const int32_t* dst,
                             int64_t n, const rmsnorm_options_t* opts, void* stream);

/*
 * Makes sequence children[i] a copy of parents[i] for i < n (int32 on the device; either
 * below 0: nothing is done). Full pages are shared (refs + 1); the tokens of a last page that is
 * not full are copied into a free page, the lowest ones in the order of i; the rest of the
 * child's row becomes -1. lengths are those before the call. A child must be empty
 * (length 0; its row is overwritten). Reported by rmsnorm_check_device_status and left as it
 * is: a child that is not empty, named twice (all but the first), or its own parent; a row
 * past the table; a parent whose tokens exceed its row; a child for which no free page is
 * left. Entries of a parent's tokens that name no page of the cache, the last one's among
 * them, are copied as they are and reported (the free page that a last one would have taken
 * stays free).
 *   workspace  rmsnorm_cache_pages_workspace_size() bytes, 16-byte aligned
 */
int rmsnorm_cache_fork(const rmsnorm_cache_t* cache, const rmsnorm_cache_pages_t* pages,
                       const int32_t* parents, const int32_t* children, int64_t n, void* workspace,
                       int64_t workspace_bytes, const rmsnorm_options_t* opts, void* stream);

/* Frees the sequences rows[i], i < n (int32 on the device; below 0: none): the pages of their
 * rows lose a reference each, the rows become -1, the lengths 0. A row named twice is freed
 * once. A row past the table, an entry past the cache and a page without references are
 * skipped and reported by rmsnorm_check_device_status. */
int rmsnorm_cache_free(const rmsnorm_cache_pages_t* pages, const int32_t* rows, int64_t n,
                       const rmsnorm_options_t* opts, void* stream);

/*
 * Brings the live pages (refs > 0) together: with L of them, those from page L on move, in
 * their order, into the free pages below L, in theirs. refs_out and table_out (each may be
 * pages.refs and pages.table themselves) name the pages where they are then; live[0] = L.
 * Codes and scales of moved pages are copied, and what lies in the pages from L on stays.
 * Entries past the cache are kept and reported, those that name a free page kept.
 *   workspace  as in rmsnorm_cache_fork
 */
int rmsnorm_cache_compact(const rmsnorm_cache_t* cache, const rmsnorm_cache_pages_t* pages,
                          int32_t* refs_out, int32_t* table_out, int32_t* live, void* workspace,
                          int64_t workspace_bytes, const rmsnorm_options_t* opts, void* stream);

/* Bytes of workspace that rmsnorm_cache_fork (of n children, in a table of `sequences` rows)
 * and rmsnorm_cache_compact (n and sequences 0) need. No CUDA call. */
int rmsnorm_cache_pages_workspace_size(int64_t pages, int64_t sequences, int64_t n, int64_t* bytes);

/* Synchronises `stream`, then reads and clears the current device's status
 * word. Returns RMSNORM_OK, RMSNORM_ERR_DEVICE_TIMEOUT if any kernel since the
 * last check gave up a bounded wait, RMSNORM_ERR_DEVICE_INDEX if one met an
 * index out of range (where both happened, the next check reports the index), or
 * RMSNORM_ERR_CUDA. */
int rmsnorm_check_device_status(void* stream);

/* Static text for a status code. */
const char* rmsnorm_strerror(int status);

/* Detail of the last failed call on this thread ("" if none). */
const char* rmsnorm_last_error(void);

/* RMSNORM_GB300_VERSION of the loaded library. */
int rmsnorm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* RMSNORM_GB300_H */
