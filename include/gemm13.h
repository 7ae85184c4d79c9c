/*
 * gemm13.h -- C ABI of the GB300 (sm_103a) GEMM library.
 *
 * One operation, in two calls:
 *
 *     C = cast( act( alpha * A.B + bias ) + beta * R )
 *
 * with A, B in FP32, FP16 or BF16, all products accumulated in FP32, and the
 * whole epilogue applied in registers before C is written once.
 *
 * Where the operation is defined:
 *   - "DeepGEMM" (discosf.com), sec. 1.2: FP16/BF16 input, FP32 accumulation,
 *     and a fusion hook so activation, residual add and scaling happen before
 *     the result leaves the kernel; sec. 3.1: K is the outer loop and C is
 *     stored once; sec. 3.4: accumulate in FP32 even for 16-bit inputs;
 *     sec. 2.3 / 4.3: per-shape tile choice with a configuration cache and a
 *     small-block variant for small M or N.
 *   - "CUDA Tile ... GEMM" (pgsm.cn), sec. 4.1: row-major A (M x K), B (K x N),
 *     C (M x N): A[row*K+k], B[k*N+col], C[row*N+col]; sec. 2: the FFN
 *     linear Y = X W^T + b (B given as W[N,K]) and the batched per-head QK^T.
 *   - "SGEMM ... 83% of cuBLAS" (cf-1.com), sec. 2-3: the FP32 SGEMM on CUDA
 *     cores (FFMA), which this library keeps as its FP32 path.
 * Readings where the pages are silent: the epilogue order above, GELU in its
 * erf form, FP32 bias and residual, round-to-nearest-even output casts.
 *
 * Conventions for every call below:
 *   - Pointers to matrices are DEVICE pointers of the current CUDA device;
 *     the caller owns them.  Leading dimensions and batch strides are in
 *     ELEMENTS of the buffer's own type.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default stream).
 *   - Every int-returning call returns a gemm_status_t; none of them aborts,
 *     traps or prints (set GEMM_LOG=1 in the environment to print plan
 *     decisions to stderr).
 */
#ifndef GEMM13_H
#define GEMM13_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GEMM_F32 = 0, GEMM_F16 = 1, GEMM_BF16 = 2 } gemm_dtype_t;

/* Microscaled 4-bit formats (see "4-bit floats" below). */
typedef enum { GEMM_MXFP4 = 0, GEMM_NVFP4 = 1 } gemm_fp4_format_t;

typedef enum {
    GEMM_ACT_NONE = 0,
    GEMM_ACT_GELU_ERF = 1, /* 0.5*y*(1+erf(y/sqrt(2))) */
    GEMM_ACT_RELU = 2,     /* max(y, 0); of a NaN: 0 in gemm_run, NaN in gemm_fp4_run */
    GEMM_ACT_SOFTMAX = 3   /* softmax over each output row: exp(y_ij - max_j y_ij) divided by
                              sum_j exp(y_ij - max_j y_ij), with y = alpha*A.B + bias over all N
                              columns -- the attention step Softmax(QK^T) of "CUDA Tile ...
                              GEMM", sec. 2, fused into the GEMM.  16-bit inputs, N <= 512,
                              K >= 1, no residual (else GEMM_ERR_UNSUPPORTED). */
} gemm_act_t;

typedef enum {
    GEMM_B_KN = 0, /* B[k*ldb + n]: row-major K x N */
    GEMM_B_NK = 1  /* B[n*ldb + k]: row-major N x K ("K-major", e.g. a weight W for X.W^T) */
} gemm_blayout_t;

typedef enum {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_ARG = -1,   /* a size, stride, enum or pointer is invalid */
    GEMM_ERR_UNSUPPORTED = -2,   /* valid request this build does not implement */
    GEMM_ERR_MISALIGNED = -3,    /* a base pointer breaks the alignment the plan assumed */
    GEMM_ERR_CUDA = -4,          /* a CUDA runtime/driver call failed */
    GEMM_ERR_DEVICE_TIMEOUT = -5,/* a kernel gave up waiting on a barrier (status word) */
    GEMM_ERR_BAD_PLAN = -6,      /* NULL, destroyed or foreign plan handle */
    GEMM_ERR_NO_DEVICE = -7,     /* no usable CUDA device, or not an sm_103 device */
    GEMM_ERR_OUT_OF_MEMORY = -8, /* plan workspace could not be allocated */
    GEMM_ERR_SCRATCH_LIMIT = -9  /* gemm_run_noalloc: staged operands exceed its fixed scratch */
} gemm_status_t;

/* Plan flags (gemm_epilogue_t.flags). */
#define GEMM_FLAG_FP32_TENSOR 0x1u       /* FP32 inputs: the dispatcher may pick the 3xTF32
                                            tensor-core kernel (GEMM_KERNEL_TF32X3) for large
                                            problems instead of the CUDA-core FFMA kernel; the
                                            result meets the same tolerance */
#define GEMM_FLAG_TEST_STALL 0x80000000u /* test only: the first CTA's producer withholds one
                                            operand tile so its waits run out; with a short
                                            timeout_ms this exercises the timeout path */
#define GEMM_FLAG_TEST_STALL_PEER 0x40000000u /* test only: as GEMM_FLAG_TEST_STALL, for the
                                                 second CTA (tensor-core kernel: the odd CTA of
                                                 the first CTA pair) */

/*
 * Everything about a call besides (dtype, M, N, K, lda, ldb, ldc).  Pass NULL
 * to gemm_plan for plain C = alpha*A.B in FP32 with B in KN layout, batch 1.
 * Start from gemm_epilogue_init() so new fields keep their defaults.
 */
typedef struct {
    gemm_blayout_t b_layout; /* default GEMM_B_KN */
    gemm_dtype_t out_dtype;  /* GEMM_F32 (default), GEMM_BF16 or GEMM_F16; RNE cast */
    int has_bias;            /* 1: bias[N] FP32 added after the alpha scale */
    gemm_act_t act;          /* applied after bias, before the residual (softmax: per row) */
    int has_residual;        /* 1: beta * R[M,N] (FP32, row-major, ldr) added last */
    float beta;              /* residual scale, default 1 */
    int64_t ldr;             /* residual leading dimension; 0 means ldc */
    int64_t batch;           /* number of independent products, default 1 */
    int64_t stride_a;        /* elements between consecutive A matrices (0: shared A) */
    int64_t stride_b;        /* elements between consecutive B matrices (0: shared B) */
    int64_t stride_c;        /* elements between consecutive C matrices; >= M*ldc if batch > 1 */
    int64_t stride_r;        /* elements between consecutive R matrices (0: shared R) */
    uint32_t flags;          /* GEMM_FLAG_* */
    uint32_t timeout_ms;     /* per-wait device timeout; 0 means 2000 ms */
} gemm_epilogue_t;

/* Kernel families a plan can use. */
typedef enum {
    GEMM_KERNEL_AUTO = 0,   /* let the dispatcher choose */
    GEMM_KERNEL_TC = 1,     /* tcgen05 tensor cores, TMA + mbarrier ring, TMEM accumulators (16-bit in) */
    GEMM_KERNEL_FFMA = 2,   /* CUDA-core FP32 FFMA, TMA-fed (FP32 in) */
    GEMM_KERNEL_SKINNY = 3, /* memory-bound streaming kernel for small M or N (any input type;
                               the dispatcher uses it for min(M, N) <= 4 and for K == 0) */
    GEMM_KERNEL_TF32X3 = 4  /* FP32 in on the tensor cores (tcgen05 kind::tf32): each operand
                               is split x = hi + lo into two TF32 numbers by a pre-pass and
                               A.B ~ Ahi.Bhi + Ahi.Blo + Alo.Bhi (the "SGEMM ... 83% of cuBLAS"
                               page, sec. 6, names the TF32 tensor-core path as the next step
                               past FFMA; splitting recovers FP32-level accuracy).  Needs a plan
                               workspace of 2 x (M + N) x K FP32 values per batch entry. */
} gemm_kernel_t;

/* A tile configuration: what the dispatcher chose, or what a caller forces. */
typedef struct {
    gemm_kernel_t kernel;
    int32_t bm, bn, bk;   /* output tile and K step (elements) */
    int32_t stages;       /* shared-memory pipeline depth */
    int32_t split_k;      /* K slices reduced deterministically (1 = none) */
    int32_t raster_group; /* M tiles walked together for L2 reuse */
    int32_t stage_a;      /* 1: A is first copied to an aligned plan workspace */
    int32_t stage_b;      /* 1: B likewise */
    int32_t num_ctas;     /* persistent grid size; 0 = one per SM */
    int32_t variant;      /* family-specific main-loop variant; FFMA: 0 scalar FFMA,
                             1 packed fma.rn.f32x2 (KN layout only), 2 32 x 32 tiles from
                             plain loads for small M x N (bm = bn = bk = 32, any stride or
                             alignment, no stream-K); TC: 0 single CTAs with
                             4 epilogue warps, 1 single CTAs with 8 epilogue warps (short K),
                             2 CTA pairs (cta_group::2, 256 x 256 tiles, no split-K),
                             3 CTA pairs with 8 epilogue warps (bn 256, 5 stages);
                             TF32X3: 0 single CTAs (bn 128), 2 CTA pairs (bn 256) */
    int32_t stream_k;     /* FFMA and TC: 1 = persistent grid with (tile, K-step) units split
                             evenly over the CTAs (CTA pairs); a tile cut between them is
                             finished by the holder of its first K step, which adds the others'
                             partial sums in a fixed order (deterministic).  Needs a plan
                             workspace of grid x 64 KB (FFMA) or grid x 128 x bn x 4 bytes (TC);
                             TC: no split-K, no row softmax. */
} gemm_config_t;

typedef struct gemm_plan_s* gemm_plan_t;

/* Fills *e with the defaults listed above. */
void gemm_epilogue_init(gemm_epilogue_t* e);

/*
 * Validates a problem, picks (or fetches from the per-process cache) a tile
 * configuration, and allocates the plan's device state on the CURRENT device:
 * a status word and, only when a stride or base alignment rules out direct TMA
 * loads, a workspace for aligned operand copies (gemm_plan_info reports its
 * size).  No kernel runs.
 *   M, N, K >= 0 (M or N == 0: runs do nothing; K == 0: C = epilogue(0)).
 *   lda >= K, ldb >= N (KN) or >= K (NK), ldc >= N, ldr >= N.
 * Errors: INVALID_ARG, UNSUPPORTED, NO_DEVICE, OUT_OF_MEMORY, CUDA.
 * On success *out_plan owns its state until gemm_plan_destroy.
 */
int gemm_plan(gemm_dtype_t dtype, int64_t M, int64_t N, int64_t K,
              int64_t lda, int64_t ldb, int64_t ldc,
              const gemm_epilogue_t* epilogue, gemm_plan_t* out_plan);

/* As gemm_plan, with the configuration forced (cfg->kernel may not be AUTO).
 * Fields a family does not use are ignored; invalid combinations return
 * INVALID_ARG or UNSUPPORTED.  Meant for tests and tuning. */
int gemm_plan_with_config(gemm_dtype_t dtype, int64_t M, int64_t N, int64_t K,
                          int64_t lda, int64_t ldb, int64_t ldc,
                          const gemm_epilogue_t* epilogue, const gemm_config_t* cfg,
                          gemm_plan_t* out_plan);

/*
 * Enqueues the GEMM on `stream` and returns without synchronising.
 *   A: dtype, [batch][M][lda];  B: dtype, [batch][K][ldb] (KN) or [batch][N][ldb] (NK);
 *   C: out_dtype, [batch][M][ldc];  bias: FP32 [N] (must be NULL iff !has_bias);
 *   residual: FP32 [batch][M][ldr] (NULL iff !has_residual).
 * C must not overlap A, B, bias or residual.  Allocates nothing.  Runs of
 * one plan on different streams may overlap on the GPU unless the plan has a
 * staging workspace (gemm_plan_info(...).workspace_bytes > 0): those runs
 * share it and must be ordered.
 * Errors: BAD_PLAN, INVALID_ARG (NULL pointer), MISALIGNED, CUDA (launch failed).
 * A device-side timeout is reported later by gemm_plan_status.
 */
int gemm_run(gemm_plan_t plan, const void* A, const void* B, void* C,
             const void* bias, const void* residual, float alpha, void* stream);

/* Synchronises the device, then reports GEMM_ERR_DEVICE_TIMEOUT if any kernel
 * of this plan gave up on a wait since the plan was made, else GEMM_OK.  The
 * condition is sticky.  Errors: BAD_PLAN, CUDA. */
int gemm_plan_status(gemm_plan_t plan);

/* Information about a plan. */
typedef struct {
    gemm_config_t config;
    int64_t workspace_bytes; /* device bytes owned by the plan besides its status word */
    int32_t num_sms;         /* SMs of the plan's device */
    int32_t device;          /* CUDA ordinal */
    int32_t cache_hit;       /* 1 if gemm_plan found the config in the cache */
    int32_t kernels_per_run; /* kernel launches one gemm_run makes (0 for empty problems) */
} gemm_plan_info_t;

int gemm_plan_info(gemm_plan_t plan, gemm_plan_info_t* out);

/* Releases a plan (NULL is a no-op).  Runs still in flight must finish first. */
void gemm_plan_destroy(gemm_plan_t plan);

/*
 * Host-only: the configuration the dispatcher would choose for this problem
 * on a device with `num_sms` SMs.  Touches no CUDA state and does not use the
 * cache.  Errors: INVALID_ARG, UNSUPPORTED.
 */
int gemm_select_config(gemm_dtype_t dtype, int64_t M, int64_t N, int64_t K,
                       int64_t lda, int64_t ldb, int64_t ldc,
                       const gemm_epilogue_t* epilogue, int32_t num_sms,
                       gemm_config_t* out);

/* Configuration cache: entries, hits and misses since start (or last clear). */
void gemm_cache_stats(int64_t* entries, int64_t* hits, int64_t* misses);
void gemm_cache_clear(void);

/* Static text for a status code ("unknown status" for others). */
const char* gemm_strerror(int status);

/* Library version string. */
const char* gemm_version(void);

/*
 * gemm_run_noalloc -- the same GEMM as gemm_plan + gemm_run in one call that
 * allocates no memory (no cudaMalloc, no plan, no host heap) once its
 * per-device set-up (below) has run.  The
 * pages have no counterpart: this exists for callers that cannot allocate
 * device memory where they run a GEMM -- code inside an allocator or memory-
 * pool callback, code holding a lock the allocator also takes, or programs
 * that reserve all device memory up front.
 *
 * Arguments: as gemm_plan followed by gemm_run (same meaning, layout and
 * validation; epilogue may be NULL).  A, B, C, bias and residual are the
 * caller's device buffers; the call enqueues on `stream` and returns.
 *
 * Scratch: operands that TMA cannot read in place (strides or base addresses
 * not 16-byte aligned) are copied into a fixed 64 MiB device array inside the
 * library, one per GPU, resident from the set-up until process exit.  The
 * array also holds the status word.  If the staged copies need more than
 * that (each staged row padded to 16 bytes, 256 bytes reserved), the call
 * returns GEMM_ERR_SCRATCH_LIMIT and does nothing.
 *
 * Sharing: every call on a device uses the same array and finds the previous
 * call's data in it (it rewrites what it uses).  Calls whose work overlaps on
 * the GPU -- on different streams or from several threads -- race on the
 * array; order them on one stream.
 *
 * Device timeouts: if a kernel gives up on a device-side wait (default limit
 * 2 s per wait), C is left undefined (partly written).  This call cannot
 * report that (there is no plan whose status could be queried); callers that
 * need to know use gemm_plan / gemm_run / gemm_plan_status.
 *
 * Set-up: the first call on each device and CUDA context (with that device
 * current) looks up the array's device address and loads every kernel this
 * entry point can launch.  Under CUDA's lazy module loading both steps make
 * the CUDA driver allocate device memory, so make that first call before the
 * code that must not allocate, and before any stream capture.  A call with
 * M = 0 or N = 0 performs the set-up and nothing else.
 *
 * Errors: INVALID_ARG, UNSUPPORTED, SCRATCH_LIMIT, NO_DEVICE, CUDA.
 */
int gemm_run_noalloc(gemm_dtype_t dtype, int64_t M, int64_t N, int64_t K,
                     const void* A, int64_t lda, const void* B, int64_t ldb,
                     void* C, int64_t ldc, const gemm_epilogue_t* epilogue,
                     const void* bias, const void* residual, float alpha, void* stream);

/*
 * 4-bit floats.  A matrix [rows][cols] in 4 bits is two device arrays, and for
 * GEMM_NVFP4 an FP32 scale g of the whole tensor:
 *   codes   E2M1 values (+-0, 0.5, 1, 1.5, 2, 3, 4, 6; bit 3 is the sign), two
 *           to a byte, the first in the low half; rows of
 *           gemm_fp4_row_bytes(cols) bytes (cols padded to 32 elements).
 *   scales  one byte per block of a row, gemm_fp4_scales_bytes() bytes in all,
 *           in tiles of 128 rows x 4 blocks, 512 bytes each: row r, block c of
 *           a tile at byte (r % 32) * 16 + (r / 32) * 4 + c; the tiles of a row
 *           of tiles follow one another.  (The order in which the tensor cores
 *           take them.)
 *   GEMM_MXFP4  blocks of 32; byte b is the scale 2^(b - 127) (255: NaN);
 *               element = code * scale.
 *   GEMM_NVFP4  blocks of 16; the byte is an E4M3 scale s >= 0 (0x7F: NaN);
 *               element = code * fl32(s * g), g from a device pointer
 *               (NULL: 1), positive and finite.
 * Padding in both arrays is zero; gemm_fp4_quantize writes all of it.  Both
 * arrays are 16-byte aligned.  The two calls below return 0 for sizes or formats
 * that the library does not take.
 */
int64_t gemm_fp4_row_bytes(int64_t cols);
int64_t gemm_fp4_scales_bytes(gemm_fp4_format_t format, int64_t rows, int64_t cols);

/*
 * Quantises src (dtype, [rows][ld], any alignment of its element type) into
 * codes and scales on `stream`.
 *   GEMM_MXFP4  scale 2^E, E = floor(log2 max|x|) - 2 of the block, kept in
 *               [-127, 127] (a block of zeros: -127).
 *   GEMM_NVFP4  s = nearest E4M3 to fl32(max|x| / fl32(6 g)), ties to even, at
 *               most 448.  g = max|tensor| / (6 * 448) uses the format's whole
 *               range.
 *   code        nearest E2M1 value to fl32(x / scale), ties to the even code,
 *               saturating at 6; all zero where the scale is zero.
 * A block that holds an infinity or a NaN gets a NaN scale (its codes mean
 * nothing), so every product that reads it is NaN.
 * src must not overlap codes or scales.  tensor_scale: g for GEMM_NVFP4 (NULL:
 * 1); must be NULL for GEMM_MXFP4.  Allocates nothing.
 * Errors: INVALID_ARG, MISALIGNED, UNSUPPORTED (sizes), NO_DEVICE, CUDA.
 */
int gemm_fp4_quantize(gemm_fp4_format_t format, gemm_dtype_t dtype, int64_t rows, int64_t cols,
                      const void* src, int64_t ld, const float* tensor_scale, void* codes,
                      void* scales, void* stream);

/* The values that codes and scales stand for: FP32 code * scale, rounded to
 * nearest even to dtype, into dst ([rows][ld], any alignment of its element
 * type; elements past cols are left as they were).  Errors: as
 * gemm_fp4_quantize. */
int gemm_fp4_dequantize(gemm_fp4_format_t format, gemm_dtype_t dtype, int64_t rows, int64_t cols,
                        const void* codes, const void* scales, const float* tensor_scale, void* dst,
                        int64_t ld, void* stream);

/*
 * C = cast( act( alpha * A.B^T + bias ) + beta * R ) with A [M][K] and
 * B [N][K] in 4 bits of one format (a weight as it lies for X.W^T), on the
 * block-scaled tensor cores with FP32 accumulation; from one row (a token) up.
 *
 * gemm_fp4_plan validates the problem, chooses the tile and allocates a status
 * word on the current device; no workspace.  epilogue: NULL (plain FP32 C), or
 * as for gemm_plan with b_layout GEMM_B_NK, batch 1 and no row softmax (else
 * UNSUPPORTED); strides a, b, c, r are ignored.
 * gemm_fp4_run enqueues on `stream`: arrays as described above, tensor scales
 * for GEMM_NVFP4 only (NULL: 1); bias, residual and C as for gemm_run; C must
 * not overlap any input.  Runs of one plan may overlap on the GPU.  GELU is
 * max(y, 0) - z Q(z), z = |y|, Q the normal distribution's tail: off by at most
 * (20 + 1.5 z^2) 2^-24 z Q(z) (2.2e-7, near z = 0.8) and the casts' rounding.
 * Errors: as gemm_plan and gemm_run; MISALIGNED where codes or scales are not
 * 16-byte aligned, or another array not to its element type.
 */
typedef struct gemm_fp4_plan_s* gemm_fp4_plan_t;
int gemm_fp4_plan(gemm_fp4_format_t format, int64_t M, int64_t N, int64_t K, int64_t ldc,
                  const gemm_epilogue_t* epilogue, gemm_fp4_plan_t* out_plan);
int gemm_fp4_run(gemm_fp4_plan_t plan, const void* a_codes, const void* a_scales,
                 const float* a_tensor_scale, const void* b_codes, const void* b_scales,
                 const float* b_tensor_scale, void* C, const void* bias, const void* residual,
                 float alpha, void* stream);
/* As gemm_plan_status and gemm_plan_destroy. */
int gemm_fp4_status(gemm_fp4_plan_t plan);
void gemm_fp4_destroy(gemm_fp4_plan_t plan);
/* Host-only: the tile that gemm_fp4_plan would choose on a device with num_sms
 * SMs: rows of A per tile (bn; 128 rows of B), and the CTAs that share a tile's
 * K (split_k).  Errors: INVALID_ARG, UNSUPPORTED (sizes that gemm_fp4_plan refuses). */
int gemm_fp4_select_config(int64_t M, int64_t N, int64_t K, int32_t num_sms, gemm_config_t* out);

/*
 * 8-bit floats (mxfp8).  A matrix [rows][cols] is two device arrays, both
 * 16-byte aligned:
 *   codes   E4M3 values (sign, 4 exponent bits, 3 mantissa bits; up to 448), a
 *           byte each, in rows of gemm_fp8_row_bytes(cols) bytes (cols padded to
 *           32 elements).
 *   scales  as for GEMM_MXFP4: blocks of 32 along a row, byte b the scale
 *           2^(b - 127) (255: NaN), in the same tiles of 128 rows x 4 blocks,
 *           gemm_fp8_scales_bytes() bytes in all.  element = code * scale.
 * Padding in both arrays is zero; gemm_fp8_quantize and gemm_rms_norm write all of it.
 *
 * gemm_fp8_quantize: scale 2^E, E the least with max|x| <= 448 * 2^E over the
 * block, kept in [-127, 127] (a block of zeros: -127); code the nearest E4M3 value
 * to x / scale, ties to the even code.  A block that holds an infinity or a NaN
 * gets a NaN scale (its codes mean nothing).
 * The calls are as the gemm_fp4_ calls of the same names, without the format and
 * the tensor scales; the product's K elements of a stage are 128 instead of 256.
 */
int64_t gemm_fp8_row_bytes(int64_t cols);
int64_t gemm_fp8_scales_bytes(int64_t rows, int64_t cols);
int gemm_fp8_quantize(gemm_dtype_t dtype, int64_t rows, int64_t cols, const void* src, int64_t ld, void* codes,
                      void* scales, void* stream);
int gemm_fp8_dequantize(gemm_dtype_t dtype, int64_t rows, int64_t cols, const void* codes, const void* scales,
                        void* dst, int64_t ld, void* stream);
typedef struct gemm_fp8_plan_s* gemm_fp8_plan_t;
int gemm_fp8_plan(int64_t M, int64_t N, int64_t K, int64_t ldc, const gemm_epilogue_t* epilogue,
                  gemm_fp8_plan_t* out_plan);
int gemm_fp8_run(gemm_fp8_plan_t plan, const void* a_codes, const void* a_scales, const void* b_codes,
                 const void* b_scales, void* C, const void* bias, const void* residual, float alpha, void* stream);
int gemm_fp8_status(gemm_fp8_plan_t plan);
void gemm_fp8_destroy(gemm_fp8_plan_t plan);
int gemm_fp8_select_config(int64_t M, int64_t N, int64_t K, int32_t num_sms, gemm_config_t* out);

/*
 * Root-mean-square norm of rows, with the residual's addition before it:
 *
 *     H = cast(X + R)                 to R's type, round to nearest even (has_residual; else H is X)
 *     Y = cast( H / sqrt(mean_k H^2 + eps) * (weight + weight_offset) )
 *
 * sums and all steps in FP32.  Y is computed from the rounded H, so that a later call on H
 * alone gives the same.  With mxfp8, Y is written as 8-bit floats (above): codes and scales are those of
 * the exact values of the formula, but that the sum of squares is off by some 2^-40 of itself, so a value that close to a border
 * of the codes or the scales may fall on its other side (sum and factor are held in two FP32 numbers each; values next to a
 * border are worked out again with both).
 * A row's sum of squares must stay below 2^128; where it and eps are below 2^-90, or in mxfp8 results below 2^-100,
 * digits are lost.  NaN and infinities: as the formula has them.
 */
typedef struct {
    gemm_dtype_t dtype;          /* X; default GEMM_BF16 */
    int has_residual;            /* 1: R is added */
    gemm_dtype_t residual_dtype; /* R and H: GEMM_F32 or `dtype`; default GEMM_BF16 */
    gemm_dtype_t weight_dtype;   /* default GEMM_BF16 */
    gemm_dtype_t out_dtype;      /* Y, unless mxfp8; default GEMM_BF16 */
    int mxfp8;                   /* 1: Y holds codes, `scales` the scales */
    int64_t rows, cols;          /* cols: 1 to 2^22 */
    int64_t ldx, ldr, ldh, ldy;  /* in elements; 0 means cols (ldy: not used with mxfp8) */
    float eps;                   /* default 1e-6; finite, >= 0 */
    float weight_offset;         /* default 0; finite */
} gemm_norm_desc_t;

/* Fills *d with the defaults listed above (0 elsewhere). */
void gemm_norm_desc_init(gemm_norm_desc_t* d);

/*
 * Enqueues the norm (one kernel) on `stream`.  All pointers are device pointers aligned to
 * their element type (codes and scales to 16 bytes); rows that all start on 16 bytes go
 * fastest.  residual: R, NULL iff !has_residual.  weight: [cols], or NULL for ones.  H: NULL
 * (not wanted), and without a residual always.  scales: NULL iff !mxfp8.  H, and Y unless mxfp8, may be
 * X or R itself (same type and stride; not both the same one); they overlap nothing else.
 * Allocates nothing and needs no workspace; calls may overlap.
 * Errors: INVALID_ARG, MISALIGNED, UNSUPPORTED (sizes), NO_DEVICE, CUDA.
 */
int gemm_rms_norm(const gemm_norm_desc_t* desc, const void* X, const void* residual, const void* weight, void* H,
                  void* Y, void* scales, void* stream);

/*
 * 4-bit weights with group scales.  W [N][K] (rows: output columns, as a weight
 * lies for X.W^T) in integers 0..15:  w = (q - z) * s  with a 16-bit scale s
 * (GEMM_F16 or GEMM_BF16) and an integer zero z in 0..15 for each `group` (a multiple of 32) columns of
 * a row; without an array of zeros z = 8.  Device arrays, 16-byte aligned:
 *   codes   gemm_w4_codes_bytes() bytes in blocks of 16 rows x 64 columns, 512
 *           bytes each, the blocks of 16 rows one after another along K.  Row r,
 *           column k of a block are in its 32-bit word
 *           ((r % 8) * 4 + k % 32 / 8) * 4 + k / 32 * 2 + r / 8  (little endian),
 *           at bits 4 * (k % 2 * 4 + k % 8 / 2).
 *   scales, zeros (a byte each)   gemm_w4_scales_count() entries; row r, group c
 *           at ((r / 16) * groups + c) * 16 + r % 8 * 2 + r % 16 / 8,
 *           groups = ceil(K / group).
 * Padding is zero; the two calls that write them write all of it.  N up to 2^28,
 * K and group up to 65536, codes below 2^31 blocks; the size calls return 0 for others.
 */
int64_t gemm_w4_codes_bytes(int64_t N, int64_t K);
int64_t gemm_w4_scales_count(int64_t N, int64_t K, int64_t group);

/*
 * Quantises src (dtype, [N][ld]) to the nearest codes.  With zeros: lo = min(w, 0)
 * and hi = max(w, 0) of the group, s = (hi - lo) / 15 rounded to scale_dtype,
 * z = -lo / s rounded, in 0..15; zeros NULL: s = max|w| / 7.5.  q = w / s rounded + z, kept in
 * 0..15 (FP32; halves to even).  A group that holds an infinity or a NaN gets a NaN scale.
 * src overlaps no output.  Errors: INVALID_ARG, MISALIGNED, UNSUPPORTED, NO_DEVICE, CUDA.
 */
int gemm_w4_quantize(gemm_dtype_t dtype, gemm_dtype_t scale_dtype, int64_t N, int64_t K, int64_t group,
                     const void* src, int64_t ld, void* codes, void* scales, void* zeros, void* stream);
/* Codes of a checkpoint, a byte each (q [N][ldq], its low four bits), scales (16 bits, [N][lds]) and
 * zeros (a byte each, [N][ldz]; NULL with `zeros` NULL) of its groups, into the arrays above.  Errors: as above. */
int gemm_w4_pack(int64_t N, int64_t K, int64_t group, const void* q, int64_t ldq, const void* s, int64_t lds,
                 const void* z, int64_t ldz, void* codes, void* scales, void* zeros, void* stream);
/* (q - z) * s in FP32, rounded to nearest even to dtype, into dst ([N][ld]).  Errors: as above. */
int gemm_w4_dequantize(gemm_dtype_t dtype, gemm_dtype_t scale_dtype, int64_t N, int64_t K, int64_t group,
                       const void* codes, const void* scales, const void* zeros, void* dst, int64_t ld, void* stream);

/*
 * Y = cast( act( alpha * X.W^T + bias ) + beta * R ) for 1 to 64 tokens.  X [M][K] in the scales'
 * type.  No weight is rounded: a group's sum of (q - z) x is added in FP32 and multiplied by its scale (from 17
 * tokens on that sum has to stay within FP32, up to 16 the result); a result is off by some 2^-19 of sum |x| (q + z) s at most before the
 * epilogue.  Up to 16 tokens (and where rows of X do not start on 16 bytes) BF16 values below 2^-31, FP16 values below
 * 2^-28 of the largest of their 128 columns, k / 128 alike, count to 2^-39 of it.  A token that holds an infinity or a
 * NaN gives sums that are not finite; a NaN before the activation (any of them) is one after it.  More tokens:
 * gemm_w4_dequantize, then gemm_run.
 */
typedef struct {
    gemm_dtype_t dtype;     /* X and the scales: GEMM_BF16 (default) or GEMM_F16 */
    gemm_dtype_t out_dtype; /* default GEMM_BF16 */
    int64_t M;              /* tokens, 0 to 64 */
    int64_t N, K, group;    /* group: default 128 */
    int has_zeros;
    int has_bias;           /* FP32 [N] */
    gemm_act_t act;         /* none, GELU (as in gemm_fp4_run) or ReLU (of a NaN: NaN) */
    int has_residual;       /* FP32 [M][ldr] */
    float beta;             /* default 1 */
    int64_t ldx, ldy, ldr;  /* in elements; 0 means K, N and ldy */
    uint32_t flags;         /* GEMM_FLAG_TEST_STALL, or 0 */
    uint32_t timeout_ms;    /* bound on each wait inside the kernel; 0 means 2000 ms */
} gemm_w4_desc_t;

/* Fills *d with the defaults listed above (0 elsewhere). */
void gemm_w4_desc_init(gemm_w4_desc_t* d);

/* Enqueues the product (one kernel) on `stream`.  Pointers aligned to their element type
 * (codes, scales, zeros: 16 bytes); Y overlaps no input.  Allocates nothing and needs no
 * workspace; calls may overlap.  (Should a wait inside the kernel run out, the tile of 128 rows of W that was
 * worked on gives NaN for all tokens, with any activation.)  Errors: INVALID_ARG, MISALIGNED, UNSUPPORTED, NO_DEVICE, CUDA. */
int gemm_w4_run(const gemm_w4_desc_t* desc, const void* X, const void* codes, const void* scales, const void* zeros,
                void* Y, const void* bias, const void* residual, float alpha, void* stream);

/*
 * Routing to experts: the choice of each token's experts, and their weights, from
 * its logits z [T][E] (any number of tokens):
 *
 *     s = softmax(z) over all E experts, or sigmoid(z)
 *     c = s + bias                     (bias FP32 [E], NULL: none)
 *     groups > top_groups: the experts lie in `groups` equal groups, one after
 *       another; the top_groups groups with the largest score stay, the score
 *       being their largest c, or the sum of their two largest c
 *     the top_k experts of a token are those with the largest c among the groups that stay
 *     weight = s, with normalize divided by the sum of the chosen s; times scale
 *
 * Experts come in falling order of c, groups and experts that are equal by the lowest index.
 * The order is that of c as a real number: without a bias the logits themselves are compared,
 * and where c in FP32 leaves two in doubt it is computed in 64 bits, whose rounding is the limit (scores below
 * e^-700 count as equal).  NaN comes last.  Weights are FP32 throughout, and with normalize relative to the
 * largest of them, so that scores below FP32's range keep their ratios; a token whose logits hold a NaN or +infinity, or
 * none above -infinity, gets NaN weights with softmax (with sigmoid only a chosen NaN does so), and with normalize
 * one whose chosen scores are all exactly 0.
 */
typedef enum { GEMM_ROUTE_SOFTMAX = 0, GEMM_ROUTE_SIGMOID = 1 } gemm_route_scores_t;
typedef enum { GEMM_ROUTE_GROUP_MAX = 0, GEMM_ROUTE_GROUP_TOP2 = 1 } gemm_route_group_t;
typedef struct {
    gemm_dtype_t dtype;             /* logits; default GEMM_F32 */
    int64_t T;                      /* tokens, >= 0 */
    int64_t E;                      /* experts, 1 to 512 */
    int64_t top_k;                  /* 1 to min(E / groups * top_groups, 32) */
    gemm_route_scores_t scores;     /* default GEMM_ROUTE_SOFTMAX */
    int64_t groups, top_groups;     /* default 1, 1; groups divides E, at most 32 */
    gemm_route_group_t group_score; /* default GEMM_ROUTE_GROUP_MAX */
    int normalize;                  /* default 1 */
    float scale;                    /* default 1; finite */
    int64_t ld;                     /* logits' row stride in elements; 0 means E */
} gemm_route_desc_t;

/* Fills *d with the defaults listed above (0 elsewhere). */
void gemm_route_desc_init(gemm_route_desc_t* d);

/* Enqueues the routing (one kernel) on `stream`: expert_ids int32 [T][top_k], expert_weights FP32
 * [T][top_k].  Pointers aligned to their element type; outputs overlap no input.  Allocates nothing; calls may
 * overlap.  Errors: INVALID_ARG, MISALIGNED, UNSUPPORTED, NO_DEVICE, CUDA. */
int gemm_route(const gemm_route_desc_t* desc, const void* logits, const float* bias, int32_t* expert_ids,
               float* expert_weights, void* stream);

/*
 * A mixture-of-experts layer for a few tokens, all of it: router, choice of
 * experts, both products of each chosen expert, and their weighted sum.
 *
 *     z = X.Wr^T                          [T][E], FP32
 *     p = softmax(z) over all E experts
 *     the top_k experts of a token are those with the largest z (equal ones:
 *     the lowest index; NaN comes last); their weights are p, or, with
 *     normalize, p divided by its sum over them
 *     Y[t] = cast( sum_j weight_j * W2[e_j] . h_j ),  h_j = act(W1[e_j] . X[t])
 *
 * in FP32 accumulation; cast rounds to nearest even to `dtype`, that of X, Wr,
 * W1, W2 and Y (GEMM_F16 or GEMM_BF16).  Between the products h is held as two
 * numbers of that type, its rounding and the rest (GEMM_F16: values beyond its
 * range, up to 2^32, in units of 2^16, which takes longer, and further on as
 * infinities; an infinite weight in W2 may give NaN where h alone gives an
 * infinity).  Every weight of a chosen expert is read once.  A token with a
 * logit that is NaN or +infinity, or with none above -infinity, gets a row of
 * NaN, and nothing of it enters another token's row.  (What the tokens choose decides
 * where sums are cut: a row's last bits may depend on the other tokens of its call.)
 */
typedef enum {
    GEMM_MOE_GELU = 0,  /* GELU (erf form) of W1[e] . x, W1[e] [I][H] */
    GEMM_MOE_RELU = 1,  /* max(W1[e] . x, 0); of a NaN: NaN */
    GEMM_MOE_SWIGLU = 2 /* silu(gate) * up, W1[e] [2I][H]: gate rows, then up rows */
} gemm_moe_act_t;

typedef struct {
    gemm_dtype_t dtype;  /* GEMM_BF16 (default) or GEMM_F16 */
    int64_t T;           /* tokens, 0 to 64 */
    int64_t E;           /* experts, 1 to 512 */
    int64_t top_k;       /* experts per token, 1 to min(E, 32) */
    int64_t H;           /* length of a token, 1 to 16384 */
    int64_t I;           /* inner length of an expert, 1 to 2^20 */
    gemm_moe_act_t act;  /* default GEMM_MOE_SWIGLU */
    int normalize;       /* 1 (default): weights of a token sum to one */
    /* strides in elements; 0 means contiguous (H; H; H and rows of W1 times
       ld_w1; I and H * ld_w2; H) */
    int64_t ldx;                /* X [T][ldx] */
    int64_t ld_router;          /* Wr [E][ld_router] */
    int64_t ld_w1, stride_w1;   /* W1 [E][I or 2I][ld_w1], experts stride_w1 apart */
    int64_t ld_w2, stride_w2;   /* W2 [E][H][ld_w2], experts stride_w2 apart */
    int64_t ldy;                /* Y [T][ldy] */
    uint32_t flags;             /* GEMM_FLAG_TEST_STALL, or 0 */
    uint32_t timeout_ms;        /* bound on the device-side wait; 0 means 2000 ms */
} gemm_moe_desc_t;

typedef struct gemm_moe_plan_s* gemm_moe_plan_t;

/* Fills *d with the defaults listed above. */
void gemm_moe_desc_init(gemm_moe_desc_t* d);

/* Validates the layer and allocates a status word on the current device.
 * Errors: INVALID_ARG, UNSUPPORTED (FP32; sizes beyond those above; 2^30 or more
 * pieces of 16 rows x 64 elements in W1 or W2), NO_DEVICE, OUT_OF_MEMORY, CUDA. */
int gemm_moe_plan(const gemm_moe_desc_t* desc, gemm_moe_plan_t* out_plan);

/* Device bytes that each run needs as its workspace; 0 for a bad plan. */
int64_t gemm_moe_workspace_bytes(gemm_moe_plan_t plan);

/*
 * Enqueues the layer (two kernels) on `stream`.  All pointers are device pointers,
 * aligned to their element type; weights whose rows all start on 32 bytes (16) and
 * whose H and I are multiples of 16 (8) load fastest.  (Rows anyhow are read in whole
 * 16-byte pieces of memory, each of which holds at least one of their elements.)  expert_ids (int32 [T][top_k], largest weight first)
 * and expert_weights (FP32 [T][top_k]) may be NULL.  workspace: 256-byte aligned,
 * gemm_moe_workspace_bytes() long, any contents; it belongs to the run until the run
 * has finished on the GPU.  Runs with workspaces of their own may overlap.  No output
 * may overlap an input, the workspace or another output.  Allocates nothing.
 * Errors: BAD_PLAN, INVALID_ARG, MISALIGNED, CUDA.
 */
int gemm_moe_run(gemm_moe_plan_t plan, const void* X, const void* Wr, const void* W1, const void* W2,
                 void* Y, int32_t* expert_ids, float* expert_weights, void* workspace, void* stream);
/*
 * The same layer with a choice made beforehand (gemm_route, say) instead of the router:
 * expert_ids int32 [T][top_k] and expert_weights FP32 [T][top_k], read as they are
 * (normalize does not count).  An id outside 0 .. E - 1 takes no part, an expert that a token names twice
 * counts with the sum of its weights, and a token without experts gets zeros.
 */
int gemm_moe_run_routed(gemm_moe_plan_t plan, const void* X, const int32_t* expert_ids, const float* expert_weights,
                        const void* W1, const void* W2, void* Y, void* workspace, void* stream);
/* As gemm_plan_status and gemm_plan_destroy. */
int gemm_moe_status(gemm_moe_plan_t plan);
void gemm_moe_destroy(gemm_moe_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* GEMM13_H */
