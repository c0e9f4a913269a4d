/*
 * dense_int8_matrix: dense matrix multiply C = A x B on one NVIDIA GB300
 * (sm_103a).  C ABI of libgemm_gb300.so.
 *
 * The operation is the one the TPU's 256x256 INT8 multiply-accumulate array
 * evaluates ("文章导读: Motivation for and Evaluation of the First Tensor
 * Processing Unit", sections "TPU介绍" and "TPU使用的技术"):
 *
 *     C[i][j] = sum_{kk < k} A[i][kk] * B[kk][j]
 *
 * in two forms: int8 x int8 -> int32 (exact) and bf16 x bf16 -> fp32
 * (fp32 accumulation).  The tile configuration of each problem is chosen on
 * the host by the five-step method of patent CN114238853A
 * ("一種矩陣乘分片配置選擇方法及系統", claims 1-7), re-derived for sm_103a.
 *
 * Layout (all operands dense, leading dimensions implied):
 *   A   m x k row-major              A[i][kk] = A[i*k + kk]
 *   Bt  n x k row-major: B stored K-major (transposed), B[kk][j] = Bt[j*k + kk]
 *   C   m x n row-major              C[i][j]  = C[i*n + j]
 *
 * Ownership: the caller owns every buffer.  The library never frees caller
 * memory.  Device scratch (the f16 copies of int8 operands) is taken from a
 * private stream-ordered memory pool inside gemm_*_run and returned to it on
 * the same stream.  A plan is plain data: copy it freely, nothing to free.
 *
 * Asynchrony: gemm_*_run only enqueues work on `stream` (a cudaStream_t;
 * NULL = the legacy default stream) and returns.  Launch errors are returned
 * as GEMM_ERR_CUDA.  Errors found while kernels run (a wait that ran past its
 * time limit) are reported by gemm_device_error().  The library's kernels
 * are launched with programmatic stream serialization, so a call's kernels
 * may start (set up, prefetch into L2) before the work in front of them on
 * the stream has finished; none of them reads or writes A, Bt, C or scratch
 * before that work has completed, so stream order holds as usual.  C must
 * not overlap A or Bt of the same call.
 *
 * Thread safety: every entry point may be called from several host threads.
 */
#ifndef DENSE_INT8_MATRIX_H
#define DENSE_INT8_MATRIX_H

#include <stdint.h>

/* Only the entry points below are exported; the library is built with
 * hidden default visibility. */
#if defined(__GNUC__)
#define GEMM_API __attribute__((visibility("default")))
#else
#define GEMM_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gemm_status {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_ARG = 1,        /* null pointer, size out of range, bad plan */
    GEMM_ERR_MISALIGNED = 2,         /* A or Bt not 16-byte aligned, C not 4-byte aligned */
    GEMM_ERR_UNSUPPORTED_DEVICE = 3, /* current device is not sm_103 */
    GEMM_ERR_CUDA = 4,               /* a CUDA runtime call failed */
    GEMM_ERR_OVERFLOW_RISK = 5,      /* int8: k > 131071, so |C| could exceed int32 */
    GEMM_ERR_TIMEOUT = 6             /* a kernel wait ran past its limit (see gemm_device_error) */
} gemm_status;

enum { GEMM_PATH_TENSOR = 0, GEMM_PATH_SKINNY = 1 };
enum { GEMM_DTYPE_I8 = 0, GEMM_DTYPE_BF16 = 1 };

/* Kernel kinds counted by the trace (gemm_trace_*). */
enum {
    GEMM_KERNEL_STAGE = 0,  /* operand staging: int8 -> f16 widening / re-pitching */
    GEMM_KERNEL_TC = 1,     /* tcgen05 tensor-core GEMM */
    GEMM_KERNEL_SKINNY = 2, /* skinny-m GEMM */
    GEMM_KERNEL_REQUANT = 3, /* elementwise requantisation (gemm_i8_run_requant: K-split tiles, skinny path) */
    GEMM_KERNEL_KINDS = 4
};

/* Output types of gemm_i8_run_requant. */
enum { GEMM_OUT_BF16 = 1, GEMM_OUT_I8 = 2 };

#define GEMM_PLAN_VERSION 2
#define GEMM_I8_MAX_K 131071 /* 131071 * 128 * 128 < 2^31 */

/*
 * The selected configuration (patent CN114238853A claim 7: "input the size,
 * select the configuration and its kernel, run").  Filled by gemm_*_plan.
 *
 * Tail split (an addition to the patent's five steps, int8 only): when the
 * tiles do not fill a whole number of waves, the tiles of the last, partial
 * wave are split along K into split_k slices run by otherwise idle CTAs (CTA
 * pairs for the two-SM tile).  The staging kernel zeroes C over those tiles
 * and every slice adds its exact int32 partial sums into C (TMA reduce-add,
 * or atomics when C cannot take TMA); no slice waits on another.  Integer
 * addition is exact and order-free, so the result is bit-identical to the
 * unsplit one.  gemm_*_run recomputes the split for the tile and grid it
 * actually launches.
 */
typedef struct gemm_plan {
    int32_t version;   /* GEMM_PLAN_VERSION */
    int32_t path;      /* GEMM_PATH_* */
    int32_t dtype;     /* GEMM_DTYPE_* */
    int32_t num_sms;   /* SM count the plan was made for */
    int64_t m, k, n;
    int32_t bm, bn, bk;  /* CTA tile; bk = K elements per pipeline stage */
    int32_t stages;      /* depth of the shared-memory operand ring */
    int32_t tiles;       /* output tiles: Thread_Blocks of claim 4 */
    int32_t bpc;         /* CTAs per SM: block_per_cu of claim 6 */
    int32_t grid;        /* CTAs launched (persistent): min(tiles, num_sms * bpc) */
    int32_t waves;       /* ceil(tiles / (num_sms * bpc)): Launch_kernel_times of claim 6 */
    int32_t k_pitch;     /* row pitch (elements) of the staged 16-bit operands */
    int32_t chunk_k;     /* K elements accumulated in fp32 before an exact int32 drain */
    int32_t fallback;    /* 1 if no tile filled the chip (claim 4 S3) */
    int32_t split_k;     /* K slices of each tile in the last, partial wave (1 = none) */
    double ratio;        /* compute-to-memory ratio of the tile (claim 5), flop per byte */
    int64_t workspace_bytes; /* device scratch gemm_*_run takes from its pool (16-bit operand copies) */
    int32_t split_from;  /* tiles [split_from, tiles) are split into split_k K slices */
    int32_t a_on_chip;   /* 1: the two-SM kernel loads int8 A and widens it on chip (no f16 copy of A);
                            int8, bm == 256 and k % 16 == 0 only (see gemm_i8_plan) */
    int64_t reserved[3];
} gemm_plan;

/*
 * Plan an int8 problem (m x k) x (k x n) for the current CUDA device.
 * Routing: m <= 64, or m <= 128 with k % 16 == 0 -> skinny path (streams Bt
 * once, widening it on chip); otherwise the five
 * steps of CN114238853A claim 1 select a (BM, BN) tile.  When the two-SM tile
 * runs a narrow C (n <= 512) with k % 16 == 0, a_on_chip = 1: A is widened
 * from int8 inside the GEMM instead of through a staged f16 copy, which for
 * such shapes would move more bytes than the multiply.  Host-only apart from
 * one cached query of the device's SM count.
 * Errors: GEMM_ERR_INVALID_ARG (out == NULL, m/k/n outside [1, 2^31-1]),
 * GEMM_ERR_OVERFLOW_RISK (k > GEMM_I8_MAX_K), GEMM_ERR_CUDA (no device).
 */
GEMM_API gemm_status gemm_i8_plan(int64_t m, int64_t k, int64_t n, gemm_plan *out);

/* Plan a bf16 problem for the current device (always the tensor-core path). */
GEMM_API gemm_status gemm_bf16_plan(int64_t m, int64_t k, int64_t n, gemm_plan *out);

/*
 * Pure host planner: the same selection for an explicit SM count, with no
 * CUDA call at all.  dtype is GEMM_DTYPE_*.  Same errors as the above.
 */
GEMM_API gemm_status gemm_plan_for_sms(int32_t dtype, int64_t m, int64_t k, int64_t n, int32_t num_sms,
                              gemm_plan *out);

/*
 * C (int32, m x n) = A (int8, m x k) x B, with B given as Bt (int8, n x k).
 * All pointers are device pointers on the current device.  A and Bt must be
 * 16-byte aligned, C 4-byte aligned.  Exact: every element equals the int64
 * sum, which the plan's k limit keeps inside int32.
 * A plan may be edited before the call to force another compiled tile (bm in
 * {64, 128}, bn in {32, 64, 128, 256}) or another grid size (>= 1); every
 * such choice gives the same result.
 * Errors: GEMM_ERR_INVALID_ARG (null pointer, plan not from gemm_i8_plan or
 * of another version, tile not compiled), GEMM_ERR_MISALIGNED,
 * GEMM_ERR_UNSUPPORTED_DEVICE, GEMM_ERR_CUDA.  Nothing is launched when an
 * error is returned.
 */
GEMM_API gemm_status gemm_i8_run(const gemm_plan *plan, const int8_t *A, const int8_t *Bt, int32_t *C,
                        void *stream);

/*
 * C (fp32, m x n) = A (bf16, m x k) x B, B given as Bt (bf16, n x k); bf16
 * values are passed as their 16-bit patterns.  fp32 accumulation:
 * |C - exact| <= 1e-3 * sum_k |a*b| elementwise.  Same rules and errors as
 * gemm_i8_run.
 */
GEMM_API gemm_status gemm_bf16_run(const gemm_plan *plan, const uint16_t *A, const uint16_t *Bt, float *C,
                          void *stream);

/*
 * Requantising int8 GEMM: D = q( (float(C[i][j]) * row_scale[i]) * col_scale[j] )
 * for the exact int32 product C = A x B of gemm_i8_run, the usual consumer of
 * an int8 GEMM (per-row activation scales, per-column weight scales, a
 * narrower output).  The pages do not define requantisation; its arithmetic is
 * the library's and is stated here: every step is one IEEE-754 binary32
 * operation rounded to nearest, ties to even - (1) int32 -> float, (2) times
 * the row scale, (3) times the column scale - then q:
 *   GEMM_OUT_BF16  bfloat16, round to nearest even (overflow gives infinity,
 *                  NaN stays NaN); D holds m x n 16-bit patterns;
 *   GEMM_OUT_I8    int8: nearest integer, ties to even, then clamped to
 *                  [-128, 127]; NaN gives 0; D holds m x n int8.
 * Where one CTA completes a tile of C, the tile is requantised in the GEMM's
 * epilogue and C never reaches memory (the shared-memory staged write-back of
 * "先导杯比赛回顾", section "Epilogue 写回优化", carried one step further).  The
 * tiles of a K split and the skinny path's C are completed in int32 scratch
 * from the library's pool and converted by a second, elementwise kernel.
 * Same plan and operand rules as gemm_i8_run.  row_scale (m floats) and
 * col_scale (n floats) are device pointers, 16-byte aligned; D is a device
 * pointer (2-byte aligned for bfloat16), row pitch n.
 * Errors: GEMM_ERR_INVALID_ARG (null pointer, bad plan or out_type),
 * GEMM_ERR_MISALIGNED, GEMM_ERR_UNSUPPORTED_DEVICE, GEMM_ERR_CUDA.
 */
GEMM_API gemm_status gemm_i8_run_requant(const gemm_plan *plan, const int8_t *A, const int8_t *Bt,
                                         const float *row_scale, const float *col_scale, int32_t out_type, void *D,
                                         void *stream);

/*
 * gemm_i8_run without any device-memory allocation.  The pages have no
 * counterpart to this entry point.
 *
 * For callers that may not allocate device memory, directly or through a
 * library: runtimes that plan all device memory up front and forbid libraries
 * to take more, and latency-critical loops where an allocation could block,
 * synchronise the device or fail mid-run.  The f16 operand copies that
 * gemm_i8_run takes from a memory pool go instead into one fixed scratch
 * array of GEMM_NOALLOC_SCRATCH_BYTES (64 MiB) in the library's device image,
 * which every GPU that loads the library holds until the process exits.  The
 * call makes no cudaMalloc, cudaFree or other allocating call.
 *
 * Same arguments, rules and result as gemm_i8_run.  Extra rules:
 *   - the tensor-core path needs round256(m*k_pitch*2) + round256(n*k_pitch*2)
 *     bytes of scratch; larger problems return GEMM_ERR_INVALID_ARG and
 *     launch nothing; the skinny path needs m*k*2 bytes (at most 32 MiB) for
 *     the f16 copy of A when k % 16 == 0, and none otherwise;
 *   - the first call on each device, with that device current, looks up the
 *     array's device address (cudaGetSymbolAddress) and caches it; make that
 *     first call before any stream capture;
 *   - every call shares the one array and it keeps the last call's contents
 *     (each call overwrites what it reads and clears its own time-out word),
 *     so calls whose work overlaps on the GPU race and give wrong results:
 *     order them on one stream or with events;
 *   - a kernel wait that runs past its limit ends the call's kernels early
 *     (C incomplete) and records its code in the device error word that all
 *     entry points share (a static device variable, not an allocation):
 *     gemm_device_error reports it as for gemm_i8_run.
 */
#define GEMM_NOALLOC_SCRATCH_BYTES (64ll << 20)
GEMM_API gemm_status gemm_i8_run_noalloc(const gemm_plan *plan, const int8_t *A, const int8_t *Bt, int32_t *C,
                                void *stream);

/*
 * End-to-end forms: A, Bt and C are HOST pointers (pinned or pageable).  The
 * call takes device buffers from the library's pool, copies A and Bt to the
 * device, runs the plan, copies C back and waits for `stream` to finish, so
 * C is ready when it returns.  Large tensor-path problems (at least 2048
 * rows of C, at least 32 MiB of A, Bt and C together) run as a pipeline on
 * four library streams that
 * follow `stream`: A and Bt are cut into bands of at least 1024 rows (at most
 * 8 each), copied up one band at a time and widened once; each band's arrival
 * completes a rectangle of C, which is multiplied and copied down while later
 * bands go up.  Rectangles run the two-SM 256 x 256 tile, so an edited
 * plan's tile applies only to calls that are not pipelined.  Calls on one
 * device take the pipeline one at a time.
 */
GEMM_API gemm_status gemm_i8_run_host(const gemm_plan *plan, const int8_t *A, const int8_t *Bt, int32_t *C,
                             void *stream);
GEMM_API gemm_status gemm_bf16_run_host(const gemm_plan *plan, const uint16_t *A, const uint16_t *Bt, float *C,
                               void *stream);

/* ------------------------------------------------------------------------
 * 8-bit operators around the GEMM: FP8 products with a scale for each block
 * of 128, the same products grouped by expert, the FP8 quantisation that
 * makes their operands, and the RMS norm that writes an 8-bit activation.
 *
 * FP8 values are one byte each (GEMM_F8_E4M3: 4 exponent bits, largest value
 * 448; GEMM_F8_E5M2: 5 exponent bits, largest value 57344), rows contiguous,
 * with a row pitch in elements.  An FP8 operand of the product needs a
 * 16-byte aligned address and a row pitch that is a multiple of 16; k itself
 * may be any size, and the bytes between k and the pitch are never used.
 *
 * A scale is an fp32 factor: the element stands for (8-bit value) * scale.
 *   GEMM_SCALE_ROWS    one scale per row and block of 128 columns, stored
 *                      block-major: scale[b * rows + i], b < ceil(k / 128);
 *   GEMM_SCALE_BLOCKS  one scale per 128 x 128 block, stored
 *                      scale[(j / 128) * ceil(k / 128) + b].
 * Quantising takes scale = max(amax * (1 / M), 2^-126), amax the block's
 * largest magnitude and M the type's largest value, and rounds x * (1 / scale)
 * to the nearest 8-bit value, ties to even; each step, 1 / M among them, is
 * one fp32 operation.  A
 * block of zeros gets the scale 2^-126.  An infinity in a block makes its
 * scale infinite, its own 8-bit value NaN and the block's others zero, so
 * every product that reads the block is NaN; a NaN element is a NaN of the
 * 8-bit type and leaves its block's scale to the others.
 *
 * The entry points below take device pointers, enqueue on `stream` and
 * return, like gemm_*_run; the trace counts quantisation and norms as
 * GEMM_KERNEL_STAGE, products as GEMM_KERNEL_TC or GEMM_KERNEL_SKINNY.
 * ------------------------------------------------------------------------ */
enum { GEMM_F8_E4M3 = 0, GEMM_F8_E5M2 = 1 };
enum { GEMM_SCALE_ROWS = 0, GEMM_SCALE_BLOCKS = 1 };
enum { GEMM_OUT_F32 = 3 };    /* beside GEMM_OUT_BF16: output types of gemm_f8_*run */
enum { GEMM_DTYPE_F32 = 2 };  /* beside GEMM_DTYPE_BF16: input types of gemm_f8_quantize* and gemm_norm_* */

/* How a product is grouped by expert. */
enum {
    GEMM_GROUP_NONE = 0, /* one product */
    GEMM_GROUP_ROWS = 1, /* the rows of A (and of D) belong to groups, each with its own Bt */
    GEMM_GROUP_K = 2     /* the K columns of A and Bt belong to groups, each with its own D */
};

#define GEMM_PLAN_F8_VERSION 1
#define GEMM_F8_MAX_GROUPS 1024
#define GEMM_NORM_MAX_D 32768

/* The configuration of an FP8 product.  Plain data, filled by gemm_f8_*plan*. */
typedef struct gemm_plan_f8 {
    int32_t version;    /* GEMM_PLAN_F8_VERSION */
    int32_t path;       /* GEMM_PATH_TENSOR: two-SM tiles; GEMM_PATH_SKINNY: few rows, Bt streamed */
    int32_t num_sms;    /* SM count the plan was made for */
    int32_t group_mode; /* GEMM_GROUP_* */
    int64_t m, k, n;
    int32_t groups;     /* 1 for GEMM_GROUP_NONE */
    int32_t a_type, b_type; /* GEMM_F8_* */
    int32_t b_scale;    /* GEMM_SCALE_*: layout of b_scale (a_scale is always GEMM_SCALE_ROWS) */
    int32_t bm, bn;     /* rows and columns of D per tile */
    int32_t split_k;    /* skinny path: CTAs that share a tile along K and join their sums */
    int32_t reserved32;
    int64_t reserved[4];
} gemm_plan_f8;

/*
 * Plan D (m x n) = A (m x k) x B with FP8 A and Bt (n x k).  Grouped:
 *   GEMM_GROUP_ROWS  A is m x k, D m x n, and Bt holds `groups` matrices of
 *                    n x k one after the other (group g starts at row g*n);
 *                    rows offsets[g] .. offsets[g+1]-1 of A are multiplied
 *                    with group g's Bt: the forward product of a layer of
 *                    experts, and its input gradient.
 *   GEMM_GROUP_K     A is m x k and Bt n x k as gemm_f8_quantize_cols writes
 *                    them (k = gemm_f8_padded_k(rows, groups)); D holds
 *                    `groups` matrices of m x n, and group g's is the sum
 *                    over that group's columns: the weight gradient.  A
 *                    group without rows gets zeros.
 * Host-only apart from one cached query of the device's SM count;
 * gemm_f8_plan_for_sms makes no CUDA call.
 * Errors: GEMM_ERR_INVALID_ARG (NULL out; m, k or n outside [1, 2^30];
 * groups outside [1, GEMM_F8_MAX_GROUPS], or not 1 without grouping;
 * groups * n (ROWS) or groups * m (K) above 2^30; k no multiple of 128
 * (K); unknown type, scale layout or mode), GEMM_ERR_CUDA (no device).
 */
GEMM_API gemm_status gemm_f8_plan(int64_t m, int64_t k, int64_t n, int32_t a_type, int32_t b_type, int32_t b_scale,
                                  gemm_plan_f8 *out);
GEMM_API gemm_status gemm_f8_grouped_plan(int32_t group_mode, int32_t groups, int64_t m, int64_t k, int64_t n,
                                          int32_t a_type, int32_t b_type, int32_t b_scale, gemm_plan_f8 *out);
GEMM_API gemm_status gemm_f8_plan_for_sms(int32_t group_mode, int32_t groups, int64_t m, int64_t k, int64_t n,
                                          int32_t a_type, int32_t b_type, int32_t b_scale, int32_t num_sms,
                                          gemm_plan_f8 *out);

/*
 * D[i][j] = sum_b (a_scale[b][i] * b_scale[..]) * sum_{kk in block b} A[i][kk] * Bt[j][kk]
 * with fp32 accumulation: each block of 128 is summed, scaled and added to an
 * fp32 running sum, which is rounded once to the output type (GEMM_OUT_BF16
 * or GEMM_OUT_F32).  lda, ldb, ldd: row pitches in elements (lda, ldb >= k
 * and multiples of 16, ldd >= n).  D needs its element's alignment only.
 * A plan may be edited to force the path, bn (skinny: 16, 32, 64 or 128 rows
 * in bm) or split_k (1, 2, 4 or 8) before the call; the sums then join in
 * another order, so results agree to fp32 rounding, not bit for bit.  One
 * plan always gives the same bits.
 * Errors: GEMM_ERR_INVALID_ARG (null pointer, bad plan, a grouped plan, pitch
 * too small, out_type), GEMM_ERR_MISALIGNED (A or Bt not 16-byte aligned, lda
 * or ldb not a multiple of 16, a scale not 4-byte or D not element aligned),
 * GEMM_ERR_UNSUPPORTED_DEVICE, GEMM_ERR_CUDA.
 */
GEMM_API gemm_status gemm_f8_run(const gemm_plan_f8 *plan, const uint8_t *A, int64_t lda, const float *a_scale,
                                 const uint8_t *Bt, int64_t ldb, const float *b_scale, int32_t out_type, void *D,
                                 int64_t ldd, void *stream);

/*
 * The grouped product; plan from gemm_f8_grouped_plan.  offsets: groups + 1
 * int32 on the device, non-decreasing, read by the kernels only (the host
 * never waits for them): rows for GEMM_GROUP_ROWS; for GEMM_GROUP_K the same
 * row offsets that gemm_f8_quantize_cols was given.  Values are clamped to
 * the matrix, so a wrong list gives wrong sums but no access outside the
 * operands.  Rows of D outside every group are not written.  Scales of the
 * groups' Bt lie one after the other (GEMM_SCALE_BLOCKS: groups x ceil(n/128)
 * x ceil(k/128); GEMM_SCALE_ROWS: ceil(k/128) x (groups * n)).
 * Same rules and errors as gemm_f8_run.
 */
GEMM_API gemm_status gemm_f8_grouped_run(const gemm_plan_f8 *plan, const uint8_t *A, int64_t lda,
                                         const float *a_scale, const uint8_t *Bt, int64_t ldb, const float *b_scale,
                                         const int32_t *offsets, int32_t out_type, void *D, int64_t ldd,
                                         void *stream);

/*
 * Quantise X (rows x cols, x_type GEMM_DTYPE_BF16 or GEMM_DTYPE_F32, row
 * pitch ldx) to FP8: Q (rows x cols, row pitch ldq) and its scales, in the
 * layout `scale_mode` (GEMM_SCALE_ROWS or GEMM_SCALE_BLOCKS).
 * Errors: GEMM_ERR_INVALID_ARG (null pointer, size outside [1, 2^30],
 * pitch below cols, unknown type or mode), GEMM_ERR_MISALIGNED (X or scale
 * not element aligned), GEMM_ERR_UNSUPPORTED_DEVICE, GEMM_ERR_CUDA.
 */
GEMM_API gemm_status gemm_f8_quantize(const void *X, int32_t x_type, int64_t rows, int64_t cols, int64_t ldx,
                                      int32_t f8_type, int32_t scale_mode, uint8_t *Q, int64_t ldq, float *scale,
                                      void *stream);

/*
 * The transposed form, for products that sum over rows (weight gradients):
 * Q (cols x kp, row pitch ldq >= kp, kp = gemm_f8_padded_k(rows, groups))
 * holds X^T, one GEMM_SCALE_ROWS scale per column and block of 128 rows:
 * scale[b * cols + j].  offsets == NULL: one group of all rows (groups must
 * be 1).  Otherwise offsets (groups + 1 int32 on the device) gives each
 * group's rows; a group's columns of Q start at a multiple of 128 behind the
 * group before it and are filled up to a multiple of 128 with zeros.
 * Columns behind the last group are not written.  Q must be 16-byte aligned
 * with ldq a multiple of 16.  Same errors as gemm_f8_quantize, and
 * GEMM_ERR_MISALIGNED for Q and ldq.
 */
GEMM_API gemm_status gemm_f8_quantize_cols(const void *X, int32_t x_type, int64_t rows, int64_t cols, int64_t ldx,
                                           int32_t f8_type, const int32_t *offsets, int32_t groups, uint8_t *Q,
                                           int64_t ldq, float *scale, void *stream);

/* Columns that `rows` rows in `groups` groups can take when each group is
 * filled up to a multiple of 128: floor((rows + 127 * groups) / 128) * 128.
 * 0 if rows is outside [1, 2^30] or groups below 1. */
GEMM_API int64_t gemm_f8_padded_k(int64_t rows, int32_t groups);

/*
 * Residual addition, RMS norm and 8-bit quantisation in one pass over rows x
 * d elements (x_type GEMM_DTYPE_BF16 or GEMM_DTYPE_F32):
 *   h    = X + R, rounded to x_type        (R == NULL: h = X)
 *   rstd = 1 / sqrt(mean_j(h_j^2) + eps)   (fp32)
 *   y_j  = h_j * rstd * W[j]
 * gemm_norm_f8 writes y as e4m3 with GEMM_SCALE_ROWS scales, ready as A of
 * gemm_f8_run.  gemm_norm_i8 writes int8 with one scale per row (M = 127),
 * nearest integer, ties to even: ready as A and
 * row_scale of gemm_i8_run_requant.  int8 holds no NaN, so a row with a NaN
 * among its y_j (in h or W, 0 * infinity, or a row of zeros with eps = 0), or
 * whose mean square is infinite, has a NaN scale.  H (may be NULL if R is NULL) gets h and may be X or R itself (with
 * that one's pitch); rstd (rows floats, may be NULL) is kept for the
 * backward pass.  W: d floats.  Pitches ldx, ldr, ldh, ldq in elements.
 * d <= GEMM_NORM_MAX_D; eps >= 0.
 * Errors: as gemm_f8_quantize.
 */
GEMM_API gemm_status gemm_norm_f8(const void *X, int64_t ldx, const void *R, int64_t ldr, const float *W, float eps,
                                  int32_t x_type, int64_t rows, int64_t d, void *H, int64_t ldh, float *rstd,
                                  uint8_t *Q, int64_t ldq, float *scale, void *stream);
GEMM_API gemm_status gemm_norm_i8(const void *X, int64_t ldx, const void *R, int64_t ldr, const float *W, float eps,
                                  int32_t x_type, int64_t rows, int64_t d, void *H, int64_t ldh, float *rstd,
                                  int8_t *Q, int64_t ldq, float *row_scale, void *stream);

/*
 * The gradient of y = h * rstd * W (the quantisation passes gradients
 * through unchanged), from dY, h and rstd as the forward call wrote them:
 *   xhat = h * rstd,  g = dY * W
 *   dX = dR + rstd * (g - xhat * mean_j(g * xhat))   (dR may be NULL: 0)
 *   dW_j = sum_i dY_ij * xhat_ij                      (fp32, overwritten)
 * dR is the gradient that reaches h as the residual; dX (x_type, pitch lddx)
 * is the gradient of X and of R, and may be dR itself (with its pitch).  dW
 * may be NULL.  Sums are taken in a fixed order: the same call gives the same
 * bits.  Errors: as gemm_norm_f8.
 */
GEMM_API gemm_status gemm_norm_backward(const void *dY, int64_t lddy, const void *H, int64_t ldh, const float *W,
                                        const float *rstd, const void *dR, int64_t lddr, int32_t x_type, int64_t rows,
                                        int64_t d, void *dX, int64_t lddx, float *dW, void *stream);

/* ------------------------------------------------------------------------
 * Operators of a bfloat16 layer around the GEMM: the product with bias,
 * activation and residual in its epilogue and the products of its backward
 * pass, the activation's gradient with the bias's, the layer norm and its
 * gradient, and the balance loss of a router, whose offsets the grouped
 * products take.
 *
 * They take device pointers, enqueue on `stream` and return, like
 * gemm_*_run; scratch comes from the library's pool.  The trace counts
 * products as GEMM_KERNEL_TC or GEMM_KERNEL_SKINNY, everything else (copies
 * of unaligned operands among it) as GEMM_KERNEL_STAGE.
 * ------------------------------------------------------------------------ */

/* How the operands of a product lie in memory.  Rows are contiguous. */
enum {
    GEMM_FORM_NT = 0, /* A m x k, B stored n x k (the weights of a forward product) */
    GEMM_FORM_NN = 1, /* A m x k, B stored k x n (input gradient: A = dZ, B the same weights) */
    GEMM_FORM_TN = 2  /* A stored k x m, B stored k x n (weight gradient: A = dZ, B = X, k the rows) */
};

/* Activations, v in fp32, s(v) = 1 / (1 + exp(-v)), Phi the normal distribution:
 *   RELU v > 0 ? v : 0;  GELU v * Phi(v);  SILU v * s(v);
 *   GELU_TANH v * s(2 sqrt(2 / pi) (v + 0.044715 v^3)), GELU with the tanh form of Phi.
 * NaN stays NaN.  GELU, GELU_TANH and SILU of -infinity are NaN (0 times it),
 * and so may be their derivatives at an infinity. */
enum {
    GEMM_ACT_NONE = 0,
    GEMM_ACT_RELU = 1,
    GEMM_ACT_GELU = 2,
    GEMM_ACT_GELU_TANH = 3,
    GEMM_ACT_SILU = 4,
    GEMM_ACT_GRADIENT = 16 /* added to one of them: multiply by its derivative at Z */
};

#define GEMM_PLAN_LINEAR_VERSION 1
#define GEMM_BALANCE_MAX_EXPERTS 1024

/* The configuration of a bfloat16 product.  Plain data, filled by gemm_bf16_linear_plan*. */
typedef struct gemm_plan_linear {
    int32_t version;  /* GEMM_PLAN_LINEAR_VERSION */
    int32_t path;     /* GEMM_PATH_TENSOR: two-SM tiles; GEMM_PATH_SKINNY: small tiles, split along K */
    int32_t num_sms;  /* SM count the plan was made for */
    int32_t form;     /* GEMM_FORM_* */
    int64_t m, k, n;
    int32_t bm, bn;   /* rows and columns of D per tile */
    int32_t split_k;  /* skinny path: CTAs that share a tile along K and join their sums */
    int32_t reserved32;
    int64_t reserved[4];
} gemm_plan_linear;

/*
 * Plan D (m x n) = A (m x k) x B (k x n).  Host-only apart from one cached
 * query of the device's SM count; the _for_sms form makes no CUDA call.
 * Errors: GEMM_ERR_INVALID_ARG (NULL out; m, k or n outside [1, 2^30];
 * unknown form; num_sms < 1), GEMM_ERR_CUDA (no device).
 */
GEMM_API gemm_status gemm_bf16_linear_plan(int32_t form, int64_t m, int64_t k, int64_t n, gemm_plan_linear *out);
GEMM_API gemm_status gemm_bf16_linear_plan_for_sms(int32_t form, int64_t m, int64_t k, int64_t n, int32_t num_sms,
                                                   gemm_plan_linear *out);

/*
 *   v[i][j] = sum_kk A[i][kk] * B[kk][j] + bias[j]      (fp32 accumulation)
 *   D[i][j] = act(v) + residual[i][j]                   activation = GEMM_ACT_*
 *   D[i][j] = v * act'(Z[i][j]) + residual[i][j]        activation = GEMM_ACT_* | GEMM_ACT_GRADIENT
 * rounded once to out_type (GEMM_OUT_BF16 or GEMM_OUT_F32).  bias (n floats)
 * and residual (out_type, pitch ldr) may be NULL; residual may be D itself
 * (with its pitch): D += the product.  Z (bfloat16, pitch ldz): without
 * GEMM_ACT_GRADIENT, if not NULL, it gets v rounded to bfloat16, for the
 * backward pass (act itself is taken of the fp32 v); with it Z is read, and
 * may be NULL only for GEMM_ACT_NONE.  With RELU's gradient v is selected,
 * not multiplied: 0 where Z <= 0, NaN where Z is NaN.
 * A, B: bfloat16 with row pitches lda, ldb in elements, in the plan's form.
 * Operands whose address is not 16-byte aligned or whose pitch is not a
 * multiple of 8 are first copied into scratch with such a pitch.  D, residual
 * and Z need their element's alignment only; no output may overlap an operand
 * or another output.
 * A plan may be edited to force the path, the tile (GEMM_PATH_TENSOR: bm 256,
 * bn 128 or 256, split_k 1; GEMM_PATH_SKINNY: bm 16, 32, 64 or 128 rows, for
 * GEMM_FORM_TN 64 or 128, bn 128) or split_k (1, 2, 4 or 8); sums then join
 * in another order.  One plan always gives the same bits.
 * Errors: GEMM_ERR_INVALID_ARG (null pointer, bad plan, pitch too small or
 * above 2^31, unknown type or activation, residual == D with another pitch,
 * an output that is an operand or the other output),
 * GEMM_ERR_MISALIGNED (A, B, D, residual, Z or bias not element aligned),
 * GEMM_ERR_UNSUPPORTED_DEVICE, GEMM_ERR_CUDA.
 */
GEMM_API gemm_status gemm_bf16_linear_run(const gemm_plan_linear *plan, const uint16_t *A, int64_t lda,
                                          const uint16_t *B, int64_t ldb, const float *bias, int32_t activation,
                                          uint16_t *Z, int64_t ldz, const void *residual, int64_t ldr,
                                          int32_t out_type, void *D, int64_t ldd, void *stream);

/*
 * The gradient of an activation and of the bias before it, rows x cols:
 *   dZ = dY * act'(Z), rounded to bfloat16;  dbias[j] = sum_i dY[i][j] * act'(Z[i][j]) (fp32, before that rounding)
 * dY, Z, dZ: bfloat16 with pitches in elements.  Z may be NULL for
 * GEMM_ACT_NONE.  dZ or dbias may be NULL, not both; dZ may be dY or Z itself
 * (with its pitch).  Sums are taken in a fixed order.
 * Errors: GEMM_ERR_INVALID_ARG (null pointer, size outside [1, 2^30], pitch,
 * unknown activation, dZ in place with another pitch, dbias that is dY, Z or
 * dZ), GEMM_ERR_MISALIGNED (not element aligned), GEMM_ERR_UNSUPPORTED_DEVICE, GEMM_ERR_CUDA.
 */
GEMM_API gemm_status gemm_activation_backward(const uint16_t *dY, int64_t lddy, const uint16_t *Z, int64_t ldz,
                                              int32_t activation, int64_t rows, int64_t cols, uint16_t *dZ,
                                              int64_t lddz, float *dbias, void *stream);

/*
 * Residual addition and layer norm in one pass over rows x d elements
 * (x_type, y_type: GEMM_DTYPE_BF16 or GEMM_DTYPE_F32):
 *   h    = X + R, rounded to x_type        (R == NULL: h = X)
 *   mean = mean_j(h_j),  rstd = 1 / sqrt(mean_j((h_j - mean)^2) + eps)   (fp32)
 *   Y_j  = (h_j - mean) * rstd * W[j] + bias[j], rounded to y_type
 * W: d floats; bias: d floats or NULL.  H (x_type; may be NULL if R is NULL)
 * gets h and may be X or R itself (with that one's pitch).  mean and rstd
 * (rows floats each, may be NULL) are kept for the backward pass.  Pitches in
 * elements; d <= GEMM_NORM_MAX_D; eps >= 0.  The mean is corrected by the mean
 * of h - mean, so that its error goes by the row's spread, not by its size, and
 * a constant row gives Y = bias exactly (NaN with eps = 0; magnitudes to 1e22).
 * A row that holds an infinity or a NaN gives NaN, and so does one whose sum
 * leaves fp32's range; one whose squares do has rstd = 0.
 * Errors: as gemm_norm_f8; GEMM_ERR_INVALID_ARG also for any other output that
 * is an operand or another output.
 */
GEMM_API gemm_status gemm_layer_norm(const void *X, int64_t ldx, const void *R, int64_t ldr, const float *W,
                                     const float *bias, float eps, int32_t x_type, int32_t y_type, int64_t rows,
                                     int64_t d, void *H, int64_t ldh, float *mean, float *rstd, void *Y, int64_t ldy,
                                     void *stream);

/*
 * Its gradient, from dY (y_type), h (x_type), mean and rstd as the forward
 * call wrote them:
 *   xhat = (h - mean) * rstd,  g = dY * W
 *   dX = dR + rstd * (g - mean_j(g) - xhat * mean_j(g * xhat))    (dR may be NULL: 0)
 *   dW_j = sum_i dY_ij * xhat_ij,  dbias_j = sum_i dY_ij          (fp32, overwritten)
 * dR (x_type) is the gradient that reaches h as the residual; dX (x_type) is
 * the gradient of X and of R, and may be dR itself, or dY if the types are
 * the same (with that one's pitch).  dW and dbias may be NULL.  Sums are
 * taken in a fixed order: the same call gives the same bits.
 * Errors: as gemm_norm_f8; GEMM_ERR_INVALID_ARG also for any other output that
 * is an operand or another output.
 */
GEMM_API gemm_status gemm_layer_norm_backward(const void *dY, int64_t lddy, const void *H, int64_t ldh, const float *W,
                                              const float *mean, const float *rstd, const void *dR, int64_t lddr,
                                              int32_t x_type, int32_t y_type, int64_t rows, int64_t d, void *dX,
                                              int64_t lddx, float *dW, float *dbias, void *stream);

/*
 * Balance loss of a router and the experts' counts.  X: logits, rows x
 * experts (GEMM_DTYPE_BF16 or GEMM_DTYPE_F32, pitch ldx); index: the experts
 * chosen for each row, rows x top_k int32 without gaps.  An index outside
 * [0, experts) is a slot that is not taken (a token that a full expert has
 * turned away); a row without a taken slot is padding and takes no part.  So a
 * token that every expert it chose has turned away leaves the loss and the
 * gradient: where such tokens are to count, pass the router's choices as they
 * were before any was turned away, and take the offsets of the rows that stay
 * from a call with those that remain.
 *   counts[e]  = number of slots with index e
 *   offsets[e] = counts[0] + .. + counts[e-1], experts + 1 values: the row
 *                offsets that gemm_f8_grouped_run takes (may be NULL)
 *   used       = number of rows that take part, T
 *   lse[i]     = log(sum_e exp(X[i][e])); +infinity for padding
 *   probs[e]   = (1 / T) sum over the used rows of p[i][e], p = softmax of the row
 *   loss       = coef * experts * sum_e (counts[e] / sum counts) * probs[e]
 * counts, used: int32; lse (rows), probs (experts), loss (1): fp32.  Without
 * a used row, probs and loss are 0.  Logits of -infinity have p = 0; a used
 * row of nothing else has p = 0 throughout and lse = -infinity.  A NaN or
 * +infinity in a used row makes its lse and the loss NaN.
 * Sums are taken in a fixed order.
 * Errors: GEMM_ERR_INVALID_ARG (null pointer; rows outside [1, 2^30];
 * experts outside [1, GEMM_BALANCE_MAX_EXPERTS]; top_k below 1; rows * top_k
 * above 2^31 - 1; pitch; unknown type; an output that is an operand or another
 * output), GEMM_ERR_MISALIGNED (not element aligned), GEMM_ERR_UNSUPPORTED_DEVICE, GEMM_ERR_CUDA.
 */
GEMM_API gemm_status gemm_balance(const void *X, int64_t ldx, int32_t x_type, int64_t rows, int32_t experts,
                                  const int32_t *index, int32_t top_k, float coef, int32_t *counts, int32_t *offsets,
                                  int32_t *used, float *lse, float *probs, float *loss, void *stream);

/*
 * Its gradient: with f_e = counts[e] / sum counts (a constant) and p as above
 *   dX[i][e] = dR[i][e] + dloss * coef * experts / T * p[i][e] * (f_e - sum_j f_j p[i][j])
 * lse (which rows are padding; p is formed anew), counts and used as
 * gemm_balance wrote them; dloss: one float on the device.  dR (x_type, may
 * be NULL: 0) is the gradient that reaches the logits by other ways; dX
 * (x_type) may be dR itself (with its pitch).  Rows that are padding, or whose
 * lse is -infinity, get dR (or 0), whatever their logits are.
 * Errors: as gemm_balance; dR is the only operand that dX may be.
 */
GEMM_API gemm_status gemm_balance_backward(const void *X, int64_t ldx, int32_t x_type, int64_t rows, int32_t experts,
                                           const float *lse, const int32_t *counts, const int32_t *used, float coef,
                                           const float *dloss, const void *dR, int64_t lddr, void *dX, int64_t lddx,
                                           void *stream);

/*
 * Waits for `stream`, then reads and clears the current device's error word,
 * which the kernels of every run entry point (gemm_i8_run_noalloc included)
 * write when a wait gives up; the first code since the last read is kept.
 * Returns GEMM_OK, GEMM_ERR_TIMEOUT (a kernel wait ran past its 2 s limit
 * and the kernel returned early; *code gets the stage that gave up) or
 * GEMM_ERR_CUDA.  `code` may be NULL.
 */
GEMM_API gemm_status gemm_device_error(void *stream, int32_t *code);

/*
 * The library's private stream-ordered memory pool on the current device
 * (the scratch of gemm_*_run and the device buffers of gemm_*_run_host):
 * bytes it holds now (*reserved_bytes) and the most bytes in use at once
 * since the pool was created or the mark was last reset (*used_high_bytes).
 * reset_high != 0 restarts that mark from the current use after reading it.
 * For callers that budget device memory; the pool keeps freed memory for the
 * next call and returns it only when the process exits.
 * Errors: GEMM_ERR_INVALID_ARG (NULL output), GEMM_ERR_UNSUPPORTED_DEVICE,
 * GEMM_ERR_CUDA.
 */
GEMM_API gemm_status gemm_pool_usage(int64_t *reserved_bytes, int64_t *used_high_bytes, int32_t reset_high);

/*
 * Tracing.  While enabled, every kernel launch made by gemm_*_run is counted
 * per GEMM_KERNEL_* kind, and every `every`-th gemm_*_run call (the first,
 * the (every+1)-th, ...) records a pair of CUDA events on its stream around
 * each timed unit (at most `capacity` units are recorded): the staging
 * launch and the GEMM launch of the tensor path separately (kinds STAGE and
 * TC); on the skinny tensor-core path the prologue launch (A to f16, C
 * zeroed) and the skinny launch together, as kind SKINNY, because the skinny
 * kernel starts while the prologue runs (programmatic dependent launch).
 * Calls that are not sampled record no events, so sampling keeps the timing
 * from slowing the work it measures.  Back-to-back skinny calls on one
 * stream overlap (each call's kernels start before the previous call's
 * end); an event recorded between two calls, as a sampled call records,
 * makes them run one after the other.  gemm_trace_collect waits for the events and writes,
 * per kind (arrays of GEMM_KERNEL_KINDS entries): the summed device time in
 * ms of the timed units, the number of timed units, and the number of
 * launches counted; it then disables tracing.  every >= 1.
 */
GEMM_API gemm_status gemm_trace_begin(int32_t capacity, int32_t every);
GEMM_API gemm_status gemm_trace_collect(float *ms_per_kind, int32_t *timed_per_kind, int32_t *launches_per_kind);

/* Registers per thread and CTAs per SM of the compiled tensor-core kernel for
 * a tile (-1 / 0 if no such kernel); needs a device. */
GEMM_API gemm_status gemm_tc_kernel_info(int32_t bm, int32_t bn, int32_t dtype, int32_t *regs, int32_t *ctas_per_sm);

/*
 * Failure-detection self-test.  Launches one CTA that waits on a barrier
 * nothing completes, with a limit of `timeout_us` microseconds (1 .. 2e6)
 * instead of the kernels' 2 s.  The wait gives up, records code 5 in the
 * device error word and the kernel returns: a following gemm_device_error()
 * returns GEMM_ERR_TIMEOUT with *code = 5, and the CUDA context stays usable.
 * Nothing faults, traps or hangs.
 */
GEMM_API gemm_status gemm_selftest_wait_timeout(int32_t timeout_us, void *stream);

/* Human-readable name of a status. */
GEMM_API const char *gemm_status_string(gemm_status s);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_INT8_MATRIX_H */
