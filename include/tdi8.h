/*
 * tdi8.h -- C ABI of the MI355X (gfx950) tiled int8 matrix-multiply library.
 *
 * Operation.  C = A x B with signed int8 A (M x K) and B (K x N) and int32 C
 * (M x N): C[i][j] = sum_k A[i][k] * B[k][j], accumulated in int32.  This is
 * the product the TPU notes describe being fed, in passes, through a 256 x 256
 * INT8 multiply-accumulate array ("Motivation for and Evaluation of the First
 * Tensor Processing Unit" notes, sections "TPU介绍" and "TPU使用的技术"), and
 * the matrix multiply whose tiling the CUDA tutorial analyses ("CUDA编程实践",
 * section 3).  The kernel that runs is chosen per problem size from a table
 * of compiled tile configurations, as the system of patent application
 * CN114238853A does (claim 7: one kernel compiled per configuration, the
 * configuration parameters being the kernel's template parameters, the best
 * one selected at run time from the input size).
 *
 * Results are exact: every partial sum is an int32 and integer addition is
 * associative, so the bytes of C do not depend on the tiling, the K split or
 * the order of accumulation.  C is defined modulo 2^32 (two's-complement
 * wrap); no wrap occurs while K <= 131071.
 *
 * Memory.  A, B and C are device pointers (hipMalloc'd, or a torch tensor's
 * data_ptr()) owned by the caller.  The library allocates nothing and keeps no
 * pointer after a call returns.  A and B are read only.  Only the window
 * C[0:M, 0:N] is written; bytes of C's rows beyond column N (row padding up to
 * ldc) are never touched.
 *
 * Layouts (all leading dimensions in elements):
 *   A  row-major:        A(i,k) at A[i*lda + k],  lda >= K
 *   B  row-major:        B(k,j) at B[k*ldb + j],  ldb >= N   (gemm_s8s8s32)
 *   B  column-major:     B(k,j) at B[j*ldb + k],  ldb >= K   (gemm_s8s8s32_bt)
 *   C  row-major:        C(i,j) at C[i*ldc + j],  ldc >= N
 * Any pointer alignment and any leading dimension are accepted; 16-byte
 * aligned operands (lda, ldb multiples of 16, ldc of 4) with K a multiple of
 * 16 (and, for row-major B, N a multiple of 16) take the unpredicated fast
 * kernels, whatever the other sizes: rows, columns and K positions past the
 * operands read a 16-byte zero block and stores past M or N are masked.  The
 * rest take the predicated tail kernels.
 *
 * Streams and errors.  Calls are asynchronous: work is enqueued on `stream`
 * (0 = the null stream) and the call returns without waiting.  All argument
 * checks run on the host before anything is enqueued; a call that returns an
 * error has enqueued nothing.  A failed kernel launch returns TDI8_ERR_HIP
 * and tdi8_last_hip_error() gives the hipError_t.  Faults inside a kernel
 * surface at the caller's next synchronisation.  Nothing is printed.
 *
 * Threads.  Initialisation (device query, per-kernel occupancy) happens once
 * per device on first use and is thread safe; afterwards every entry point is
 * re-entrant.  Calls on one stream execute in order.
 */
#ifndef TDI8_H
#define TDI8_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same opaque handle type as HIP's own declaration. */
typedef struct ihipStream_t *hipStream_t;

typedef enum {
    TDI8_OK = 0,
    TDI8_ERR_INVALID_VALUE = -1,     /* M, N or K < 0, or a leading dimension too small */
    TDI8_ERR_NULL_POINTER = -2,      /* a pointer the call must dereference is NULL */
    TDI8_ERR_ALIASING = -3,          /* C's window overlaps the bytes of A or B that are read */
    TDI8_ERR_UNSUPPORTED_DEVICE = -4,/* the current device is not gfx950 */
    TDI8_ERR_BAD_CONFIG = -5,        /* unknown configuration id, or it cannot run this shape */
    TDI8_ERR_HIP = -6                /* a HIP runtime call failed; see tdi8_last_hip_error() */
} tdi8_status;

/* Route by which a configuration is reached in the selection. */
typedef enum {
    TDI8_ROUTE_GENERAL = 0,   /* survived the fill-the-compute-units step */
    TDI8_ROUTE_FALLBACK = 1,  /* reuse-1 fallback of the fill step */
    TDI8_ROUTE_SKINNY = 2     /* fallback with M small enough for the skinny family */
} tdi8_route;

/* C = A x B, A row-major M x K, B row-major K x N, C row-major M x N.
 * M == 0 or N == 0: nothing is enqueued.  K == 0: the C window is set to 0.
 * The configuration is select_tile_config's, with one exception: when the
 * operands take the predicated kernels (see above) with column-major B and
 * the selected tiles number fewer than the compute units, the reuse-1
 * configuration with the most tiles, at most one per compute unit, runs
 * instead (the selection relies on the K split to fill the compute units,
 * which the predicated kernels do not have; gemm_plan reports the one that
 * runs).  Returns TDI8_OK or a negative tdi8_status. */
int gemm_s8s8s32(int M, int N, int K, const int8_t *A, int lda, const int8_t *B, int ldb,
                 int32_t *C, int ldc, hipStream_t stream);

/* Same as gemm_s8s8s32 with B column-major: B(k,j) at B[j*ldb + k], ldb >= K
 * (B stored N x K with K contiguous, as inference weights usually are).  This
 * is the operand order of a convolution lowered to a matrix product in the
 * contest write-up ("先导杯比赛回顾", 卷积转化 and 多批次展开的 Im2col 方法):
 * the filter bank, one row of reduction values per output channel, is the
 * right-hand operand with the reduction dimension contiguous, the layout
 * that write-up transposes its NCHW data into (NCHW布局空间连续性不佳,
 * NCHW_2_NHWC) so that the dimension summed over lies contiguously. */
int gemm_s8s8s32_bt(int M, int N, int K, const int8_t *A, int lda, const int8_t *B, int ldb,
                    int32_t *C, int ldc, hipStream_t stream);

/* Same product computed with a given configuration id instead of the
 * selected one (b_col_major selects the B layout).  Patent application
 * CN114238853A, claim 7: the system compiles one kernel per tiling
 * configuration, the configuration's parameters being the kernel's template
 * parameters, and runs the one the selection picks; this entry point runs a
 * compiled configuration by its id, bypassing the selection.  Any general
 * configuration runs any shape; a skinny configuration needs M <= its block
 * height times 65535 (TDI8_ERR_BAD_CONFIG otherwise).  Arguments, layouts,
 * ownership and errors as for gemm_s8s8s32; config_id outside
 * 0 .. tile_config_count()-1 gives TDI8_ERR_BAD_CONFIG.  For tests and the
 * bench, which sweep every compiled configuration. */
int gemm_s8s8s32_with_config(int config_id, int b_col_major, int M, int N, int K,
                             const int8_t *A, int lda, const int8_t *B, int ldb,
                             int32_t *C, int ldc, hipStream_t stream);

/* Configuration id that gemm_s8s8s32 / gemm_s8s8s32_bt use for an M x K by
 * K x N product on the current device (>= 0), or a negative tdi8_status.
 * The five steps of patent application CN114238853A claim 1 (claims 2-6 give
 * the details): enumerate the compiled configurations; keep those whose
 * register-limited active threads per compute unit reach the threshold;
 * keep those launching at least (compute units x resident blocks per compute
 * unit) blocks, or, if none does, every configuration reduced to reuse 1
 * (then, for M <= 32 or else N <= 32, the skinny family: the smallest block
 * height >= M, or width >= N, then the smallest extent along the other side
 * among those launching a block per compute unit); keep the largest compute-to-memory
 * ratio BM*BN/(BM+BN); keep the fewest rounds of resident blocks; first in
 * table order.  Host only; pure after the first call's initialisation. */
int select_tile_config(int M, int N, int K);

/* Description of one compiled configuration: the tiling tuple the claims of
 * patent application CN114238853A select over (claim 2: the thread split
 * block_m_threads = waves_m * mfma_m and block_n_threads = waves_n * mfma_n;
 * claims 4 and 5: the per-wave repeats m_tiles and n_tiles, the block tile
 * block_m x block_n and the K depth block_k; claim 6: the registers each
 * thread uses, the shared memory (LDS) each block uses and the resulting
 * resident blocks per compute unit, block_per_cu).  Register and LDS figures
 * are those of the configuration's column-major-B unpredicated kernel, read
 * by the build from the compiled code object's metadata. */
typedef struct {
    int id;
    int family;          /* 0 general tiled kernel, 1 skinny (split-K across waves) kernel */
    int mfma_m, mfma_n, mfma_k;  /* matrix-core instruction shape */
    int waves_m, waves_n, waves_k;
    int m_tiles, n_tiles;        /* per-wave instruction repeats (the claims' data reuse) */
    int block_m, block_n, block_k;
    int stages;          /* LDS stages of the unpredicated column-major-B kernel */
    int threads;
    int lds_bytes;       /* static LDS per block of that kernel */
    int vgprs;           /* architectural vector registers per lane of that kernel (rounded up
                            to a multiple of 4 when accumulation registers follow them) */
    int agprs;           /* accumulation vector registers per lane of that kernel (the
                            compiler keeps matrix-core accumulators in either file); the
                            lane's allocation spans vgprs + agprs registers */
    int blocks_per_cu;   /* resident blocks per compute unit, from the runtime occupancy query
                            on the current device (0 before a gfx950 device is seen) */
    int reuse1_id;       /* configuration with the same thread split and m_tiles = n_tiles = 1 */
    int excluded;        /* 1: its reuse scheme (family, m_tiles, n_tiles) was excluded by the
                            performance test of claim 3 (second alternative); the selection drops
                            it at step 2, gemm_s8s8s32_with_config still runs it */
    int sgprs;           /* scalar registers per wave of that kernel */
} tdi8_tile_config;

/* Number of compiled configurations; ids are 0 .. count-1. */
int tile_config_count(void);

/* Copies the description of configuration `id` into *out (caller-owned).
 * Everything but blocks_per_cu is static and needs no device; blocks_per_cu
 * is filled once a gfx950 device has been initialised (0 otherwise).
 * Returns TDI8_OK, TDI8_ERR_BAD_CONFIG (unknown id) or TDI8_ERR_NULL_POINTER. */
int tile_config_info(int id, tdi8_tile_config *out);

/* Hardware description used by the selection. */
typedef struct {
    int num_cu;                /* compute units */
    int max_threads_per_block;
    int min_active_threads;    /* claim-3 threshold on register-limited active threads per CU */
    int skinny_max_m;          /* largest M (or, for larger M, N) routed to the skinny family; 0: none */
} tdi8_hw_info;

typedef struct {
    int id;
    int route;                 /* tdi8_route */
    int survivors[5];          /* candidates left after steps 1..5 */
} tdi8_selection;

/* The selection of select_tile_config on explicit hardware: `blocks_per_cu`
 * holds one entry per configuration id (tile_config_count() entries).  Host
 * only, needs no device; used to test the selection on described hardware.
 * Returns the id (>= 0) or a negative tdi8_status; fills *out when non-NULL. */
int select_tile_config_for(int M, int N, int K, const tdi8_hw_info *hw,
                           const int *blocks_per_cu, tdi8_selection *out);

/* K slices the gemm entry points use with configuration `config_id` for an
 * M x K by K x N product on a device of `num_cu` compute units, when the
 * operands take the unpredicated path (16-byte aligned pointers, lda and ldb
 * multiples of 16, ldc of 4, K a multiple of 16, and with row-major B N
 * too); other operands are never split.  Splitting K with integer atomics is
 * the contest write-up's "Split K" paragraph, added after the five steps of
 * the selection: counting the partial tiles at the ends of M and N, while
 * the tiles times twice the slices still fit one block per compute unit, and
 * K over twice the slices is still at least eight K tiles, the slices double.
 * Slices are whole 16-byte chunks of K, differing by at most one; when M, N
 * and every slice are whole tiles the whole-tile form runs, else the edge
 * form.  1 = no split (always for the skinny family).
 * A split call enqueues two kernels on the stream: one zeroes the C window,
 * the other adds every slice's partial sums into it; the result is the same
 * bytes as without the split (integer addition in any order).  Host only,
 * needs no device.  Returns >= 1 or a negative tdi8_status.
 *
 * A skinny configuration with row-major B (gemm_s8s8s32), 16-byte aligned
 * operands, N and K multiples of 16 and N a multiple of 128 or above 256,
 * also enqueues two kernels: each block
 * covers 128 columns (the last ones may end at N) over one of G = 128 /
 * block width slices of K (whole 128-byte lines of every B row it reads),
 * adding into the zeroed C window.  Its K split is
 * a property of the row-major form and is not what this function reports. */
int tile_config_split_k(int config_id, int M, int N, int K, int num_cu);

/* Kernel forms a gemm call can run (gemm_plan). */
typedef enum {
    TDI8_FORM_NONE = 0,             /* M == 0 or N == 0: nothing is enqueued */
    TDI8_FORM_PREDICATED = 1,       /* register-staged tiled kernel: any K, alignment, leading dims */
    TDI8_FORM_PIPELINED = 2,        /* LDS-DMA pipelined kernel, whole tiles */
    TDI8_FORM_PIPELINED_EDGE = 3,   /* the same for sizes that end inside a tile */
    TDI8_FORM_SPLIT = 4,            /* zero fill, then the K split of the pipelined kernel (whole tiles) */
    TDI8_FORM_SPLIT_EDGE = 5,       /* zero fill, then the K split of its edge form */
    TDI8_FORM_SKINNY_DMA = 6,       /* skinny kernel fed by LDS DMA (either B layout) */
    TDI8_FORM_SKINNY_PREDICATED = 7,/* skinny kernel with masked register loads */
    TDI8_FORM_SKINNY_ROW_GROUPS = 8,/* zero fill, then the row-major-B column groups of a skinny tile */
    TDI8_FORM_PREDICATED_PREFETCH = 9, /* the predicated kernel with two K tiles of loads in flight:
                                       * column-major B, at most one block per compute unit */
    TDI8_FORM_PERSISTENT = 10       /* persistent whole-tile kernel: a fixed grid walks the tiles;
                                       run only by gemm_s8s8s32_persistent, so gemm_plan, which
                                       describes the other gemm calls, never reports it */
} tdi8_form;

typedef struct {
    int config_id;   /* configuration that runs (-1 with TDI8_FORM_NONE and no id given) */
    int form;        /* tdi8_form */
    int splits;      /* K slices (column groups for TDI8_FORM_SKINNY_ROW_GROUPS); 1 = none */
    int kernels;     /* kernels enqueued: 2 when a zero fill runs first, else 1 (0 for NONE) */
    int grid_x, grid_y, threads;  /* launch shape of the product kernel */
} tdi8_plan;

/* What a gemm call with these arguments would enqueue on the current device,
 * without enqueueing anything: the configuration (config_id -1: the
 * selection's, as gemm_s8s8s32 / gemm_s8s8s32_bt; else that id, as
 * gemm_s8s8s32_with_config), the kernel form and its launch shape.  Patent
 * application CN114238853A, claim 7: at run time the input size decides the
 * configuration and its compiled kernel; the launch wrappers of the contest
 * write-up ("先导杯比赛回顾", NCHW_2_NHWC and 多批次展开的 Im2col 方法)
 * derive the grid from the sizes before launching.  The form depends on the
 * sizes and on the alignment of the pointers and leading dimensions, so the
 * pointers are the ones the call would pass (they are not dereferenced).
 * Same argument checks and status codes as the gemm call; *out is caller
 * owned and written only on TDI8_OK.  One decision serves the call and this
 * query, so the plan is what runs.  Host only; initialises the device. */
int gemm_plan(int config_id, int b_col_major, int M, int N, int K, const int8_t *A, int lda, const int8_t *B,
              int ldb, const int32_t *C, int ldc, tdi8_plan *out);

/* Same product in the persistent form of a general configuration's
 * whole-tile kernel: `blocks` blocks (0: as many as the device holds at once,
 * the compute units times the persistent kernel's resident blocks per unit,
 * rounded down to a multiple of 8; any value is capped at the tile count)
 * each walk the tiles blocks apart in the block-to-tile order of the other
 * forms, which groups the tiles resident on one XCD into a compact region
 * (the contest write-up "先导杯比赛回顾", Swizzle 线程块映射: block order
 * chosen for cache reuse; 矩阵维度高度不均衡: flat waves of blocks lose it).
 * A block's K tiles form one load stream across its tiles, and each finished
 * tile is stored from the accumulation registers while the next tile's
 * matrix work runs, so the C write of one tile overlaps the next one's
 * product.  config_id -1 takes the selection's configuration.  Needs whole
 * tiles of that configuration (M, N, K multiples of its block_m, block_n,
 * block_k), A, B and C 16-byte aligned, lda and ldb multiples of 16 and ldc
 * a multiple of 4; otherwise, or for a skinny configuration, returns
 * TDI8_ERR_BAD_CONFIG and enqueues nothing.  blocks < 0 gives
 * TDI8_ERR_INVALID_VALUE; M == 0 or N == 0 enqueues nothing and returns
 * TDI8_OK.  Arguments, layouts, ownership and the other errors as for
 * gemm_s8s8s32_with_config.  The result is bit-identical to
 * the other forms' (integer sums). */
int gemm_s8s8s32_persistent(int config_id, int b_col_major, int M, int N, int K, const int8_t *A, int lda,
                            const int8_t *B, int ldb, int32_t *C, int ldc, int blocks, hipStream_t stream);

/* ---- int8 2-D convolution (implicit GEMM on the same kernels) ----------------
 *
 * y = conv2d(x, w) with zero padding, stride and dilation: for every image n,
 * output position (p, q) and filter k,
 *   y[n][p][q][k] = sum over r < R, s < S, c < C of
 *                   x[n][p*stride_h + r*dil_h - pad_h][q*stride_w + s*dil_w - pad_w][c] * w[k][r][s][c],
 * taps outside the image contributing 0, accumulated exactly in int32 (mod
 * 2^32 as for the matrix product).  The input position of a tap is the one
 * the contest write-up's im2col kernel uses ("先导杯比赛回顾", 多批次展开的
 * Im2col 方法), and the convolution is computed as the matrix product it
 * lowers to (卷积转化) without materialising that matrix: M = N*P*Q output
 * pixels, N = K filters, reduction R*S*C, the filters being the column-major
 * B operand.
 *
 * Layouts (dense, no padding between rows): x is N x H x W x C (NHWC), w is
 * K x R x S x C (KRSC), y is N x P x Q x K with P = conv2d_output_extent(H,
 * R, pad_h, stride_h, dil_h) and Q likewise.  The caller owns all three
 * (device memory); the library allocates nothing and keeps no pointer.
 * Requirements: y 4-byte aligned; R, S, stride and dilation >= 1, padding
 * >= 0; any channel count C and any alignment of x and w.  With C a multiple
 * of 16 and x and w 16-byte aligned, every 16-byte chunk of the lowered
 * matrix is 16 channels of one tap and goes to LDS by DMA; otherwise (the
 * first layer of a network, C = 3: reduction 27 for 3 x 3 filters) the rows
 * are gathered into registers, a slower form with the same result: with
 * dil_w = 1 a filter row's S*C bytes lie contiguously in the image and are
 * read in 16-byte pieces, else byte by byte.  Errors, all found on the host before anything is enqueued:
 * TDI8_ERR_INVALID_VALUE (a size, y's alignment, or N*P*Q or R*S*C above
 * INT_MAX),
 * TDI8_ERR_NULL_POINTER, TDI8_ERR_ALIASING (y overlaps x or w),
 * TDI8_ERR_UNSUPPORTED_DEVICE, TDI8_ERR_HIP.  N*P*Q == 0 or K == 0 enqueues
 * nothing; C == 0 writes zeros.  Asynchronous on `stream`.  The tile
 * configuration is the selection's for the (N*P*Q) x (R*S*C) by (R*S*C) x K
 * product, from the general family only. */
int conv2d_s8s8s32_nhwc(int N, int H, int W, int C, int K, int R, int S,
                        int pad_h, int pad_w, int stride_h, int stride_w, int dil_h, int dil_w,
                        const int8_t *x, const int8_t *w, int32_t *y, hipStream_t stream);

/* The same with a given general configuration (TDI8_ERR_BAD_CONFIG for a
 * skinny one); for tests and the bench. */
int conv2d_s8s8s32_nhwc_with_config(int config_id, int N, int H, int W, int C, int K, int R, int S,
                                    int pad_h, int pad_w, int stride_h, int stride_w, int dil_h, int dil_w,
                                    const int8_t *x, const int8_t *w, int32_t *y, hipStream_t stream);

/* Configuration id conv2d_s8s8s32_nhwc uses on the current device, or a
 * negative status.  Host only. */
int conv2d_select_config(int N, int H, int W, int C, int K, int R, int S,
                         int pad_h, int pad_w, int stride_h, int stride_w, int dil_h, int dil_w);

/* Output extent along one axis: (H + 2 pad - dil (R - 1) - 1) / stride + 1,
 * or 0 when the dilated filter does not fit; a negative status for invalid
 * arguments.  Host only, no device needed. */
int conv2d_output_extent(int H, int R, int pad, int stride, int dil);

/* The host-side checks of conv2d_s8s8s32_nhwc (no device needed). */
int conv2d_validate(int N, int H, int W, int C, int K, int R, int S,
                    int pad_h, int pad_w, int stride_h, int stride_w, int dil_h, int dil_w,
                    const int8_t *x, const int8_t *w, const int32_t *y);

/* ---- 8-bit operands of a layer: norm and gated activation ----------------------
 *
 * The int8 operand of a product comes from a layer's activations: a row of
 * values y becomes 8-bit values q and a scale, y ~ q * scale, and the product
 * of the q is multiplied by the scales (gemm_s8s8_grouped, gemm_f8f8_block128).
 * Two formats:
 *   s8  int8 with one scale per row: scale = max|y| / 127, q = y / scale
 *       rounded to the nearest integer, ties to even;
 *   f8  8-bit floating point (e4m3: 4 exponent and 3 mantissa bits, largest
 *       value 448, no infinity) with one scale per row and block of 128
 *       columns (the last block may be shorter): scale = max|y| / 448.
 * q is exact: the integer nearest to the real quotient, or the e4m3 value
 * nearest to its 32-bit form (as a conversion from 32 bits gives it), ties to
 * even, whatever the order of the sums: values next to a border between two
 * are decided in 64 bits.  s8 scales are computed in 64 bits and rounded once;
 * f8 scales of the activation, and of the norm of 32-bit values, come from the
 * 32-bit form of the largest value and are off by less than 2^-20.
 * A row (f8: a block) of zeros gets q = 0 and scale = 0; one that holds an
 * infinity or NaN gets q = 0 and scale = NaN.  In the norm an infinity makes
 * the row's other values zeros, NaN makes them NaN: the f8 blocks beside it get
 * q = 0 and scale = 0 or NaN.
 *
 * Types of x, residual, weight, sum, gate and up: */
typedef enum {
    TDI8_F32 = 0,
    TDI8_BF16 = 1,
    TDI8_F16 = 2
} tdi8_type;

/* RMS norm of T rows of H columns with the residual's addition, s8 output:
 *   h = x + residual, rounded to `type` (h = x without a residual),
 *   y[i][j] = h[i][j] * weight[j] / sqrt(mean over j of h[i][j]^2 + eps),
 * q (T x H int8, leading dimension ldq) and scale (T floats) the s8 form of
 * y, and sum (T x H, leading dimension ldsum) = h, the residual stream that
 * the next layer adds to.  The norm is taken of the rounded h, so that it is
 * the norm of what the stream holds.  Sums are held in 64 bits.
 * residual may be NULL (sum must be NULL then); sum may be NULL, or x or
 * residual itself (same pointer and leading dimension; in place), but no
 * output may overlap an input or another output otherwise (TDI8_ERR_ALIASING).
 * Pointers to `type` are aligned to its size, scale to 4 bytes; leading
 * dimensions are in elements, at least H, and H is at most 2^30
 * (TDI8_ERR_INVALID_VALUE otherwise, also for eps < 0 or not finite and an
 * unknown type).  T == 0 or H == 0 enqueues nothing.  One kernel on `stream`
 * (more for over two million rows, by their length);
 * ownership and the other errors as for gemm_s8s8s32. */
int rmsnorm_quant_s8(int type, int T, int H, const void *x, int ldx, const void *residual, int ldr,
                     const void *weight, float eps, void *sum, int ldsum, int8_t *q, int ldq, float *scale,
                     hipStream_t stream);

/* The same with f8 output: q holds e4m3 bytes, scale T rows of
 * ceil(H / 128) floats (leading dimension lds >= ceil(H / 128)). */
int rmsnorm_quant_f8(int type, int T, int H, const void *x, int ldx, const void *residual, int ldr,
                     const void *weight, float eps, void *sum, int ldsum, uint8_t *q, int ldq, float *scale,
                     int lds, hipStream_t stream);

/* Gated activation of T rows of N columns, s8 output:
 *   y[i][j] = gate[i][j] / (1 + exp(-gate[i][j])) * up[i][j].
 * gate and up may be the two halves of one product's rows (leading
 * dimensions at least N).  Outputs, checks and errors as for the norm. */
int swiglu_quant_s8(int type, int T, int N, const void *gate, int ldg, const void *up, int ldu, int8_t *q,
                    int ldq, float *scale, hipStream_t stream);

/* The same with f8 output. */
int swiglu_quant_f8(int type, int T, int N, const void *gate, int ldg, const void *up, int ldu, uint8_t *q,
                    int ldq, float *scale, int lds, hipStream_t stream);

/* ---- products of 8-bit operands with their scales ------------------------------ */

/* int8 products grouped by expert: row r of C belongs to the group (expert) g
 * with offsets[g] <= r < offsets[g + 1] and is
 *   C[r][n] = a_scale[i] * b_scale[g][n] * sum over k of A[i][k] * B_g[n][k],
 * i = rows[r] (or r itself when rows is NULL), the sum exact in int32 and the
 * result rounded to `type` once (fp32 in between: the sum, the scales'
 * product and their product are rounded to 24 bits each).
 *   A        a_rows rows of K int8 (one at least), leading dimension lda;
 *            a_scale a_rows floats
 *   rows     M indices of A's rows, in group order (a router's sorted token
 *            list; an index may occur any number of times), or NULL
 *   offsets  G + 1 rising row numbers on the device, offsets[0] = 0,
 *            offsets[G] <= M; groups may be empty.  NULL with G = 1: one
 *            group of all rows, the dense product
 *   B        G groups of N rows of K int8 (K contiguous), leading dimension
 *            ldb, group_b bytes from one group to the next; b_scale G x N floats
 *   C        M x N values of `type`, leading dimension ldc
 * Rows from offsets[G] on are left as they are.  A row whose index lies
 * outside 0 .. a_rows - 1 becomes zeros (a padding entry).  Offsets that do
 * not rise or that pass M leave some rows undefined; none is read or written
 * outside the operands.  The sizes of the groups are never needed on the
 * host: the call only enqueues one kernel, and may be captured into a graph
 * whose replays see other offsets.
 * K is at most 131071 (no sum can wrap) and the other sizes at most 2^30; a
 * group_b below one group's extent, a_rows < M without rows, a_rows = 0, an
 * unknown type or pointers that are not aligned to their element give
 * TDI8_ERR_INVALID_VALUE, and so does a product whose grid would pass 2^31
 * threads in every tile that its operands allow: never below 4 * 10^6 tiles of
 * 64 x 128 results, each group's rows filled up to 64 (scaled_product_plan
 * says so beforehand).  C may not overlap an input (TDI8_ERR_ALIASING).
 * M, N or G = 0 enqueues nothing; K = 0 writes zeros, whatever the scales.
 * 16-byte aligned A and B with lda, ldb, group_b and K multiples of 16 take
 * the faster kernels.
 * Ownership, streams and the other errors as for gemm_s8s8s32. */
int gemm_s8s8_grouped(int type, int G, int M, int N, int K, const int8_t *A, int lda, int a_rows,
                      const float *a_scale, const int32_t *rows, const int32_t *offsets, const int8_t *B, int ldb,
                      int64_t group_b, const float *b_scale, void *C, int ldc, hipStream_t stream);

/* Product of e4m3 operands with a scale for each block of 128:
 *   C[m][n] = sum over blocks b of a_scale[m][b] * b_scale[n / 128][b] *
 *             (sum over k in 128 b .. 128 b + 127 of A[m][k] * B[n][k]),
 * rounded to `type` once.  With fp32 and fp16 results all sums are held in
 * fp32.  With bf16 results the inner sums are those of the e4m3 matrix
 * instructions, at twice the rate: of 8 consecutive products each is cut,
 * toward zero, to 2^-13 of the largest one's power of two before fp32 takes
 * over.  A result is off by at most 7 * 2^-13 times the sum of the largest
 * product's magnitude of each 8: about 1.5 * 10^-5 of the results' size on
 * normal operands, less than half a step of bf16 (2^-9) wherever large products
 * do not cancel; where they do, ask for fp32 or fp16.
 *   A        M rows of K e4m3 bytes; a_scale M rows of ceil(K / 128) floats
 *            (leading dimension ldas): the f8 form of rmsnorm_quant_f8
 *   B        N rows of K e4m3 bytes (K contiguous); b_scale ceil(N / 128)
 *            rows of ceil(K / 128) floats (leading dimension ldbs)
 *   C        M x N values of `type`
 * NaN operands give NaN.  Checks, errors and the rest as for
 * gemm_s8s8_grouped (K at most 2^30). */
int gemm_f8f8_block128(int type, int M, int N, int K, const uint8_t *A, int lda, const float *a_scale, int ldas,
                       const uint8_t *B, int ldb, const float *b_scale, int ldbs, void *C, int ldc,
                       hipStream_t stream);

/* Kernel forms of the scaled products, for the plan query below. */
typedef enum {
    TDI8_SCALED_NONE = 0,              /* nothing to do */
    TDI8_SCALED_STREAM = 1,            /* few rows: every wave streams its share of K */
    TDI8_SCALED_STREAM_UNALIGNED = 2,  /* the same for operands off 16 bytes */
    TDI8_SCALED_LDS = 3,               /* many rows: both operands staged in LDS */
    TDI8_SCALED_STAGED = 4             /* many rows off 16 bytes: staged through registers */
} tdi8_scaled_form;

typedef struct {
    int form;              /* tdi8_scaled_form */
    int block_m, block_n;  /* the tile */
    int threads;           /* of a block */
    int64_t blocks;        /* of the grid */
} tdi8_scaled_plan;

/* What gemm_s8s8_grouped (f8 = 0) or gemm_f8f8_block128 (f8 = 1, G = 1) would
 * enqueue for these sizes on a device of num_cu compute units; aligned: A, B,
 * lda, ldb, group_b and K are multiples of 16 (and leading dimensions of e4m3
 * operands below 8 * 10^6, beyond which the LDS tiles do not address them).
 * TDI8_ERR_INVALID_VALUE where the call would give it for its sizes.  Needs no
 * device; the calls take the same decision. */
int scaled_product_plan(int f8, int type, int G, int M, int N, int K, int aligned, int num_cu, tdi8_scaled_plan *out);

/* Host-side argument check shared by every gemm entry point (no device
 * needed): returns TDI8_OK or the status the entry point would return. */
int tdi8_validate(int b_col_major, int M, int N, int K, const int8_t *A, int lda,
                  const int8_t *B, int ldb, const int32_t *C, int ldc);

/* Static string for a status code (never NULL; "unknown status" for a value
 * outside tdi8_status; the caller must not free it).  The contest write-up's
 * launch wrappers ("先导杯比赛回顾", NCHW_2_NHWC and 多批次展开的 Im2col 方法)
 * read hipGetLastError after each launch and print its error string; a
 * library prints nothing, so the status code and this text take its place. */
const char *tdi8_status_string(int status);

/* hipError_t of the last failed HIP call made by this thread (0 if none):
 * the error those launch wrappers obtain from hipGetLastError, kept per
 * thread for the caller after an entry point returned TDI8_ERR_HIP. */
int tdi8_last_hip_error(void);

/* Identity of the GPU code of the GEMM and convolution kernels compiled into
 * this library: the first 16 hex digits of the SHA-256 of the gfx950 code
 * objects of every configuration, in configuration order (static string; the
 * caller must not free it).  Two builds report the same value exactly when
 * those kernels are the same machine code, so a measurement taken on one build
 * (a counter pass, a kernel trace) can record it and be matched against the
 * library that runs later.  Not part of the pages' method: a build identity
 * for measurements. */
const char *tdi8_kernel_code_hash(void);

/* The same for the kernels of the 8-bit layer operators (rows, grouped and
 * block-scaled products). */
const char *tdi8_layer_code_hash(void);

#ifdef __cplusplus
}
#endif

#endif /* TDI8_H */
