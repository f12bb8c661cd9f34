/*
 * batchlas -- batched Cholesky factorisation (potrf) and positive-definite
 * solve (posv) for many small independent Hermitian positive-definite
 * matrices, on AMD Instinct MI355X (gfx950), and the operators of layers whose
 * 4-bit weights those solves calibrate ("Low-bit layer operators" below).
 *
 * The operations are the ones described on the BatchLAS documentation's
 * perf_potrf page:
 *   potrf  factors every matrix of a batch as A = L L^H (Lower) or
 *          A = U^H U (Upper); Upper is the same recurrence applied to
 *          S(i,c) = conj(A(c,i)) (section "Selection", can_run() terms);
 *   posv   factors A and then solves A X = B with a forward solve L y = b and
 *          a backward solve L^H x = y per right-hand side (sections "posv
 *          selection", "The fused posv tier", "The fused potrs solve").
 * Per-matrix failure is reported through info, with the first failing
 * column winning (section "potrf: correctness findings", item 6).
 *
 * Conventions shared by the potrf and posv entry points
 * -----------------------------------------------------
 * Memory   All array pointers are DEVICE pointers owned by the caller.  The
 *          library allocates nothing persistent, keeps no pointer after it
 *          returns and makes no host<->device copy of its own.
 * Layout   Column-major.  Matrix b's element (i, c) is at
 *          A[b * strideA + c * lda + i].  lda, ldb and the strides count
 *          ELEMENTS and are 64-bit.  Complex elements are interleaved
 *          (re, im) pairs of the real type.  Matrices must not overlap
 *          (strideA >= lda * n).
 * Effects  potrf overwrites the referenced triangle of each A with L (Lower)
 *          or U (Upper); the diagonal is real and positive, with imaginary
 *          part +0.  The other triangle and all padding are neither read nor
 *          written.  posv also overwrites B with X for every item whose info
 *          is 0 and leaves B unchanged for an item whose info is nonzero.
 *          The imaginary part of an input diagonal is ignored.
 * info     int32[batch] device array: 0 on success, else the 1-based column
 *          of the first Schur pivot d with !(d > 0) (zero, negative and NaN
 *          pivots fail); a later failure never overwrites it.  For a failed
 *          item the leading info-1 columns hold the factor of the leading
 *          block; the rest of the referenced triangle is unspecified.  info
 *          may be NULL, in which case nothing is written.
 * Errors   Arguments are checked synchronously, before anything is enqueued
 *          and with no writes, in this order: n, nrhs, batch >= 1; lda, ldb
 *          >= n; strideA >= lda*n, strideB >= ldb*nrhs; non-null A (and B);
 *          dtype and uplo valid; the route runnable.  Numerical failure is
 *          never a status: it is reported only through info.  No C++
 *          exception crosses this interface.
 * Streams  Work is enqueued on `stream` (a hipStream_t; NULL is the default
 *          stream) with no internal synchronisation: results are valid once
 *          the stream has been synchronised.  The environment (route pins,
 *          trace) is read once, at the first call; there is no other global
 *          state, so calls from several host threads are safe.
 */
#ifndef BATCHLAS_H
#define BATCHLAS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same underlying type as hipStream_t, so a hipStream_t converts implicitly. */
typedef struct ihipStream_t *batchlas_stream_t;

typedef enum { BATCHLAS_LOWER = 0, BATCHLAS_UPPER = 1 } batchlas_uplo;

typedef enum {
    BATCHLAS_F32 = 0,   /* float                    */
    BATCHLAS_F64 = 1,   /* double                   */
    BATCHLAS_C64 = 2,   /* complex float  (re, im)  */
    BATCHLAS_C128 = 3   /* complex double (re, im)  */
} batchlas_dtype;

typedef enum {
    BATCHLAS_OK = 0,
    BATCHLAS_INVALID_VALUE = 1,   /* a size, leading dimension, stride, dtype, uplo or alignment is out of range */
    BATCHLAS_NULL_POINTER = 2,    /* A (or B, or an operator's array) is NULL                        */
    BATCHLAS_NOT_SUPPORTED = 3,   /* no kernel family serves this shape / the pinned family cannot   */
    BATCHLAS_HIP_ERROR = 4,       /* the HIP runtime reported an error while enqueueing              */
    BATCHLAS_INTERNAL = 5         /* an internal invariant failed                                    */
} batchlas_status;

/* Kernel families (the route).  AUTO lets the size dispatcher choose. */
typedef enum {
    BATCHLAS_FAMILY_AUTO = 0,
    BATCHLAS_FAMILY_TINY = 1,       /* registers, several matrices per wavefront          */
    BATCHLAS_FAMILY_LDS = 2,        /* one workgroup per matrix, matrix staged in LDS      */
    BATCHLAS_FAMILY_BLOCKED = 3,    /* panel factor + solve, MFMA trailing rank-k update   */
    BATCHLAS_FAMILY_POSV_TINY = 4,  /* fused factor + both solves in registers (posv only) */
    BATCHLAS_FAMILY_POSV_SPLIT = 5  /* potrf by any family, then a fused two-solve kernel  */
} batchlas_family;

/* Launch geometry chosen for a call (for tests and tracing). */
typedef struct {
    int32_t family;             /* batchlas_family actually used                         */
    int32_t lanes_per_matrix;   /* tiny / posv: lanes that share one matrix (P); in the
                                   wide fp32 window (orders 65..192) the workgroup         */
    int32_t rows_per_lane;      /* tiny / posv: rows each lane holds (R)                  */
    int32_t matrices_per_wave;  /* tiny / posv: matrices packed in one wavefront (G); 1
                                   in the wide window (one matrix per workgroup)           */
    int32_t block_threads;      /* threads per workgroup of the main kernel              */
    int32_t panel;              /* lds / blocked: panel width (nb); wide fp32 tiles: their
                                   column count; 0 otherwise                               */
    int64_t grid;               /* workgroups of the main kernel (first launch)          */
    int64_t lds_bytes;          /* LDS per workgroup of the main kernel                   */
} batchlas_route_info;

/*
 * potrf: factor `batch` Hermitian positive-definite n x n matrices in place.
 *   dt, uplo   element type; which triangle is referenced and overwritten
 *   n          order, >= 1
 *   A          device pointer to the first matrix (see Layout)
 *   lda        leading dimension in elements, >= n
 *   strideA    distance between consecutive matrices in elements, >= lda*n
 *   batch      number of matrices, >= 1
 *   info       device int32[batch] or NULL (see info)
 *   stream     HIP stream for the work
 * Returns BATCHLAS_OK once the work is enqueued.
 */
batchlas_status batchlas_potrf(batchlas_dtype dt, batchlas_uplo uplo, int64_t n,
                               void *A, int64_t lda, int64_t strideA, int64_t batch,
                               int32_t *info, batchlas_stream_t stream);

/*
 * posv: factor each A as potrf does, then solve A X = B for nrhs right-hand
 * sides per item, overwriting B with X.
 *   B          device pointer, n x nrhs per item, column-major
 *   ldb        >= n;  strideB >= ldb * nrhs
 * Other arguments as for batchlas_potrf.  A is overwritten with the factor.
 * Small orders with nrhs <= 4 run fused in one kernel (POSV_TINY); every
 * other shape that potrf serves runs as potrf followed by one kernel for both
 * triangular solves (POSV_SPLIT), which also keeps B of failed items when
 * info is NULL (it reads the failure off the factor's diagonal).
 */
batchlas_status batchlas_posv(batchlas_dtype dt, batchlas_uplo uplo, int64_t n, int64_t nrhs,
                              void *A, int64_t lda, int64_t strideA,
                              void *B, int64_t ldb, int64_t strideB, int64_t batch,
                              int32_t *info, batchlas_stream_t stream);

/*
 * Same operations with an explicit family instead of the dispatcher's choice
 * (or the environment pin).  A family that cannot run the shape returns
 * BATCHLAS_NOT_SUPPORTED before anything is enqueued.
 */
batchlas_status batchlas_potrf_family(batchlas_family family, batchlas_dtype dt,
                                      batchlas_uplo uplo, int64_t n, void *A, int64_t lda,
                                      int64_t strideA, int64_t batch, int32_t *info,
                                      batchlas_stream_t stream);
batchlas_status batchlas_posv_family(batchlas_family family, batchlas_dtype dt,
                                     batchlas_uplo uplo, int64_t n, int64_t nrhs,
                                     void *A, int64_t lda, int64_t strideA,
                                     void *B, int64_t ldb, int64_t strideB, int64_t batch,
                                     int32_t *info, batchlas_stream_t stream);

/* Typed wrappers (s = float, d = double, c = complex float, z = complex double). */
batchlas_status batchlas_spotrf(batchlas_uplo uplo, int64_t n, float *A, int64_t lda,
                                int64_t strideA, int64_t batch, int32_t *info,
                                batchlas_stream_t stream);
batchlas_status batchlas_dpotrf(batchlas_uplo uplo, int64_t n, double *A, int64_t lda,
                                int64_t strideA, int64_t batch, int32_t *info,
                                batchlas_stream_t stream);
batchlas_status batchlas_cpotrf(batchlas_uplo uplo, int64_t n, void *A, int64_t lda,
                                int64_t strideA, int64_t batch, int32_t *info,
                                batchlas_stream_t stream);
batchlas_status batchlas_zpotrf(batchlas_uplo uplo, int64_t n, void *A, int64_t lda,
                                int64_t strideA, int64_t batch, int32_t *info,
                                batchlas_stream_t stream);
batchlas_status batchlas_sposv(batchlas_uplo uplo, int64_t n, int64_t nrhs, float *A,
                               int64_t lda, int64_t strideA, float *B, int64_t ldb,
                               int64_t strideB, int64_t batch, int32_t *info,
                               batchlas_stream_t stream);
batchlas_status batchlas_dposv(batchlas_uplo uplo, int64_t n, int64_t nrhs, double *A,
                               int64_t lda, int64_t strideA, double *B, int64_t ldb,
                               int64_t strideB, int64_t batch, int32_t *info,
                               batchlas_stream_t stream);
batchlas_status batchlas_cposv(batchlas_uplo uplo, int64_t n, int64_t nrhs, void *A,
                               int64_t lda, int64_t strideA, void *B, int64_t ldb,
                               int64_t strideB, int64_t batch, int32_t *info,
                               batchlas_stream_t stream);
batchlas_status batchlas_zposv(batchlas_uplo uplo, int64_t n, int64_t nrhs, void *A,
                               int64_t lda, int64_t strideA, void *B, int64_t ldb,
                               int64_t strideB, int64_t batch, int32_t *info,
                               batchlas_stream_t stream);

/*
 * Route query: the family and launch geometry a call with these arguments
 * would use (nrhs = 0 asks about potrf, nrhs >= 1 about posv).  `family`
 * pins a family as in the *_family entry points; AUTO applies the dispatcher
 * and the environment pin.  Host-only: makes no HIP call.  Validates its
 * arguments like the operation would (pointers are not checked).
 */
batchlas_status batchlas_route(batchlas_family family, batchlas_dtype dt, batchlas_uplo uplo,
                               int64_t n, int64_t nrhs, int64_t lda, int64_t strideA,
                               int64_t batch, batchlas_route_info *out);

/*
 * Low-bit layer operators
 * -----------------------
 * What a layer with 4-bit weights runs beside the solves that calibrate it: the
 * weights' rounding in groups (its error is pushed onto the columns not yet
 * rounded by a positive-definite solve), products of a few tokens with such
 * weights, and the root-mean-square norm that writes their activations in 8
 * bits, with its gradient.
 *
 * Layout   Matrices here are ROW-major: element (i, c) of x is x[i * ldx + c]
 *          with ldx >= the row's length, in elements.  Rows may start at any
 *          address that is a multiple of the element size, except for codes.
 * Memory   Device pointers owned by the caller, as above.  Buffers do not
 *          overlap, except that h of rmsnorm_quant may be x or r itself, and
 *          dx of rmsnorm_grad may be dy, h or dh itself (same leading
 *          dimension).
 * Empty    rows (m) may be 0: nothing is computed (dw is set to zero).
 * Errors   Checked synchronously, before anything is enqueued and with no
 *          writes, in this order: types, formats and group; sizes; leading
 *          dimensions; non-null pointers; alignment; the shape supported.
 * Streams  As above.  Every operator gives the same bits on every run, and can
 *          be captured in a graph.
 *
 * 8-bit values are e4m3 floats (1 sign, 4 exponent, 3 mantissa bits, bias 7, no
 * infinity, 0x7f is NaN, largest 448).  Their scales are either one per row (a
 * float) or one per block of 32 columns (a byte b meaning 2^(b - 127), 255
 * meaning NaN; the last block of a row may be shorter).  A value is its e4m3
 * float times its scale.
 *
 * 4-bit weights are codes, two to a byte, column c of a row in byte c / 2, even
 * columns in the low four bits.  Rows of codes are held in whole 16 bytes,
 * which weight_matvec reads (the padding may hold anything): codes and ldc (in
 * bytes, >= (k + 1) / 2) are multiples of 16.  Each group of `group` columns has a scale (the last group of a row may be shorter):
 *   INTEGER  code u in 0..15 is (u - z) * scale, scale in bf16, z the group's
 *            byte in `zeros` (0..15), 8 where zeros is NULL; group 32, 64 or 128
 *   FLOAT    code is an e2m1 float (1 sign bit, then 0 0.5 1 1.5 2 3 4 6) times
 *            scale, a byte b meaning 2^(b - 127), 255 meaning NaN; group 32
 */
typedef enum {
    BATCHLAS_TYPE_F32 = 0,    /* float                          */
    BATCHLAS_TYPE_F16 = 1,    /* half                           */
    BATCHLAS_TYPE_BF16 = 2,   /* bfloat16                       */
    BATCHLAS_TYPE_E4M3 = 3    /* 8-bit float, only with scales  */
} batchlas_type;

typedef enum {
    BATCHLAS_SCALE_NONE = 0,
    BATCHLAS_SCALE_ROW = 1,     /* float[rows]                                    */
    BATCHLAS_SCALE_BLOCK = 2    /* a byte per 32 columns, row stride in bytes     */
} batchlas_scale;

typedef enum {
    BATCHLAS_FORMAT_INTEGER = 0,
    BATCHLAS_FORMAT_FLOAT = 1
} batchlas_format;

/*
 * rmsnorm_quant: for every row,
 *   h = x + r,   v = w * h / sqrt(mean(h^2) + eps),   q = e4m3(v / scale)
 * in 32 bits; v comes from h before h is rounded to the type.
 *   type     F32, F16 or BF16: of x, r, w and h
 *   scale    ROW: scales[i] = max(max|v| / 448, 2^-126), a float;
 *            BLOCK: 2^e with the least e in -127..127 for which
 *            max|v| <= 448 * 2^e, a byte e + 127, at scales[i * lds + block]
 *   r        NULL: no residual, and h must be NULL
 *   h        receives x + r, rounded to the type; NULL: not stored
 *   eps      >= 0
 *   lds      >= (n + 31) / 32 for BLOCK; not read for ROW
 * A row (block) that holds a v that is not finite gets a NaN scale and NaN
 * values; a row of zeros gets the smallest scale and zeros.
 * n is at most 32768, else NOT_SUPPORTED.
 */
batchlas_status batchlas_rmsnorm_quant(batchlas_type type, batchlas_scale scale, int64_t rows,
                                       int64_t n, const void *x, int64_t ldx, const void *r,
                                       int64_t ldr, const void *w, double eps, void *h,
                                       int64_t ldh, uint8_t *q, int64_t ldq, void *scales,
                                       int64_t lds, batchlas_stream_t stream);

/*
 * rmsnorm_grad: the gradient of the norm at the stored h.  With
 * s = 1 / sqrt(mean(h^2) + eps), and dy the gradient of v,
 *   dx = dh + s * (dy * w - h * s^2 * mean(dy * w * h))      (of x and of r)
 *   dw = sum over rows of dy * h * s                         (float[n])
 *   dh       the gradient that reaches h on the residual path; NULL: zero
 *   dw       NULL: not computed
 *   workspace  device memory of at least the bytes that
 *            batchlas_rmsnorm_grad_workspace gives, aligned to 4 bytes; not
 *            used (may be NULL) where that is 0 or dw is NULL
 * n is at most 16384, else NOT_SUPPORTED.
 */
batchlas_status batchlas_rmsnorm_grad(batchlas_type type, int64_t rows, int64_t n, const void *dy,
                                      int64_t lddy, const void *h, int64_t ldh, const void *w,
                                      const void *dh, int64_t lddh, double eps, void *dx,
                                      int64_t lddx, float *dw, void *workspace,
                                      int64_t workspace_bytes, batchlas_stream_t stream);

/* Host-only: the workspace that rmsnorm_grad of this size needs, in bytes. */
batchlas_status batchlas_rmsnorm_grad_workspace(batchlas_type type, int64_t rows, int64_t n,
                                                int64_t *bytes);

/*
 * weight_quant: rounds the rows of W (n x k) to 4 bits.  Per group of columns:
 *   INTEGER, zeros NULL:  scale = max(bf16(max|w| / 7), 2^-126),
 *       u = clamp(rint(w / scale), -8, 7) + 8
 *   INTEGER, zeros given: lo = min(w, 0), hi = max(w, 0),
 *       scale = max(bf16((hi - lo) / 15), 2^-126),
 *       z = clamp(rint(-lo / scale), 0, 15), u = clamp(rint(w / scale) + z, 0, 15)
 *   FLOAT: scale 2^e with the least e in -127..127 for which
 *       max|w| <= 6 * 2^e, code = e2m1(w / scale)
 * Every rounding is to nearest, ties to even; quotients are rounded to 32 bits.
 *   type     F32, F16 or BF16: of W and of values
 *   scales   bf16 (INTEGER) or bytes (FLOAT), group g of row i at
 *            scales[i * lds + g]; zeros likewise with ldz, NULL for FLOAT
 *   values   receives what the codes stand for, rounded to the type; NULL: not
 *            stored
 * A group that holds a weight that is not finite, or whose hi - lo overflows,
 * gets a NaN scale, codes of zero (and z = 8) and NaN values.  The unused half byte of an odd k is a code
 * of zero; bytes beyond (k + 1) / 2 of a row are not written.
 */
batchlas_status batchlas_weight_quant(batchlas_type type, batchlas_format format, int64_t group,
                                      int64_t n, int64_t k, const void *W, int64_t ldw,
                                      uint8_t *codes, int64_t ldc, void *scales, int64_t lds,
                                      uint8_t *zeros, int64_t ldz, void *values, int64_t ldv,
                                      batchlas_stream_t stream);

/*
 * weight_matvec: y = x W^T, y (m x n), x (m x k), W (n x k) held as codes, sums
 * in 32 bits.  Made for the few rows of a decoding step (m up to about 64);
 * any m up to 2^21 is computed, reading W once per 64 rows.  x and the codes
 * less their zero points go into the products exactly, so the error follows
 * sum |x| |W|.  Where a sum of codes times x leaves the range of 32 bits, the
 * element is computed again in 64 bits (much more slowly), so that y is
 * finite, infinite or NaN as the definition has it.
 *   xtype, xscale   F16 or BF16 with NONE, or E4M3 with ROW (xscales float[m])
 *            or BLOCK (bytes, row stride ldxs >= (k + 31) / 32)
 *   ytype    F32, F16 or BF16
 *   workspace  device memory of at least the bytes that
 *            batchlas_weight_matvec_workspace gives, aligned to 16 bytes; not
 *            used (may be NULL) where that is 0, which it is for m <= 16
 * NOT_SUPPORTED: m beyond 2^21, n beyond 2^24, ldx or ldc beyond 2^27, m * k
 * beyond 2^34.
 */
batchlas_status batchlas_weight_matvec(batchlas_type xtype, batchlas_scale xscale,
                                       batchlas_type ytype, batchlas_format format, int64_t group,
                                       int64_t m, int64_t n, int64_t k, const void *x,
                                       int64_t ldx, const void *xscales, int64_t ldxs,
                                       const uint8_t *codes, int64_t ldc, const void *scales,
                                       int64_t lds, const uint8_t *zeros, int64_t ldz, void *y,
                                       int64_t ldy, void *workspace, int64_t workspace_bytes,
                                       batchlas_stream_t stream);

/* Host-only: the workspace that weight_matvec of this size needs, in bytes. */
batchlas_status batchlas_weight_matvec_workspace(int64_t m, int64_t k, int64_t *bytes);

/* Static text for a status code. */
const char *batchlas_status_string(batchlas_status s);

/* The message of the last failing call made by this host thread ("" if none). */
const char *batchlas_last_error(void);

/* Library version, major * 10000 + minor * 100 + patch. */
int32_t batchlas_version(void);

#ifdef __cplusplus
}
#endif

#endif /* BATCHLAS_H */
