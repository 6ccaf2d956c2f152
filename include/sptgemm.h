/*
 * sptgemm.h -- C ABI of the software-pipelined tiled GEMM library for
 * NVIDIA GB300 (sm_103a).
 *
 * The operation is the tiled matrix multiply C = A * B of "Hiding Memory
 * Latency in CUDA: Asynchronous Loads and Software Pipelines" (opening
 * section: load A and B tiles, stage them in shared memory, multiply on the
 * tensor cores, advance to the next K tile), software-pipelined so that the
 * load of K-tile k+1 overlaps the multiply-accumulate of K-tile k (same
 * page, sections 1, 5 and 11; "Pipeline GPU Kernel", Step 3). Pipelining
 * reorders loads and leaves the arithmetic alone ("Pipeline GPU Kernel",
 * Step 5 item 4): the result is the plain product.
 *
 * Layouts (all dense, leading dimensions implied by the shape):
 *   A  row-major    M x K : element (i, k) at A[i*K + k]
 *   B  column-major K x N : element (k, j) at B[j*K + k]
 *   C  row-major    M x N : element (i, j) at C[i*N + j]
 *
 * Ownership: the caller owns A, B and C, which are device pointers (any
 * allocation the CUDA runtime can address on the current device). The
 * library keeps no pointer past a call. It owns one cached scratch area per
 * (device, stream) for the paths that need one (int8 operand conversion,
 * split-K partial sums), grown on demand and released at unload.
 *
 * Streams: every call is asynchronous on `stream` (a cudaStream_t; NULL is
 * the legacy default stream) and never synchronizes. Inputs must stay valid
 * and C untouched by others until the stream reaches the call.
 *
 * Errors: functions return an int status, 0 on success, a negative
 * SPTG_ERR_* code otherwise. No call aborts the process and there is no CPU
 * fallback: on a machine without an sm_103 device the call fails.
 */
#ifndef SPTGEMM_H
#define SPTGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Input/output element pairs. Float inputs accumulate in fp32; int8 inputs
 * accumulate exactly and return int32. */
typedef enum {
  SPTG_F16_F32 = 0,   /* binary16 A, B -> fp32 C                 */
  SPTG_F16_F16 = 1,   /* binary16 A, B -> binary16 C (RN-even)   */
  SPTG_S8_S32 = 2,    /* int8 A, B -> int32 C, bit-exact while the
                         sum fits int32 (any inputs for K < 131072);
                         beyond, it wraps modulo 2^32               */
  SPTG_BF16_BF16 = 3, /* bfloat16 A, B -> bfloat16 C (RN-even)   */
  SPTG_BF16_F32 = 4,  /* bfloat16 A, B -> fp32 C                 */
  /* range markers, not dtypes: they make sptg_dtype span every 32-bit int,
     so any value a caller passes is representable and is rejected with
     SPTG_ERR_ARG unless it names one of the pairs above */
  SPTG_DTYPE_RANGE_MIN_ = -2147483647 - 1,
  SPTG_DTYPE_RANGE_MAX_ = 2147483647
} sptg_dtype;

enum {
  SPTG_OK = 0,
  SPTG_ERR_ARG = -1,         /* null pointer with a nonzero extent, negative or
                                too-large dimension, unknown dtype or option   */
  SPTG_ERR_ALIGN = -2,       /* a pointer not 16-byte aligned, or a row pitch
                                (K*sizeof(in), N*sizeof(out)) not a multiple
                                of 16 bytes, as the tensor-copy engine needs  */
  SPTG_ERR_UNSUPPORTED = -3, /* no CUDA device of compute capability 10.3    */
  SPTG_ERR_LAUNCH = -4,      /* a CUDA runtime error; see sptg_last_error()  */
  SPTG_ERR_TIMEOUT = -5,     /* a kernel gave up a bounded wait (reported by
                                sptg_device_error); C's contents are then
                                unspecified                                   */
  SPTG_ERR_NOMEM = -6,       /* scratch memory could not be allocated        */
  SPTG_ERR_CONFIG = -7       /* a forced configuration does not fit          */
};

/*
 * C = A * B.  M, N, K >= 0.  M == 0 or N == 0: nothing is done.  K == 0:
 * C is set to zero (the empty sum).  Shapes need not be multiples of any
 * tile: edges are zero-filled on load and clipped on store.
 *
 * Alignment: A, B, C 16-byte aligned; K * sizeof(input) and
 * N * sizeof(output) multiples of 16 bytes.  Otherwise SPTG_ERR_ALIGN.
 */
int sptg_gemm(int64_t M, int64_t N, int64_t K, sptg_dtype dtype,
              const void* A, const void* B, void* C, void* stream);

/* Kernel selection for sptg_gemm_ex; fields left at 0 mean "choose". */
typedef struct {
  int kernel;   /* 0 auto, 1 square, 2 skinny swap-AB with stream-K split,
                   3 skinny swap-AB with the K split across a cluster of
                   CTAs (splits = cluster size, 1, 2 or 4), 4 skinny
                   (M <= 64, float) with one CTA per strip of output columns
                   over the whole of K (bn = strip width), 5 skinny swap-AB
                   (M <= 256, float) on CTA pairs with the 2-SM MMA over the
                   whole of K (bn = output columns per CTA)                  */
  int bn;       /* square: tile columns, 112 to 256 in steps of 16 for
                   float types (int8: 128, 160, 192, 224 or 256), or 512 for
                   float CTA pairs; skinny column strips (kernel 4):
                   a multiple of 8 from 8 to 256; skinny CTA pairs (kernel
                   5): a multiple of 8 from 8 to 128                         */
  int stages;   /* shared-memory ring depth (1 = synchronous load/compute)  */
  int splits;   /* square: cap on persistent workers; skinny stream-K: CTAs
                   sharing the work (0 = SM count); skinny cluster: cluster
                   size                                                      */
  int timeout_ms; /* bounded-wait limit inside the kernel (0 = default 2000) */
  int inject_stall; /* test hook: 1 makes the producer withhold one k-tile so
                       the consumer's bounded wait runs out; 0 = off          */
  int cta_pair; /* square: 0 choose, 1 one CTA (128-row tiles), 2 a CTA pair on
                   two SMs with the 2-SM MMA (256-row tiles); every CTA
                   copies its own operand tiles (no multicast copies)       */
  int no_overlap; /* 1: launch without programmatic dependent launch (the
                     kernel then starts only after the previous one ends)    */
  void* trace;  /* optional device buffer of SPTG_TRACE_WORDS uint64 (8-byte
                   aligned, zeroed by the caller): word [8*cta + e] is the
                   %globaltimer ns of event e of CTA cta (first 1024 CTAs):
                   0 set-up done, 1 first copy issued, 2 first stage full at
                   the MMA issuer, 3 last copy issued, 4 last MMA committed,
                   5 epilogue done, 6 exit, 7 last split-K reduction; then
                   for CTA 0, the issue time of K-tiles 0..63 (words 8192..)
                   and the time the MMA issuer found each full (8256..);
                   NULL = off                                               */
  int stream_k; /* square kernel: 0 choose (the tiles of a partial last
                   round are cut along K over all workers), 1 never, 2 every
                   tile (a test setting)                                    */
} sptg_config;

#define SPTG_TRACE_WORDS (8 * 1024 + 2 * 64)

/* sptg_gemm with an explicit configuration (NULL = sptg_gemm). */
int sptg_gemm_ex(int64_t M, int64_t N, int64_t K, sptg_dtype dtype,
                 const void* A, const void* B, void* C, void* stream,
                 const sptg_config* cfg);

/*
 * sptg_gemm_ex on matrices inside larger row-pitched buffers ("Pipeline GPU
 * Kernel", pitfalls: boundary handling; the tiles are read and written
 * through the row pitch, never past a row's K or N elements).
 *
 *   lda  elements between rows of A        (>= K)
 *   ldb  elements between the K-long columns of B, i.e. rows of the N x K
 *        array Bcm                          (>= K)
 *   ldc  elements between rows of C        (>= N)
 *
 * Besides the alignment rules of sptg_gemm (which still apply to K and N),
 * lda * sizeof(in), ldb * sizeof(in) and ldc * sizeof(out) must be multiples
 * of 16 bytes (SPTG_ERR_ALIGN), and each leading dimension must be below
 * 2^31 (SPTG_ERR_ARG). Elements between N and ldc of a row of C are never
 * written. lda = ldb = K and ldc = N give sptg_gemm_ex.
 */
int sptg_gemm_strided(int64_t M, int64_t N, int64_t K, sptg_dtype dtype,
                      const void* A, int64_t lda, const void* B, int64_t ldb,
                      void* C, int64_t ldc, void* stream, const sptg_config* cfg);

/*
 * sptg_gemm_ex on HOST buffers: A (M x K), B (the N x K array Bcm) and C
 * (M x N), dense, in host memory. The call enqueues on `stream` the copies of
 * A and B to device buffers the library owns (one set per device and stream,
 * grown on demand and freed in stream order), the product, and the copy of
 * C back to the host, and returns without waiting. The caller keeps A, B and
 * C alive and leaves C alone until the stream has reached this point.
 * Page-locked (pinned) host memory makes the copies asynchronous; pageable
 * memory works but the driver then stages it and the call may block. The
 * pitch rules of sptg_gemm apply (SPTG_ERR_ALIGN); the pointers themselves
 * need no alignment. The pages have no counterpart: this is the call a
 * caller whose data lives in host memory makes, and bench.py's end-to-end
 * measurement goes through it.
 */
int sptg_gemm_host(int64_t M, int64_t N, int64_t K, sptg_dtype dtype,
                   const void* A, const void* B, void* C, void* stream,
                   const sptg_config* cfg);

/*
 * The software-pipelined ring on its own: out[i] = alpha * in[i] for
 * i < n, binary32, one rounding per element. This is the minimal working
 * example of "Hiding Memory Latency in CUDA: Asynchronous Loads and Software
 * Pipelines" (section 8: a vector streamed through a multi-stage
 * shared-memory ring and scaled by two), here for any alpha; it measures the
 * copy pipeline against memory bandwidth.
 *
 * in and out are device pointers, 16-byte aligned (else SPTG_ERR_ALIGN),
 * and may be the same buffer (in place); they must not otherwise overlap.
 * n >= 0 of any size (n == 0: nothing). Asynchronous on `stream`.
 */
int sptg_stream_scale(int64_t n, float alpha, const float* in, float* out, void* stream);

/* sptg_stream_scale with the timeout_ms, inject_stall, no_overlap and trace
 * fields of a configuration (the others are ignored; NULL = defaults). */
int sptg_stream_scale_ex(int64_t n, float alpha, const float* in, float* out, void* stream,
                         const sptg_config* cfg);

/* Static text for a status code. */
const char* sptg_status_string(int status);

/* Text of the last CUDA runtime error seen by this thread ("" if none). */
const char* sptg_last_error(void);

/* Writes "kernel=... bm=... bn=... bk=... stages=... ..." for the last call
 * made by this thread into buf (NUL-terminated, truncated to len).
 * Returns the length the full text needs. */
int sptg_last_config(char* buf, size_t len);

/* Synchronizes `stream`, then reads and clears the current device's error
 * word written by timed-out waits. Returns SPTG_OK or SPTG_ERR_TIMEOUT
 * (or SPTG_ERR_LAUNCH if synchronization itself failed). */
int sptg_device_error(void* stream);

/*
 * Allocation-free variant of the skinny (M <= 64) kernel.
 *
 * This call has no counterpart in the paper. It exists for callers that
 * cannot let a library allocate device memory: a serving process that reserves the GPU's
 * memory for its own pool up front (a library cudaMalloc would then fail or
 * fragment that pool), and latency-critical code that cannot accept the
 * device-wide synchronisation a cudaMalloc or cudaFree may imply.
 *
 * It computes exactly what sptg_gemm computes for the same arguments, with
 * the same kernel, but keeps its split-K partial sums and arrival counters in
 * one fixed array compiled into the library (SPTG_NOALLOC_PARTIAL_BYTES +
 * SPTG_NOALLOC_COUNTER_BYTES of device memory, held on every GPU that loads
 * the library until the process exits). It calls no cudaMalloc, cudaFree or
 * other allocating routine.
 *
 *  - dtype: the float pairs only (not SPTG_S8_S32), and M <= 64; otherwise
 *    SPTG_ERR_CONFIG. A, B, C, stream, alignment and return codes as for
 *    sptg_gemm.
 *  - A shape whose split needs more partial-tile bytes (column tiles of 128 x
 *    contributing CTAs x 32 KiB) or counter bytes than the fixed array holds
 *    is rejected with SPTG_ERR_CONFIG; sptg_last_error() gives the sizes.
 *  - The first call on a device looks up the array's device address (with
 *    that device current); make that first call before any stream capture.
 *  - Every call uses the same array, which keeps the last call's partial
 *    sums and counters. Each call tags the counters it uses with a new call
 *    number, so whatever an earlier call left there (even one whose kernel
 *    gave up a wait) is never taken for this call's. Calls whose kernels
 *    overlap on the GPU (two streams, or two threads) race on the array:
 *    serialise them.
 */
#define SPTG_NOALLOC_PARTIAL_BYTES (8u << 20)
#define SPTG_NOALLOC_COUNTER_BYTES (64u << 10)
int sptg_gemm_skinny_noalloc(int64_t M, int64_t N, int64_t K, sptg_dtype dtype,
                             const void* A, const void* B, void* C, void* stream);

/* Library ABI version (major*100 + minor). */
int sptg_version(void);

/*
 * The square kernel's plan for a shape, computed on the host alone (no
 * device is touched), for a GPU of `sm_count` SMs: the tile shape and the
 * schedule sptg_gemm_ex would choose with configuration `cfg` (NULL =
 * defaults), before any fallback for a missing ring depth. On success
 * out[0..6] = tile columns BN, tile mode (0 one CTA, 1 CTA pair), tiles of
 * the schedule, workers (CTAs or pairs), tiles cut along K (stream-K),
 * workers sharing them, and the most contributors one cut tile can have. The
 * worker count assumes every SM holds one CTA; the library itself asks the
 * device how many pairs fit. SPTG_ERR_ARG for a non-positive dimension, fewer
 * than 2 SMs, an unknown dtype or an invalid field; SPTG_ERR_CONFIG when a
 * forced width does not exist for the dtype and pairing.
 */
int sptg_plan_square(int64_t M, int64_t N, int64_t K, sptg_dtype dtype, int sm_count,
                     const sptg_config* cfg, int* out);

/*
 * The whole kernel choice sptg_gemm_ex would make for a shape with
 * configuration `cfg` (NULL = defaults) on a GPU of `sm_count` SMs, computed
 * on the host alone (no device is touched). On success out[0..5] = kernel
 * (1 square, 2 skinny stream-K, 3 skinny cluster split, 4 skinny column
 * strips, 5 skinny CTA pairs -- the sptg_config.kernel numbering), tile width
 * (square: BN; 2 and 3: 128; 4: strip width; 5: output columns per CTA),
 * CTAs launched, CTAs per cluster (1, 2 or 4), the rows of A on a skinny
 * MMA's N side (64, 128 or 256; 0 for the square kernel) and, for the square
 * kernel, the tiles cut along K. Assumes every SM holds one CTA and every
 * cluster of the chosen size fits the GPU (the library asks the device; a
 * cluster split it cannot place goes to stream-K or the square kernel).
 * Errors as for sptg_plan_square; SPTG_ERR_CONFIG when a forced kernel does
 * not take the shape.
 */
int sptg_plan(int64_t M, int64_t N, int64_t K, sptg_dtype dtype, int sm_count,
              const sptg_config* cfg, int* out);

/*
 * ------------------------------------------------------------------------
 * The operators around the products of a language model's layer. All are
 * asynchronous on `stream`, allocate nothing, copy nothing to the host and
 * may be captured in a CUDA graph. They keep all sums in fp32 and give the
 * same bits for the same inputs on every call. Dimensions are at most
 * 2^31 - 4096 (SPTG_ERR_ARG).
 */

/* Element types of these operators. */
typedef enum {
  SPTG_T_F16 = 0,   /* binary16 */
  SPTG_T_BF16 = 1,  /* bfloat16 */
  SPTG_T_S8 = 2,    /* int8; quantised values are -127 ... 127 */
  SPTG_T_E4M3 = 3,  /* 8-bit float, 4 exponent and 3 fraction bits, largest 448 */
  SPTG_T_F32 = 4,   /* binary32 (a router's logits, sums of gradients) */
  SPTG_T_RANGE_MIN_ = -2147483647 - 1, /* as for sptg_dtype: any int is rejected cleanly */
  SPTG_T_RANGE_MAX_ = 2147483647
} sptg_type;

/*
 * Residual addition and root-mean-square norm of each row, with the next
 * product's operand as output:
 *
 *   t = x + residual                            (fp32)
 *   h = t rounded to the rows' type             (the new residual stream)
 *   v = t * weight / sqrt(mean(t^2) + eps)      (fp32; mean over the row)
 *   y = v rounded to the rows' type             (out_type == in_type), or
 *   scale = max|v| / Q,  y = v / scale rounded to nearest even
 *                                               (out_type SPTG_T_S8, Q = 127,
 *                                                or SPTG_T_E4M3, Q = 448)
 *
 * so that y * scale stands for v. scales holds one fp32 for each row (unused,
 * may be NULL, for 16-bit outputs). A row of zeros gives y = 0, scale = 0, as
 * does one whose max|t * weight| is below about 1e-36 or whose sum of squares
 * passes the fp32 range. A row holding an infinity or a NaN gives y = 0, scale
 * = NaN.
 *
 * x, residual, h: rows x cols of in_type (SPTG_T_F16 or SPTG_T_BF16) with row
 * pitches ldx, ldr, ldh; weight: cols of in_type; y: rows x cols of out_type
 * with row pitch ldy (pitches in elements, >= cols). h may be x or residual
 * itself (same pointer and pitch); nothing else may overlap. Any cols, pitch
 * and element-aligned pointers are taken; rows are read in 16-byte pieces when
 * cols and every pitch are multiples of 8 and every pointer is 16-byte aligned
 * (an 8-bit y: 8-byte). eps > 0. rows == 0 or cols == 0: nothing is done
 * (no scales are written).
 */
int sptg_add_rms_norm(int64_t rows, int64_t cols, sptg_type in_type, sptg_type out_type,
                      const void* x, int64_t ldx, const void* residual, int64_t ldr,
                      const void* weight, float eps, void* h, int64_t ldh, void* y, int64_t ldy,
                      float* scales, void* stream);

/* sptg_add_rms_norm with the timeout_ms and inject_stall fields of a
 * configuration (the others are ignored; NULL = defaults). They concern the
 * kernel that many wide rows take, whose copies run ahead; the others wait for
 * nothing. */
int sptg_add_rms_norm_ex(int64_t rows, int64_t cols, sptg_type in_type, sptg_type out_type,
                         const void* x, int64_t ldx, const void* residual, int64_t ldr,
                         const void* weight, float eps, void* h, int64_t ldh, void* y, int64_t ldy,
                         float* scales, void* stream, const sptg_config* cfg);

/*
 * Product with 4-bit weights and group scales:
 *
 *   Y[m, n] = x_scales[m] * sum_g scales[n, g] *
 *             sum_{k in group g} X[m, k] * (code[n, k] - zeros[n, g])
 *
 *   X         M x K of x_type, row pitch ldx elements. SPTG_T_F16 or
 *             SPTG_T_BF16 (out_type must be the same; x_scales NULL), or
 *             SPTG_T_S8 or SPTG_T_E4M3 with x_scales, one fp32 for each row,
 *             as sptg_add_rms_norm writes them
 *   codes     N rows of K / 2 bytes, row pitch ldw bytes: byte j of a row holds
 *             column 2j in its low half and column 2j + 1 in its high half
 *   scales    N x (K / group) of out_type, dense
 *   zeros     N x (K / group) bytes 0 ... 15 (the low four bits count), dense;
 *             NULL: 8 everywhere
 *   Y         M x N of out_type (SPTG_T_F16 or SPTG_T_BF16), row pitch ldy
 *
 * Products are exact, a group's sum of them and the sum of the scaled groups are
 * fp32, and Y is rounded once: a weight equal to its zero point adds nothing, an
 * infinity or a NaN in X what its products are, to its own row. (A group's sum of
 * products has to stay in the fp32 range before its scale.)
 * group is 32, 64 or 128 and divides K. X and codes are 16-byte aligned with
 * row pitches of a multiple of 16 bytes (SPTG_ERR_ALIGN); N, M and ldy are
 * free. Up to 64 rows of X (with groups of 32: up to 32) share one pass over
 * the weights; more rows take as many passes as needed. M == 0 or N == 0:
 * nothing is done. K == 0: Y is zero.
 */
int sptg_gemm_w4(int64_t M, int64_t N, int64_t K, int group, sptg_type x_type, sptg_type out_type,
                 const void* X, int64_t ldx, const float* x_scales, const uint8_t* codes,
                 int64_t ldw, const void* scales, const uint8_t* zeros, void* Y, int64_t ldy,
                 void* stream);

/*
 * Products grouped by expert with ragged sizes, and their gradients. Rows
 * offsets[e] ... offsets[e + 1] - 1 of the T rows belong to expert e:
 *
 *   sptg_grouped_gemm      Y[t, n]     = sum_k X[t, k]  * W[e, n, k]
 *   sptg_grouped_gemm_dx   dX[t, k]    = sum_n dY[t, n] * W[e, n, k]
 *   sptg_grouped_gemm_dw   dW[e, n, k] = sum_t dY[t, n] * X[t, k]
 *
 * offsets: E + 1 int32 in device memory, not decreasing, 0 <= offsets[0],
 * offsets[E] <= T (read by the kernel: the host never waits for them). An
 * expert may have no rows (its dW is zero). Rows of Y and dX that belong to no
 * expert are set to zero. Offsets that break these rules are clamped to
 * [0, T], and each is raised to the largest before it; results are those of the
 * offsets that this leaves.
 *
 * X, Y, dY, dX: T rows with row pitches in elements; W and dW: E x N x K,
 * dense (N rows of K for each expert, as the weights of sptg_gemm are stored).
 * dtype: a float pair of sptg_dtype; its first type is that of X, W and dY, its
 * second that of the output. Sums are fp32; for an fp32 output they are formed
 * in parts of up to 512 terms that are added up rounded to nearest. Alignment as for sptg_gemm: 16-byte aligned
 * bases; N and K, and each pitch, a multiple of 16 bytes in the types they
 * count. E <= 1024.
 */
int sptg_grouped_gemm(int64_t E, int64_t T, int64_t N, int64_t K, sptg_dtype dtype,
                      const int32_t* offsets, const void* X, int64_t ldx, const void* W, void* Y,
                      int64_t ldy, void* stream);
int sptg_grouped_gemm_dx(int64_t E, int64_t T, int64_t N, int64_t K, sptg_dtype dtype,
                         const int32_t* offsets, const void* dY, int64_t lddy, const void* W,
                         void* dX, int64_t lddx, void* stream);
int sptg_grouped_gemm_dw(int64_t E, int64_t T, int64_t N, int64_t K, sptg_dtype dtype,
                         const int32_t* offsets, const void* dY, int64_t lddy, const void* X,
                         int64_t ldx, void* dW, void* stream);

/*
 * ------------------------------------------------------------------------
 * The operators around an expert layer: which experts a row goes to, the rows
 * sorted by expert for the grouped products, their outputs added up by row, and
 * the end of a block. As the operators above: asynchronous, no allocation, no
 * copies to the host, graph capture, the same bits on every call. Rows of
 * SPTG_T_F16 or SPTG_T_BF16 take any width, pitch and element-aligned pointer; they
 * are read in 16-byte pieces when the width and every pitch are multiples of 8
 * and every pointer is 16-byte aligned, else in words shifted together (the norms up to
 * 16376 columns, their gradients up to 8192; beyond, element by element). cols <= 2^30.
 * Outputs overlap nothing unless said.
 */

/*
 * Routing. Of each row of E logits:
 *
 *   s_e = 1 / (1 + exp(-l_e))  (sigmoid = 1)  or  exp(l_e) / sum exp(l)  (0)
 *   key_e = s_e + bias[e]                              (bias may be NULL)
 *   of `groups` groups of E / groups neighbouring experts the top_groups with the
 *   largest sums of their group_best (1 or 2) largest keys are kept, and of their
 *   experts the `top` with the largest keys, largest first
 *   w = scale * s_e                                    (renormalize = 0)
 *   w = scale * s_e / (sum of the chosen s)            (renormalize = 1)
 *
 * Keys are compared as exact arithmetic would (the kernel goes to 64 bits where
 * 32 do not settle a choice); equal ones in the order of their experts, as are
 * groups. Without a bias (or with one of zeros) that holds for scores of any size: logits
 * stand for them. With one, keys or sums of two that differ by less than 2^-42 of the
 * larger and the largest bias may count as equal. An expert whose logit or bias is
 * -infinity is never chosen: a row with fewer than `top` experts left has -1 with
 * weight 0 in its last places. A row that holds a NaN (or, with a softmax, +infinity) gets experts 0 ... top
 * - 1 with weights NaN.
 *
 * logits: rows x E of SPTG_T_F16, SPTG_T_BF16 or SPTG_T_F32, row pitch ld;
 * bias: E; weights, experts: rows x top, dense. E <= 1024, top <= 16, groups <= 32.
 *
 * The gradient: dlogits (of the logits' type, row pitch ldd, written whole) from
 * dweights (rows x top), the logits and the experts that were chosen. Experts
 * outside [0, E) add nothing; the choice and the bias have no gradient.
 */
int sptg_route_experts(int64_t rows, int64_t E, int top, sptg_type type, const void* logits, int64_t ld,
                       const float* bias, int sigmoid, int groups, int top_groups, int group_best,
                       int renormalize, float scale, float* weights, int32_t* experts, void* stream);
int sptg_route_experts_dlogits(int64_t rows, int64_t E, int top, sptg_type type, const void* logits,
                               int64_t ld, const int32_t* experts, const float* dweights, int sigmoid,
                               int renormalize, float scale, void* dlogits, int64_t ldd, void* stream);

/*
 * Dispatch: the rows * top entries (t, j), sorted by experts[t, j], entries of one
 * expert in their own order; those whose expert lies outside [0, E) come last.
 *
 *   places[t, j]            where the entry went, rows x top
 *   sorted[places[t, j]]    = x[t], rows * top rows of cols
 *   offsets[e]              the first place of expert e, E + 1 values: what
 *                           sptg_grouped_gemm takes
 *
 * rows * top <= 2^31 - 4096, E <= 1024. The gradient by x is sptg_combine_rows of
 * the sorted rows' gradient without weights.
 *
 * Combination:  out[t] = base[t] + sum_j weights[t, j] * y[places[t, j]]
 *
 * in 32 bits, rounded once. y: y_rows x cols; weights: rows x top (NULL: 1); base:
 * rows x cols, or NULL; out may be base. A place outside [0, y_rows) adds nothing.
 *
 * Its gradients:  dy[places[t, j]] = weights[t, j] * dout[t],
 *                 dweights[t, j] = <y[places[t, j]], dout[t]>
 *
 * (base's is dout). places has to name no row of y twice (one that several name gets
 * the value of one of them). A row of dy that none names is left as it was, or, in
 * sptg_combine_rows_grad_ex with zero_unnamed = 1, written with zeros. A place outside [0, y_rows)
 * has dweights 0. dweights may be NULL (then y is not read).
 */
int sptg_dispatch_rows(int64_t rows, int64_t cols, int top, int64_t E, sptg_type type, const void* x,
                       int64_t ldx, const int32_t* experts, void* sorted, int64_t lds, int32_t* places,
                       int32_t* offsets, void* stream);
int sptg_combine_rows(int64_t rows, int64_t cols, int top, int64_t y_rows, sptg_type type, const void* y,
                      int64_t ldy, const int32_t* places, const float* weights, const void* base,
                      int64_t ldb, void* out, int64_t ldo, void* stream);
int sptg_combine_rows_grad(int64_t rows, int64_t cols, int top, int64_t y_rows, sptg_type type,
                           const void* dout, int64_t ldd, const void* y, int64_t ldy, const int32_t* places,
                           const float* weights, void* dy, int64_t lddy, float* dweights, void* stream);
int sptg_combine_rows_grad_ex(int64_t rows, int64_t cols, int top, int64_t y_rows, sptg_type type,
                              const void* dout, int64_t ldd, const void* y, int64_t ldy,
                              const int32_t* places, const float* weights, void* dy, int64_t lddy,
                              float* dweights, int zero_unnamed, void* stream);

/* What a gate multiplies: nothing, a column (cols values), a row (rows values,
 * ldg apart), or an element (rows x cols, row pitch ldg). */
typedef enum {
  SPTG_GATE_NONE = 0,
  SPTG_GATE_COLS = 1,
  SPTG_GATE_ROWS = 2,
  SPTG_GATE_FULL = 3,
  SPTG_GATE_RANGE_MIN_ = -2147483647 - 1, /* as for sptg_dtype: any int is rejected cleanly */
  SPTG_GATE_RANGE_MAX_ = 2147483647
} sptg_gate;

/*
 * The end of a block: norm of its output y, gate, scaled residual, and the norm
 * before the next block.
 *
 *   u = y * block_weight / sqrt(mean(y^2) + eps)     (block_weight NULL: u = y)
 *   t = alpha * residual + gate * u                  (fp32)
 *   h = t rounded                                    (the new residual stream)
 *   v = t * weight / sqrt(mean(t^2) + eps)           rounded to the rows' type
 *
 * h may be y or residual (same pointer and pitch). A row whose sum of squares
 * passes the fp32 range is normalised to 0. The kernel goes by rows, cols and alignment, and
 * kernels multiply and add in orders of their own: the same row may differ in its last
 * bits between calls of another number of rows, pitch or alignment (not between equal calls).
 *
 * The gradients of y, residual, gate, weight and block_weight from dh and dv
 * (either may be NULL: 0). dy, dresidual and an element-wise dgate are of the rows'
 * type; dweight, dblock_weight (cols values) and dgate by column (cols) or row (rows, dense)
 * of out_type: SPTG_T_F32 or the rows' type. They are summed up in fp32 in a fixed order
 * of the rows, by way of a workspace of sptg_gate_add_rms_norm_grad_workspace
 * bytes (16-byte aligned; not shared by calls that run at the same time).
 *
 * cfg: its fields timeout_ms and inject_stall, as for sptg_add_rms_norm_ex (the
 * others are ignored; NULL = defaults).
 */
int sptg_gate_add_rms_norm(int64_t rows, int64_t cols, sptg_type type, const void* y, int64_t ldy,
                           const void* residual, int64_t ldr, const void* block_weight, const void* gate,
                           sptg_gate gate_kind, int64_t ldg, float alpha, const void* weight, float eps,
                           void* h, int64_t ldh, void* v, int64_t ldv, void* stream,
                           const sptg_config* cfg);
int64_t sptg_gate_add_rms_norm_grad_workspace(int64_t rows, int64_t cols);
int sptg_gate_add_rms_norm_grad(int64_t rows, int64_t cols, sptg_type type, const void* dh, int64_t lddh,
                                const void* dv, int64_t lddv, const void* y, int64_t ldy,
                                const void* residual, int64_t ldr, const void* block_weight,
                                const void* gate, sptg_gate gate_kind, int64_t ldg, float alpha,
                                const void* weight, float eps, void* dy, int64_t lddy, void* dresidual,
                                int64_t lddr, void* dgate, int64_t lddg, void* dweight, void* dblock_weight,
                                sptg_type out_type, void* workspace, int64_t workspace_bytes, void* stream,
                                const sptg_config* cfg);

#ifdef __cplusplus
}
#endif

#endif /* SPTGEMM_H */
