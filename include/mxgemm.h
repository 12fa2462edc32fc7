/*
 * mxgemm.h -- C ABI of libmxgemm.so: block-scaled (MX) quantized GEMM, fp16 GEMM, int8/int4
 * dequant matvec, the MX/int codecs, and the decode step's rotary positions, paged key-value cache
 * and attention, for AMD Instinct MI355X (gfx950).
 *
 * Conventions shared by every entry point
 *  - Every function returns an mx_status; 0 is success. Arguments are validated before any work
 *    is queued, and nothing is written when validation fails.
 *  - Device pointers are owned by the caller (allocated with hipMalloc or by a framework); the
 *    library never allocates, frees or retains them. Host pointers likewise.
 *  - `stream` is a hipStream_t passed as an opaque pointer (NULL = the default stream). GPU entry
 *    points only enqueue work on that stream and return; they never synchronise. Calls on
 *    different streams may run concurrently.
 *  - Debugging: with the environment variable MX_SYNC_CHECK set (to anything but "0"; read at
 *    every call), a GPU entry point that queued work waits for its stream before returning and
 *    returns MX_ERR_LAUNCH when the stream reports an error, so an asynchronous fault is reported
 *    by the call that caused it.
 *  - Device pointers must be 16-byte aligned. Matrices are dense and row-major with the leading
 *    dimension equal to the row length given below.
 *  - A GPU entry point called on a device that is not gfx950 returns MX_ERR_ARCH.
 *
 * Formats (the pages name the types, the OCP Microscaling v1.0 formats give their bits):
 *  - MX_E4M3: FP8 E4M3 "FN" (bias 7, S.1111.111 = NaN, no Inf, max 448), one byte per element.
 *  - MX_E5M2: FP8 E5M2 (bias 15, S.11111.00 = Inf, S.11111.xx = NaN, max 57344), one byte per
 *    element (the pages' fp8 / "MX scaling formats", TensorOps notes, quantized dtype matrix).
 *  - MX_E2M3 / MX_E3M2: FP6 (bias 1, max 7.5 / bias 3, max 28; no Inf or NaN), four elements per
 *    three bytes: element j in bits 6j..6j+5 of the row read as a little-endian bit stream.
 *  - MX_E2M1: FP4 E2M1 (bias 1, +-{0,.5,1,1.5,2,3,4,6}), two elements per byte, the element with
 *    the even index in the low nibble.
 *  - Scales of MX operands: E8M0 bytes, value 2^(e-127), 0xFF = NaN; one scale per 32
 *    consecutive elements along K ("Scale planes: one MTLTensor = data + scales" and the
 *    auxiliary-plane blockFactors {32,1} of the WWDC26 session 330 summary).
 *  - MX_BF16: bfloat16, and MX_F32: binary32 (not for the block-scaled GEMM, matvec and codecs).
 *  - MX_F16: IEEE binary16. MX_INT8: two's-complement bytes. MX_INT4: two's-complement nibbles,
 *    packed two per byte along the C-order linear index, the even index in the low nibble
 *    ("TensorOps ... notes", section "VALIDATED ON M4 MAX", fact 5).
 */
#ifndef MXGEMM_H
#define MXGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MX_OK = 0,
  MX_ERR_NULL = -1,    /* a required pointer is NULL */
  MX_ERR_SHAPE = -2,   /* a dimension is out of range or violates a divisibility rule */
  MX_ERR_ALIGN = -3,   /* a device pointer is not 16-byte aligned */
  MX_ERR_FORMAT = -4,  /* unsupported format or format pair */
  MX_ERR_ARCH = -5,    /* the current device is not gfx950, or no device is present */
  MX_ERR_LAUNCH = -6,  /* the HIP runtime reported an error when queueing a kernel (or, with
                          MX_SYNC_CHECK, when the stream ran it) */
  MX_ERR_NOMEM = -7,   /* host allocation of a plan failed, or a page pool has no page left */
  MX_ERR_SCRATCH = -8  /* mxmatvec_run_noalloc: the shape needs more than MXMATVEC_SCRATCH_BYTES */
} mx_status;

/* MX_E8M0 names the scale format; it is accepted only by mx_decode_host. */
typedef enum { MX_E4M3 = 0, MX_E5M2 = 1, MX_E2M3 = 2, MX_E3M2 = 3, MX_E2M1 = 4, MX_E8M0 = 8, MX_F16 = 16, MX_BF16 = 17, MX_F32 = 18, MX_INT8 = 32, MX_INT4 = 33 } mx_format;

/* Largest accepted dimension of any matrix (rows or columns). */
#define MX_MAX_DIM (1 << 20)

/* Human-readable name of a status code (static storage, never NULL; unknown codes are named as
 * such). */
const char* mx_strerror(mx_status status);

/* Library version as 10000*major + 100*minor + patch. */
int mx_version(void);

/* ------------------------------------------------------------------------------------------ */
/* GEMM plans.                                                                                  */
/* ------------------------------------------------------------------------------------------ */

typedef struct mxgemm_plan* mxgemm_t;

/* mxgemm_create flag: epilogue ReLU, C = max(A*B, 0) elementwise before the fp16 store, with
 * IEEE maxNum semantics (a NaN product gives 0). This is the postfix activation of the "Running
 * inline ML operations in a shader with Metal 4" sample, section "Combine an element-wise
 * function" (there applied with max(value, 0) to the product tile in registers). */
#define MXGEMM_RELU 1u

/* mxgemm_create flag: the A operand is given unquantised, as binary16 [M][K] (row-major), and is
 * quantised to E4M3 with E8M0 scales per 32 along K inside the GEMM, as the kernel loads its tiles,
 * with exactly the codes and scales mx_pack_run(MX_E4M3) gives for the same values (held in fp32):
 * C equals the product of mx_pack_run's A with B. This is the quantise-on-load of prefill
 * activations, which the pages' quantized matmul takes already quantized ("TensorOps ... notes",
 * section "Why this matters here": prefill is the compute-bound stage; scale rule of mx_pack_run).
 * Needs fa == fb == MX_E4M3 (else MX_ERR_FORMAT), K % 1024 == 0 and N % 4 == 0 (else MX_ERR_SHAPE);
 * mxgemm_run then takes SA = NULL (ignored). */
#define MXGEMM_QUANT_A 2u

/*
 * mxgemm_create -- validate a GEMM problem C[M,N] = A[M,K] * B[K,N] and choose its kernel.
 *
 * Operation ("TensorOps ... notes", sections "Scale planes" and "Kernel-phase findings"; WWDC26
 * session 330 summary, sections on the MXFP8 tensor type and the quantized matmul2d):
 *   C[m,n] = sum_k (dec(A[m,k]) * 2^(SA[m,k/32]-127)) * (dec(B[k,n]) * 2^(SB[n,k/32]-127)),
 * accumulated in fp32 and written once as fp16 (rounded to nearest even). C is overwritten
 * (C = A*B, not C += A*B). For fa == fb == MX_F16 there are no scales: C = A*B in fp32, fp16 out.
 *
 * Supported pairs: (MX_E4M3, MX_E4M3), (MX_E2M1, MX_E2M1), (MX_F16, MX_F16), and the mixed MX pairs
 * (MX_E4M3, MX_E2M1), (MX_E2M1, MX_E4M3) (A and B each in its own format, scales as above; the
 * scaled MFMA takes each operand's format separately), and every pair with an MX_E5M2 operand:
 * (MX_E5M2, MX_E5M2), (MX_E4M3, MX_E5M2), (MX_E5M2, MX_E4M3), (MX_E5M2, MX_E2M1),
 * (MX_E2M1, MX_E5M2), and the four FP6 pairs (MX_E2M3, MX_E2M3), (MX_E3M2, MX_E3M2),
 * (MX_E2M3, MX_E3M2), (MX_E3M2, MX_E2M3) (the pages' "MX scaling formats", TensorOps notes,
 * quantized dtype matrix). All pairs other than the three plain ones need K % 512 == 0 and
 * N % 4 == 0, else MX_ERR_SHAPE; FP6 with any other format is MX_ERR_FORMAT.
 * Shape rules: 1 <= M, N <= MX_MAX_DIM; 32 <= K <= MX_MAX_DIM; MX formats need K % 32 == 0;
 * MX_F16 needs K % 8 == 0 and N % 8 == 0.
 * `flags` is 0 or a combination of MXGEMM_RELU and MXGEMM_QUANT_A (other bits: MX_ERR_FORMAT).
 * Host only: queues no GPU work. *out
 * receives a plan that holds host metadata only; release it with mxgemm_destroy. A plan may be
 * used from several threads and streams at once.
 */
int mxgemm_create(mxgemm_t* out, int M, int N, int K, int fa, int fb, unsigned flags);

/*
 * mxgemm_run -- queue the GEMM of plan p on `stream`.
 *
 * Layouts (all device pointers, 16-byte aligned):
 *   MX:  A  codes [M][K] (E4M3, E5M2), [M][3K/4] (E2M3, E3M2: 6-bit fields, little-endian bit
 *           stream) or [M][K/2] (E2M1), K contiguous;
 *        SA E8M0 [M][K/32];
 *        B  codes stored K-contiguous, i.e. [N][K], [N][3K/4] or [N][K/2] by format: the scaled
 *           right operand is the transposed one ("Kernel-phase findings", fact 2);
 *        SB E8M0 [N][K/32];
 *   F16: A binary16 [M][K]; B binary16 [K][N] (row-major K x N); SA = SB = NULL.
 *   C:   binary16 [M][N].
 * Errors: MX_ERR_NULL (p, A, B, C, or a scale pointer of an MX plan), MX_ERR_ALIGN, MX_ERR_ARCH,
 * MX_ERR_LAUNCH. Non-finite inputs propagate: a NaN code or a 0xFF scale makes every output it
 * contributes to NaN. E5M2 Inf codes (S.11111.00) are infinities and follow IEEE arithmetic: an
 * output with one infinite term is that infinity, +Inf and -Inf terms together give NaN, and an
 * infinity times a zero element gives NaN (the products are formed exactly and summed in fp32).
 */
int mxgemm_run(mxgemm_t p, const void* A, const void* SA, const void* B, const void* SB, void* C,
               void* stream);

/* mxgemm_destroy -- release a plan (NULL is accepted and ignored). */
int mxgemm_destroy(mxgemm_t p);

/* Kernel chosen by a plan (for reports): output tile rows and columns, K elements per pipeline
 * stage, and the kernel variant (0: 4 waves, 1: 8 waves, 2: 8-wave ping-pong schedule, 3: 4-stage
 * LDS ring of 64-byte K stages, for MX formats with N % 4 == 0 and K % 512 == 0 (E4M3) or
 * K % 1024 == 0 (E2M1), and for fp16 with N % 256 == 0, K % 256 == 0 on 256x256 tiles; 4: 8-wave
 * ping-pong ring of 128-byte stage rows (FP6: 96) on 256x256 tiles, for every MX pair where
 * K % 1024 == 0 and N % 4 == 0 (the E2M1 operand of a mix with a byte format staged four K-steps
 * at a time), for fp16 where K % 512 == 0 and N % 8 == 0, and for MXGEMM_QUANT_A). The environment
 * variable MXGEMM_TILE (a tile id 0..11; 8, 9 and 10 are the 4-stage ring with 256x256, 256x224
 * and 256x192 tiles where it applies, else an 8-wave kernel: 256x256 for 8 and 10, 256x224 for 9;
 * 11 is the ping-pong ring where it applies, else as 8), read at mxgemm_create, overrides the
 * choice. */
int mxgemm_plan_info(mxgemm_t p, int* tile_m, int* tile_n, int* tile_k, int* variant);

/* ------------------------------------------------------------------------------------------ */
/* Dequant matvec for decode.                                                                   */
/* ------------------------------------------------------------------------------------------ */

/*
 * mxmatvec_run -- y[m,n] = sum_b Ws[b,n] * sum_{k=32b}^{32b+31} x[m,k] * q[k,n], accumulated in
 * fp32, y written as fp16. This is the per-32-row block form with arbitrary fp16 scales
 * ("TensorOps ... notes", section "Kernel-phase findings", revised kernel strategy; int4 packing
 * from section "VALIDATED ON M4 MAX", fact 5).
 *
 *   x  binary16 [M][K]      W int8 [K][N]  (fw = MX_INT8)  or packed int4 [K][N/2] (fw = MX_INT4)
 *   Ws binary16 [K/32][N]   y binary16 [M][N]
 * Shape rules: 1 <= M <= 256; K % 32 == 0, 32 <= K <= MX_MAX_DIM; 1 <= N <= MX_MAX_DIM;
 * N % 16 == 0 (int8) or N % 32 == 0 (int4). Device pointers, 16-byte aligned.
 * M <= 8 is the decode matvec; 9 <= M <= 256 (the W8A16 / W4A16 prefill-like GEMM with the same
 * arbitrary fp16 block scales, TensorOps notes, section "Kernel-phase findings") runs a small-M
 * GEMM kernel: each block product is still formed exactly in fp32 and scaled once by its fp16
 * block scale.
 *
 * Workspace (an addition to the call the pages' operation needs: workspace = NULL gives exactly
 * that call). The fastest kernels split K across workgroups: their fp32 partial sums and one counter
 * per column strip (M <= 8) or per tile (M > 8) live in a caller-owned device buffer of
 * mxmatvec_workspace_size() bytes (16-byte aligned). For M <= 8 that is every shape with at least
 * 8 blocks of K. For M > 8 it is the shapes whose unsplit grid is small (fewer than 128 tiles of 32
 * rows by 128 columns and K >= 512: K is split), and the shapes that run more than 256 tiles of 64
 * rows by 128 columns but fill less than 90% of their rounds of 256 workgroups (such as M=256,
 * N=12288: the tiles' 32-row blocks are dealt out in equal runs to 256 workgroups, and the runs
 * that share a tile add their partials). mxmatvec_workspace_size returns 0 for the other shapes,
 * which never touch the buffer.
 *  - The buffer must be zero-filled once before its first use (hipMemset, or any zeroed
 *    allocation). Every call leaves its counters at zero again, so the buffer stays valid for any
 *    later call whose requirement it meets.
 *  - The library cannot check the contents. A buffer whose counter region is not zero, or one that
 *    two calls use at the same time (calls on different streams, or a graph replay that overlaps an
 *    eager call), makes the wrong workgroup of a column strip (or none) add the partial sums: that
 *    strip of y is then wrong or left unwritten, and later calls on the same buffer inherit the
 *    stale counter. Zero the counter region again to recover. Calls that may overlap in time need
 *    separate workspaces.
 *  - The last workgroup of each strip (or tile) adds the partial sums in a fixed order, so results
 *    are deterministic.
 *  - With workspace == NULL, or workspace_bytes below the requirement, K is not split across
 *    workgroups and the buffer is not touched (same results up to fp32 summation order; slower
 *    when N is small compared with the number of compute units).
 */
int mxmatvec_run(int M, int N, int K, const void* x, const void* W, int fw, const void* Ws, void* y,
                 void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes mxmatvec_run uses for this shape (0: none needed, or an invalid shape). For
 * 1 <= M <= 8 the requirement never decreases as M grows for fixed N, K and fw; for M > 8 it can
 * (a larger M has more tiles and so fewer K splits). */
size_t mxmatvec_workspace_size(int M, int N, int K, int fw);

/* Size of the library's static scratch array (17 MiB), the most workspace mxmatvec_run_noalloc can
 * use. Every valid shape fits: the requirement is 16 KiB of counters, then fp32 partials of at most
 * 16 MiB (M <= 8: at most 16 splits x 8 rows x 128 strips of 256 columns; M > 8: at most 256 splits
 * x tiles of 32 x 128, 4 MiB, or two 64 x 128 tiles for each of at most 256 workgroups, 16 MiB). */
#define MXMATVEC_SCRATCH_BYTES ((size_t)17 << 20)

/*
 * mxmatvec_run_noalloc -- mxmatvec_run for callers that cannot allocate (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same operation, arguments,
 * shape rules and kernels as mxmatvec_run with a large enough workspace, and the same results bit
 * for bit, but the split kernel's workspace is a static device array inside the library
 * (MXMATVEC_SCRATCH_BYTES per GPU, held until the process ends). Nothing is allocated, by the
 * library or any library it calls.
 *  - A shape whose workspace requirement (mxmatvec_workspace_size) exceeded MXMATVEC_SCRATCH_BYTES
 *    would return MX_ERR_SCRATCH before anything is queued; no valid shape does (see above).
 *  - All calls on one GPU share that GPU's array, which keeps the last call's contents (its
 *    counters are back at zero after every call). Calls that overlap in time on one GPU (different
 *    streams, or a captured graph replaying beside another call) race on it and give wrong results:
 *    serialise them, or use mxmatvec_run with separate workspaces.
 *  - The first call on a GPU looks up the array's device address and queues a small kernel that
 *    zeroes the counters on `stream` ahead of its own work.
 */
int mxmatvec_run_noalloc(int M, int N, int K, const void* x, const void* W, int fw, const void* Ws, void* y,
                         void* stream);

/* ------------------------------------------------------------------------------------------ */
/* Codecs on the GPU (bit-exact with the host codecs below).                                    */
/* ------------------------------------------------------------------------------------------ */

/*
 * mx_pack_run -- quantise fp32 src [rows][cols] on the GPU. The pages start from tensors already
 * held in a quantized data type with an E8M0 scale plane (WWDC26 session 330 summary, the
 * multi-plane tensor of data and scale factors, blockFactors {32,1}); the scale rules below are the
 * synthetic workloads' ("floor(log2(absmax)) - emax + 127" per 32-element block along K; symmetric
 * int8 with scale = absmax/127 per 32-row group, and an int4 variant of it).
 *  f = MX_E4M3 / MX_E5M2 / MX_E2M3 / MX_E3M2 / MX_E2M1: blocks of 32 along cols. Per block:
 *      amax = max|x|; E = clamp(floor(log2 amax) - emax + 127, 0, 254) with emax = 8 (E4M3),
 *      15 (E5M2), 2 (E2M3), 4 (E3M2) or 2 (E2M1), the exponent of the format's largest element
 *      (amax = 0 gives E = 0); codes = x * 2^(127-E) rounded to the nearest element value, ties to
 *      the even code, saturated to +-448 / +-57344 / +-7.5 / +-28 / +-6, sign kept (negative
 *      values that round to zero give -0). A block holding Inf or NaN gets E = 0xFF and zero
 *      codes. codes: [rows][cols] (E4M3, E5M2), [rows][3*cols/4] (E2M3, E3M2: element j in bits
 *      6j..6j+5 of the row as a little-endian bit stream) or [rows][cols/2] (E2M1); scales: E8M0
 *      [rows][cols/32]. cols % 32 == 0.
 *  f = MX_INT8 / MX_INT4: src is a weight W [K=rows][N=cols], blocks of 32 along rows. Per
 *      column and block: s = fp16(amax / qmax) (fp32 division, nearest-even to fp16) with
 *      qmax = 127 or 7; q = clamp(round_half_even(fp32(w / s)), -qmax, qmax), q = 0 where
 *      s = 0. A block holding Inf or NaN gets s = NaN (0x7E00) and q = 0. codes: int8
 *      [rows][cols] or packed int4 [rows][cols/2] (TensorOps notes, "VALIDATED ON M4 MAX",
 *      fact 5); scales: binary16 [rows/32][cols]. rows % 32 == 0; cols % 2 == 0 for MX_INT4.
 * Errors: MX_ERR_NULL, MX_ERR_SHAPE, MX_ERR_FORMAT (f not listed), MX_ERR_ALIGN, MX_ERR_ARCH,
 * MX_ERR_LAUNCH; nothing is queued on an error.
 */
int mx_pack_run(int f, const float* src, int rows, int cols, void* codes, void* scales, void* stream);

/*
 * mx_unpack_run -- dequantise to fp32 on the GPU: out = fp32(value * scale), the exact product
 * rounded once to fp32 (nearest even; subnormals kept; overflow gives +-Inf; NaN propagates). This
 * is the dequantisation the pages' matmul applies to each element in the kernel (TensorOps notes,
 * "Scale planes": value times its block's power-of-two scale; "Kernel-phase findings": int weights
 * times their fp16 block scale), written out as its own result. Layouts as in mx_pack_run (MX:
 * scales along cols; INT8/INT4: scales along rows). Errors as for mx_pack_run.
 */
int mx_unpack_run(int f, const void* codes, const void* scales, int rows, int cols, float* out,
                  void* stream);

/* ------------------------------------------------------------------------------------------ */
/* Host codecs (CPU, synchronous, same definitions and layouts as the GPU codecs).              */
/* ------------------------------------------------------------------------------------------ */

int mx_pack_host(int f, const float* src, int64_t rows, int64_t cols, void* codes, void* scales);
int mx_unpack_host(int f, const void* codes, const void* scales, int64_t rows, int64_t cols, float* out);

/* Single-element encoder/decoder of the host codec. mx_encode_host: f = MX_E4M3, MX_E5M2,
 * MX_E2M3, MX_E3M2 or MX_E2M1, nearest code, ties to even, saturating, sign kept (0 for other f).
 * mx_decode_host: f = MX_E4M3, MX_E5M2, MX_E2M3 / MX_E3M2 (low 6 bits), MX_E2M1 (low nibble),
 * MX_E8M0, MX_INT8 or MX_INT4 (low nibble); NaN for other f. */
uint8_t mx_encode_host(int f, float v);
float mx_decode_host(int f, uint8_t code);

/* ------------------------------------------------------------------------------------------ */
/* 8-bit activations: the norm before them, the product of 8-bit integers.                      */
/* ------------------------------------------------------------------------------------------ */

/* A matrix of rows with their elements contiguous, one every `stride` elements, each row 16-byte aligned. */
typedef struct {
  void* data;
  int64_t stride;
} mx_rows;

/*
 * mxnorm_run -- root-mean-square norm of rows, with the residual's addition before it:
 *   h = x + residual, rounded to f (residual NULL: h = x);  y_i = h_i weight_i / sqrt(mean_j h_j^2 + eps).
 *  - f: MX_F16, MX_BF16 or MX_F32 (x, residual, total, weight). total (NULL: not wanted; needs a residual) receives h and may be
 *    x or residual itself. weight: [dim] (NULL: ones).
 *  - fmt: what y is written as. f: y rounded, scales unused. MX_INT8: out bytes q = rint(127 y / max|y|) of the row, ties to
 *    even, and scales, fp32 [rows], max|y| / 127, for mxgemm_i8_run; a row of zeros has scale 0, a row with an infinity
 *    or NaN scale NaN and zeros. MX_E4M3 and MX_E5M2 (dim % 32 == 0): the codes and E8M0 scales, [rows][dim / 32], that mx_pack_run's rule
 *    gives y, the scale that of y before its rounding to fp32 (within 2^-40 below a power of two, y counts as that power), for mxgemm_run
 *    (which wants out->stride == dim).
 *  - Squares are summed (for blocks in 64 bits) and y is formed in fp32, and rounded once. Rows whose squares pass fp32's range (or vanish in it) are
 *    scaled by a power of two first, and a product with the weight that does is formed otherwise, so every finite row has its norm, whatever
 *    finite weights it has. (A row of zeros with eps 0 has none: its y is NaN.)
 * 1 <= dim <= MX_MAX_DIM, 0 <= rows <= MX_MAX_DIM (0: nothing is done); strides at least dim, in multiples of 16 bytes; eps finite and
 * not negative. Besides total, outputs must not overlap inputs. Elements between dim and the stride are neither
 * read nor written.
 */
int mxnorm_run(int f, int rows, int dim, const mx_rows* x, const mx_rows* residual, const mx_rows* total, const void* weight, float eps,
               int fmt, const mx_rows* out, void* scales, void* stream);

/* mxquant_rows_run -- the same outputs of x as it is, without a norm: activations that no norm precedes, or a weight
 * [N][K] by output channel. fmt: MX_INT8, MX_E4M3 or MX_E5M2. */
int mxquant_rows_run(int f, int rows, int dim, const mx_rows* x, int fmt, const mx_rows* out, void* scales, void* stream);

/* Largest K of mxgemm_i8_run: sums of K products of 8-bit integers fit 32 bits. */
#define MXGEMM_I8_MAX_K 131071

/*
 * mxgemm_i8_run -- C[m,n] = SA[m] SB[n] sum_k A[m,k] B[n,k] (+ bias[n]): the product of 8-bit integers with one scale per
 * row of A (token) and one per row of B (output channel).
 *   A int8 [M][K], SA fp32 [M]; B int8 [N][K] (K contiguous, as the block-scaled GEMM's), SB fp32 [N]; C [M][N] in fc, MX_F16, MX_BF16 or
 *   MX_F32; bias [N] in fc (NULL: none); flags: 0 or MXGEMM_RELU (C = max(C, 0), after the bias).
 * The sum is exact; it and the scales' product are rounded to fp32, their product with the bias added once more, and the result is
 * rounded to fc (ReLU makes NaN 0, as mxgemm_run's). Results are the same bits for every workspace.
 * 0 <= M <= MX_MAX_DIM (0: nothing is done), 1 <= N <= MX_MAX_DIM, 1 <= K <= MXGEMM_I8_MAX_K, all odd ones among them. Strides: A's and B's at least K and
 * multiples of 16, at most MX_MAX_DIM; C's at least N (rows of C that are not 16-byte aligned are written by
 * elements). Every row of A and B, the last one too, is read up to the next multiple of 16 bytes past K; what stands there does
 * not matter.
 * Workspace as for mxmatvec_run, of mxgemm_i8_workspace_size() bytes, zero-filled before its first use and left reusable by every
 * call, of this or other shapes: where there are few tiles, workgroups split K and their sums meet there. Calls that may overlap in time need separate
 * workspaces, and so do calls of another kind (mxmatvec_run, attention), which keep their counters at other places. Without one, or with too small a one, K is
 * not split.
 */
int mxgemm_i8_run(int M, int N, int K, const mx_rows* A, const float* SA, const mx_rows* B, const float* SB, const void* bias, int fc,
                  const mx_rows* C, unsigned flags, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes mxgemm_i8_run uses for these sizes (0: none needed, or invalid sizes). */
size_t mxgemm_i8_workspace_size(int M, int N, int K);

/* ------------------------------------------------------------------------------------------ */
/* The decode step's cache: rotary positions, a paged key-value cache, attention over it.       */
/* ------------------------------------------------------------------------------------------ */

/* A tensor [tokens][heads][dim] with dim contiguous; strides in elements, each a multiple of 8 (of 4
 * for MX_F32), so that every row is 16-byte aligned. */
typedef struct {
  void* data;
  int heads;
  int64_t token_stride, head_stride;
} mx_heads;

/* Which elements of a head form a rotated pair: i and i + rot_dim/2, or 2i and 2i + 1. */
typedef enum { MXROPE_HALF = 0, MXROPE_PAIRS = 1 } mxrope_layout;

/* A rotation: the first rot_dim elements of every head (even, 2 <= rot_dim <= dim); freq holds
 * rot_dim/2 doubles on the device, pair i turning by freq[i] radians per position; cos and sin are
 * multiplied by factor (1 for a plain rotation). */
typedef struct {
  int rot_dim, layout;
  const double* freq;
  float factor;
} mxrope;

/* Frequency rules of mxrope_freqs_host: with f_i = base^(-2i / rot_dim),
 *  MXROPE_PLAIN   f_i;
 *  MXROPE_LINEAR  f_i / params[0] (positions interpolated);
 *  MXROPE_NTK     f_i with base * params[0]^(rot_dim / (rot_dim - 2)) (rot_dim = 2: the base as it is);
 *  MXROPE_BANDS   params {s, trained length L, low, high}: blended by turns t_i = L f_i / 2 pi with
 *                 k = clamp((t_i - low) / (high - low), 0, 1): (1 - k) f_i / s + k f_i;
 *  MXROPE_YARN    params {s, L, fast, slow}: r_i = clamp((i - a) / max(c - a, 0.001), 0, 1) with a and c
 *                 the pair indexes that make `fast` and `slow` turns over L, rounded down and up and
 *                 cut to 0 and rot_dim - 1: r f_i / s + (1 - r) f_i, and factor 0.1 ln(s) + 1 (1 for s <= 1). */
typedef enum { MXROPE_PLAIN = 0, MXROPE_LINEAR = 1, MXROPE_NTK = 2, MXROPE_BANDS = 3, MXROPE_YARN = 4 } mxrope_rule;

/* mxrope_freqs_host -- freq[rot_dim/2] (host memory) and *factor of a frequency rule. params: the
 * rule's parameters (NULL for MXROPE_PLAIN). MX_ERR_SHAPE: rot_dim odd, below 2 or above 256, or
 * base, s, L or (high - low) not positive (base and fast, slow: above 1 and 0). Errors write
 * nothing. */
int mxrope_freqs_host(int rot_dim, double base, int rule, const double* params, double* freq, float* factor);

/*
 * mxrope_run -- out[t,h] = x[t,h] with each pair (a, b) of its first rot_dim elements turned by the
 * angle w = positions[t] * freq[i]:  (a cos w - b sin w, b cos w + a sin w) * factor; the other
 * elements are copied. inverse != 0 turns by -w: the gradient of the rotation with respect to x,
 * applied to the output's gradient. f: MX_F16, MX_BF16 or MX_F32 (x and out). Angles are reduced
 * in 64 bits (far positions keep their phase), the products are formed in fp32 and rounded once.
 * x->heads == out->heads; 8 <= dim <= 256, dim % 8 == 0; 0 <= tokens <= MX_MAX_DIM (0: nothing is
 * done), 1 <= heads <= 65536, and fewer than 2^24 workgroups (MX_ERR_SHAPE; only where rot_dim / 2 is not a multiple
 * of 16 bytes of elements and x has more than 200 GB); positions: int32 [tokens], of any sign. out may be x itself (same data and strides);
 * otherwise the two must not overlap, and no two rows of out may.
 */
int mxrope_run(int f, const mxrope* rope, int tokens, int dim, const mx_heads* x, const mx_heads* out,
               const int32_t* positions, int inverse, void* stream);

/* Order of a page's elements: [heads][page_size][dim] or [page_size][heads][dim]. */
typedef enum { MXKV_HEADS_FIRST = 0, MXKV_SLOTS_FIRST = 1 } mxkv_order;

/*
 * A paged key-value cache (one layer's). k and v hold `pages` pages of page_size slots each, one
 * page every page_stride elements, in `fmt`: MX_F16, MX_BF16, or MX_E4M3 codes with E8M0 scales per
 * 32 elements of dim in ks and vs, where element e of k has its scale at ks[e / 32]. Keys and values
 * may share one allocation (k at its start, v one page further, page_stride of two pages).
 * Rules (MX_ERR_SHAPE): 8 <= dim <= 256 with dim % 8 == 0 (MX_E4M3: dim % 32 == 0);
 * 1 <= heads <= 1024; 1 <= page_size <= MX_MAX_DIM; pages >= 1; pages * page_size < 2^31;
 * page_stride >= heads * page_size * dim and a multiple of 8 (MX_E4M3: of 32).
 */
typedef struct {
  int fmt, order, pages, page_size, heads, dim;
  int64_t page_stride;
  void *k, *v, *ks, *vs;
} mxkv_cache;

/* Page tables on the device: int32 [seqs][cols]; row s, column c is the page of sequence s's positions
 * c * page_size .. c * page_size + page_size - 1. An entry outside 0 .. pages - 1 is no page: nothing
 * is written to it, and attention leaves its positions out. */
typedef struct {
  const int32_t* pages;
  int seqs, cols;
} mxkv_table;

/*
 * mxkv_append_run -- write `tokens` new keys and values into the cache, in one launch with the
 * rotation of the keys and of the step's queries. Token t belongs to sequence seq[t] (NULL: t) and
 * goes to the slot of positions[t] in that sequence's table row. f: MX_F16 or MX_BF16 (k, v, q,
 * q_out); the cache's format is f or MX_E4M3.
 *  - rope != NULL: keys are turned as by mxrope_run (and rounded to f) before they are written.
 *  - MX_E4M3: every 32 elements are quantised by the rule of mx_pack_run, with the same codes and scales.
 *  - q, q_out != NULL (both or neither; rope needed): q_out = q turned, as by mxrope_run; q_out may be
 *    q itself. A token without a slot still has its q turned.
 *  - A token whose sequence, position or page is out of range is not written. Two tokens of one call
 *    must not share a slot.
 * tokens: 0 .. MX_MAX_DIM, and fewer than 2^24 workgroups. MX_ERR_SHAPE: head counts that disagree with the cache, bad strides.
 */
int mxkv_append_run(const mxkv_cache* cache, int f, int tokens, const mx_heads* k, const mx_heads* v,
                    const int32_t* positions, const int32_t* seq, const mxkv_table* table, const mxrope* rope,
                    const mx_heads* q, const mx_heads* q_out, void* stream);

/* What mxattn_decode_run computes besides the plain softmax. scale: factor of q.k (usually
 * dim^-1/2). softcap: c > 0 replaces a score s by c tanh(s / c); 0: off. window: w > 0 leaves only the
 * last w positions; 0: off. */
typedef struct {
  float scale, softcap;
  int window;
} mxattn_opts;

/*
 * mxattn_decode_run -- attention of one new token per sequence over its paged cache:
 *   s_j = scale * q[b,h] . k_j,  out[b,h] = sum_j e^{s_j} v_j / sum_j e^{s_j},  lse[b,h] = ln sum_j e^{s_j}
 * over the positions j of sequence b with starts[b] <= j < lengths[b] (starts NULL: 0), within the
 * window, whose page exists. Head h of q reads head h / (q->heads / cache->heads) of the cache.
 *  - f: MX_F16 or MX_BF16 (q, out); the cache's format is f or MX_E4M3. q, out: [seqs][q heads][dim].
 *  - A row with no position (an empty sequence, say) gives out = 0 and lse = -inf. lse, fp32
 *    [seqs][q heads], may be NULL.
 *  - Positions outside the range are never used, whatever their slots hold (NaN included). lengths
 *    above max_len, or above cols * page_size, are taken as that bound; negative ones as 0.
 *  - Scores, statistics and sums are fp32; a probability goes to the matrix cores as two 16-bit values,
 *    which hold 21 bits of it for MX_F16 and 15 for MX_BF16. E4M3 elements are scaled into f's format (exact
 *    in bfloat16; in binary16 where the value is in its range, as every value that mxkv_append_run wrote
 *    from binary16 is).
 * Workspace, as for mxmatvec_run: the rows' keys are shared evenly among workgroups, and where a share
 * cuts a row, partial results and counters live in a caller-owned device buffer of
 * mxattn_decode_workspace_size() bytes, zero-filled before its first use and left reusable by every
 * call, of this or other shapes. Calls that may overlap in time need separate workspaces, and so do calls other than attention (mxmatvec_run,
 * mxgemm_i8_run), which keep their counters at other places. Without one, or with too small a one, a
 * row is not cut (same results up to fp32 summation order; slow for long rows). The
 * partials are joined in a fixed order: results are deterministic.
 * Rules (MX_ERR_SHAPE): q->heads a multiple of the cache's heads, out->heads == q->heads;
 * seqs * q->heads < 2^24; 1 <= max_len < 2^30; scale finite, softcap and window not negative. table->seqs is the batch
 * (0: nothing is done).
 */
int mxattn_decode_run(const mxkv_cache* cache, int f, const mx_heads* q, const mx_heads* out, float* lse,
                      const mxkv_table* table, const int32_t* lengths, const int32_t* starts, int max_len,
                      const mxattn_opts* opts, void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes mxattn_decode_run uses for these sizes (0: none needed, or invalid arguments); only
 * the geometry of `cache` is read. */
size_t mxattn_decode_workspace_size(const mxkv_cache* cache, int seqs, int q_heads, int max_len, int window);

/* Rows of a batch whose first positions are the same (a common prompt): group g is the sequences first[g] .. first[g + 1] - 1, which
 * share their positions below shared[g]. first: int32 [count + 1], not falling, and shared: int32 [count], on the device;
 * sequences before first[0] and from first[count] on share nothing. max_shared bounds shared (larger ones are taken as it). */
typedef struct {
  const int32_t *first, *shared;
  int count, max_shared;
} mxattn_groups;

/*
 * mxattn_prefix_run -- mxattn_decode_run for a batch whose rows share long beginnings: the same results, but a group's shared keys
 * and values are read once for all of its rows, through the table row of its first sequence that has positions. Each row's table still names all of
 * its pages, as after mxkv_pool_fork; lengths count all positions, the shared ones among them.
 *  - What is shared is cut to the group's shortest row that has positions, and to whole tiles of 64; a row's other positions are read through
 *    its own table row. A group with one row that has positions shares nothing.
 *  - There is no window (opts->window: 0) and there are no starts. Other rules, and the treatment of missing pages, empty rows and lse, are
 *    mxattn_decode_run's; 0 <= count <= 1024, max_shared >= 0 (MX_ERR_SHAPE).
 *  - Results are the same up to fp32 summation order and the probabilities' rounding, which hold 21 bits in binary16 and 15 in bfloat16 in both calls.
 * Workspace as for mxattn_decode_run, of mxattn_prefix_workspace_size() bytes (the buffers of the two are interchangeable where large enough). Without
 * one, or with too small a one, nothing is shared: every row is read by itself. So it is where max_len, max_shared and the numbers of rows and groups leave less
 * than some 64 MB that need not be read again, as a pass of its own would take longer; the results are those of mxattn_decode_run then. How few rows a group has
 * is not weighed: groups of two over a 16-bit cache, and of up to four over E4M3, take up to twice as long as with mxattn_decode_run, and so do short rows
 * under bounds far above them.
 */
int mxattn_prefix_run(const mxkv_cache* cache, int f, const mx_heads* q, const mx_heads* out, float* lse, const mxkv_table* table,
                      const int32_t* lengths, const mxattn_groups* groups, int max_len, const mxattn_opts* opts, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Workspace bytes mxattn_prefix_run uses for these sizes (0: none needed, or invalid arguments); only the geometry
 * of `cache` is read. */
size_t mxattn_prefix_workspace_size(const mxkv_cache* cache, int seqs, int q_heads, int groups, int max_len, int max_shared);

/*
 * mxkv_copy_run -- copy whole pages (keys, values and scales) of n_layers caches of one geometry, which
 * may be different allocations: page pairs[i][0] to page pairs[i][1] for every i < n_pairs, in every
 * layer. pairs: int32 [n_pairs][2] on the device. Pairs run in no order: the destinations must be
 * distinct, and none of them a source. Pairs with a page out of range, or of a page with itself, are
 * ignored. layers: host array, read before the call returns. n_layers, n_pairs: 0 .. MX_MAX_DIM (0:
 * nothing is done). MX_ERR_SHAPE also where the layers' geometry differs, and for pages of 16 GiB of keys and more.
 */
int mxkv_copy_run(const mxkv_cache* layers, int n_layers, const int32_t* pairs, int n_pairs, void* stream);

/* Why mxkv_step_run did nothing (bits of its status): too few free pages; more new tokens than max_tokens; a row longer than its
 * table's columns; pages given back that would overfill the stack, which then did not hold what was free. */
#define MXKV_STEP_PAGES 1
#define MXKV_STEP_TOKENS 2
#define MXKV_STEP_LONG 4
#define MXKV_STEP_STACK 8

/*
 * mxkv_step_run -- a step's page tables, tokens and slots from the rows' lengths, on the device (the pool below is the same on the
 * host, and knows shared pages). Row b has lengths[b] tokens in the cache and is to have wants[b] (negative: as
 * many as it has). All pointers are to device memory.
 *  - A row that grows takes pages for its columns from the end of free_pages[0 .. *n_free - 1]; one that shrinks gives its last pages
 *    back there, those of columns below kept[b] apart (kept NULL: 0), which it shares and does not own. Cells of the table that lose
 *    their page become -1. Pages are given back before any is taken, rows in order, columns in order; giving back what a call took
 *    restores the stack.
 *  - The step's tokens, positions lengths[b] .. wants[b] - 1 of every row that grows, rows in order: token t has row seq[t],
 *    position positions[t], and slots[t] = page * page_size + position % page_size (slots NULL: not wanted; -1 without
 *    a page). Row b's tokens are offsets[b] .. offsets[b + 1] - 1. seq, positions and slots of the places behind the last token, to
 *    max_tokens, become -1: mxkv_append_run leaves such tokens out, so a captured step may have fewer.
 *  - lengths_out = the new lengths and *n_free_out (each may be what it was read from), *status = 0. Where the step is not
 *    possible, *status is a sum of MXKV_STEP_ bits, lengths and n_free are copied, the table and the stack stay, and the step
 *    has no tokens.
 * lengths outside 0 .. cols * page_size, and n_free outside 0 .. pages, are taken as that bound. A row's cells of the positions that it has are expected
 * to hold its pages, as calls leave them, and the stack to hold free ones.
 * Rules (MX_ERR_SHAPE): 0 <= seqs (0: nothing is done), pages, page_size, max_tokens <= MX_MAX_DIM; cols * page_size and pages * page_size below 2^31.
 */
typedef struct {
  int seqs, cols, page_size, pages, max_tokens;
  int32_t* table;                         /* [seqs][cols] */
  const int32_t *lengths, *wants, *kept;  /* [seqs] */
  int32_t* free_pages;                    /* [pages] */
  const int32_t* n_free;                  /* [1] */
  int32_t *lengths_out, *n_free_out;      /* [seqs], [1] */
  int32_t *offsets;                       /* [seqs + 1] */
  int32_t *seq, *positions, *slots;       /* [max_tokens] */
  int32_t* status;                        /* [1] */
} mxkv_step;
int mxkv_step_run(const mxkv_step* step, void* stream);

/*
 * mxkv_pool -- host bookkeeping of a cache's pages: which page belongs to which sequences, as tables
 * for the calls above. Host only, queues no GPU work; not safe for concurrent calls on one pool. A new
 * page is always the free one with the lowest number. Sequences may share pages (fork); a page is free
 * when no sequence holds it. Functions that hand out page pairs expect the caller to queue
 * mxkv_copy_run for them before any later write to the cache, and before the pairs of a call that follows a
 * sequence's shrinking: a page that one call reads can be what a later one writes.
 */
typedef struct mxkv_pool_state* mxkv_pool;

/* A pool of `pages` pages for `seqs` sequences, all empty, of at most cols pages each. MX_ERR_SHAPE: a
 * value below 1 or above MX_MAX_DIM, or seqs * cols or pages * page_size of 2^31 or more. */
int mxkv_pool_create(mxkv_pool* out, int pages, int page_size, int seqs, int cols);
int mxkv_pool_destroy(mxkv_pool p);

/* Set sequence `seq`'s length to `tokens`, taking pages at its end or giving them back. Where it grows
 * and its last, partly filled page is shared, the sequence gets a copy of its own: pair[0] and pair[1]
 * are the source and the copy and *n_pairs is 1 (else 0). MX_ERR_NOMEM: too few free pages (nothing
 * has changed). MX_ERR_SHAPE: seq out of range, or tokens outside 0 .. cols * page_size. */
int mxkv_pool_resize(mxkv_pool p, int seq, int tokens, int32_t pair[2], int* n_pairs);

/* Let the empty sequence dst hold src's pages and length (MX_ERR_SHAPE if dst is not empty, or
 * src == dst). Nothing is copied until one of them grows. */
int mxkv_pool_fork(mxkv_pool p, int src, int dst);

/* Reorder: sequence i becomes what sequence from[i] was, for all i at once (from: int32 [seqs]; several
 * i may name one source, as when beams are chosen, and sources named by none are freed). */
int mxkv_pool_reorder(mxkv_pool p, const int32_t* from);

/* Move the used pages with the highest numbers into the free ones with the lowest until the used pages are
 * 0 .. used - 1. Writes at most max_pairs moves to pairs and their number to *n_pairs (further calls
 * go on); the tables name the new pages at once. */
int mxkv_pool_compact(mxkv_pool p, int32_t* pairs, int max_pairs, int* n_pairs);

/* The tables (int32 [seqs][cols], -1 where there is no page) and lengths (int32 [seqs]) in host memory
 * owned by the pool, and the number of pages in use. NULL / 0 for a NULL pool. */
const int32_t* mxkv_pool_table(mxkv_pool p);
const int32_t* mxkv_pool_lengths(mxkv_pool p);
int mxkv_pool_used(mxkv_pool p);

#ifdef __cplusplus
}
#endif
#endif /* MXGEMM_H */
