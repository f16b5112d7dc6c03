/*
 * tilegemm — tiled dense GEMM, weight-only 4-bit dequant GEMM, MX-format GEMM,
 * 2:4 structured-sparse GEMM, 8-bit integer GEMM with its quantisation, and
 * the norms between transformer blocks, for one AMD Instinct MI355X (gfx950),
 * as hand-written HIP kernels behind a C ABI.
 *
 * The operation follows the pages' problem statement:
 *   - "TileLang ... 一个高效 GEMM 内核" (mhpq.cn), section 3.2: the caller
 *     allocates A (M x K), B (K x N) and C (M x N) on the device and launches
 *     kernel(A, B, C); the result is C = A x B.  Section 3.4 checks that the
 *     inner dimensions agree before launching.
 *   - "TileLang：用Python DSL简化GPU算子开发" (gtnt.cn), section 4.3: operands
 *     are row-major unless stated otherwise; mixed precision needs an explicit
 *     cast.
 *   - "使用 Tilelang DSL 开发 GPU/CPU/加速器高性能内核" (blog.hotdry.top): an
 *     elementwise post-processing loop (ReLU) on the output tile, and the
 *     weight-only low-bit "Dequant GEMM" as a target workload.
 *
 * Conventions shared by every entry point:
 *   - All matrix pointers are DEVICE pointers owned by the caller.  The library
 *     never allocates, frees or synchronises, and keeps no per-call state.
 *   - Dense row-major storage with implied leading dimensions
 *     (lda = K, ldb = N, ldc = N; packed weights: K/2 bytes per row), unless
 *     the entry takes row strides.
 *   - Calls are asynchronous on `stream` (NULL = the null stream): they return
 *     once the kernel is enqueued.  Thread-safe.
 *   - Arguments are validated before any HIP call; on a non-OK status nothing
 *     has been launched and C is untouched (TG_ERR_HIP from an entry of two
 *     launches: the first may have run).
 *   - M == 0 or N == 0: TG_OK, nothing launched (all pointers may be NULL).
 *     K == 0: C = epilogue(0) = 0; the operand pointers may be NULL then.
 *   - Accumulation is always fp32; the output is rounded to its type once,
 *     round-to-nearest-even (fp32 -> fp16 overflow gives +-inf).
 *   - Each operand of the products without row strides must fit a 31-bit byte
 *     offset per tile row band (up to 256 rows of a k-contiguous operand, up to
 *     128 k-rows of an n-contiguous one):
 *     the library returns TG_ERR_BAD_SHAPE when 256 * K * element_size or
 *     128 * N * element_size exceeds 2^31 - 1 (and for M, N, K above 2^31 - 1).
 */
#ifndef TILEGEMM_H
#define TILEGEMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct ihipStream_t* tg_stream_t; /* same object as hipStream_t */

typedef enum {
    TG_OK = 0,
    TG_ERR_NULL_POINTER = 1, /* a required pointer is NULL                        */
    TG_ERR_BAD_SHAPE = 2,    /* negative / too large size, dequant K % 32 != 0,   */
                             /* or MX K % 128 != 0                                */
    TG_ERR_BAD_DTYPE = 3,    /* dtype not one of tg_dtype (MX: tg_mx_format)      */
    TG_ERR_BAD_EPILOGUE = 4, /* epilogue not one of tg_epilogue                   */
    TG_ERR_ALIAS = 5,        /* C overlaps an input                               */
    TG_ERR_NO_CONFIG = 6,    /* forced config index out of range / wrong op       */
    TG_ERR_HIP = 7,          /* the HIP runtime reported an error at launch       */
    TG_ERR_BAD_LAYOUT = 8,   /* trans_a / trans_b not 0 or 1; block norm: operands */
                             /* that do not go together                           */
    TG_ERR_WORKSPACE = 9,    /* workspace NULL, too small or misaligned            */
    TG_ERR_SCRATCH = 10      /* split-K partials exceed TG_SPLITK_SCRATCH_BYTES    */
} tg_status;

typedef enum { TG_F32 = 0, TG_F16 = 1, TG_BF16 = 2 } tg_dtype;

typedef enum { TG_EPI_NONE = 0, TG_EPI_RELU = 1 } tg_epilogue;

typedef enum {
    TG_OP_GEMM = 0,
    TG_OP_DEQUANT_W4 = 1,
    TG_OP_MX = 2,
    TG_OP_SP24 = 3,
    TG_OP_I8 = 4 /* tg_query_config only: its kernels are chosen by rule, not listed */
} tg_op;

/* Element format of the activations of tg_gemm_mx. */
typedef enum { TG_MX_E2M1 = 0, TG_MX_E4M3 = 1 } tg_mx_format;

/*
 * C = epilogue(A x B).
 *   A: [M][K] row-major, B: [K][N] row-major, C: [M][N] row-major, all of
 *   `dtype` (fp32, fp16 or bf16); products accumulate in fp32 on the matrix
 *   cores; TG_EPI_RELU maps every accumulated value v to (v > 0 ? v : +0)
 *   before the single rounding to `dtype`.
 *   Non-multiple-of-tile shapes are handled inside the kernel (out-of-range
 *   rows and columns are never read into the sum nor written).
 * Errors: TG_ERR_NULL_POINTER (C NULL with M, N > 0, or A or B NULL with
 *   M, N, K > 0), TG_ERR_BAD_SHAPE,
 *   TG_ERR_BAD_DTYPE, TG_ERR_BAD_EPILOGUE, TG_ERR_ALIAS (C's bytes overlap A's
 *   or B's), TG_ERR_HIP.
 */
tg_status tg_gemm(int64_t M, int64_t N, int64_t K, tg_dtype dtype, const void* A, const void* B,
                  void* C, tg_epilogue epi, tg_stream_t stream);

/*
 * C = epilogue(op(A) x op(B)) with either operand stored transposed: the
 * operand layouts of the backward products of the mhpq.cn page's autograd
 * wrapper (section 3.4: dA = dC x B^T, dB = A^T x dC) and the column-major
 * option the gtnt.cn page names (section 4.3).
 *   trans_a = 0: A is [M][K] row-major (as tg_gemm); 1: A is stored [K][M]
 *                row-major, i.e. op(A) = (stored A)^T, M x K.
 *   trans_b = 0: B is [K][N] row-major (as tg_gemm); 1: B is stored [N][K]
 *                row-major, i.e. op(B) = (stored B)^T, K x N.
 *   C: [M][N] row-major.  Same arithmetic, epilogue and rounding as tg_gemm;
 *   tg_gemm_ex(..., A, 0, B, 0, ...) is tg_gemm.
 * Every layout runs every dtype and alignment: 16-byte aligned operands whose
 * stored rows are whole 16-byte chunks take 16-byte loads (16-bit types: the
 * LDS-DMA kernel; fp32: the register-staged kernel), any other call takes
 * element loads.
 * Errors: as tg_gemm; TG_ERR_BAD_LAYOUT (trans_a or trans_b not 0 or 1),
 *   TG_ERR_BAD_SHAPE also when trans_a and 128 * M * element_size exceeds
 *   2^31 - 1.
 */
tg_status tg_gemm_ex(int64_t M, int64_t N, int64_t K, tg_dtype dtype, const void* A, int trans_a,
                     const void* B, int trans_b, void* C, tg_epilogue epi, tg_stream_t stream);

/*
 * Split-K GEMM: C = epilogue(A x B) as tg_gemm, with each output tile's K range
 * split over several workgroups, for shapes whose tile grid alone leaves most
 * compute units idle (few output tiles, long K).  The mhpq.cn page names the
 * tail effect of small problems (section 4.3); split K is the standard remedy
 * for it and, unlike tg_gemm, needs memory for partial sums: the caller brings
 * it as `workspace`.
 *   A, B, C, dtype, epi: as tg_gemm (row-major, fp32 / fp16 / bf16).
 *   splits: 0 = chosen by the library (about one workgroup per compute unit,
 *     at least two k strips per split); n >= 1 = at most n splits (fewer when
 *     K holds fewer strips); 1 = no split, identical to tg_gemm.
 *   workspace: device memory, 16-byte aligned, of at least the size
 *     tg_gemm_splitk_workspace_size reports for the same M, N, K, dtype and
 *     splits.  It holds per-tile arrival counters and fp32 partial tiles.  It
 *     must be zero-filled before its first use; every call leaves the counters
 *     zero again, so it is reused without clearing.  Calls that share a
 *     workspace must not run concurrently (issue them on one stream).
 *   Numerics: each split sums its k range in fp32 on the matrix cores; the
 *     split sums are added in fp32 in split order 0, 1, ... by whichever
 *     workgroup of the tile finishes last, so the result does not depend on
 *     the order in which workgroups run; then the ReLU and the single rounding
 *     of tg_gemm.  Integer-valued inputs give tg_gemm's result bit for bit
 *     (every partial sum is exact in fp32).
 *   When no split pays off (or the operands are not 16-byte aligned with rows
 *   of whole 16-byte chunks) the call runs tg_gemm's kernel and does not touch
 *   the workspace, which may then be NULL.
 * Errors: as tg_gemm; TG_ERR_BAD_SHAPE also for splits < 0; TG_ERR_ALIAS also
 *   when the workspace overlaps A, B or C; TG_ERR_WORKSPACE when a split is
 *   launched and the workspace is NULL, smaller than needed or not 16-byte
 *   aligned.
 */
tg_status tg_gemm_splitk(int64_t M, int64_t N, int64_t K, tg_dtype dtype, const void* A,
                         const void* B, void* C, tg_epilogue epi, int splits, void* workspace,
                         size_t workspace_bytes, tg_stream_t stream);

/*
 * Workspace bytes tg_gemm_splitk (and tg_gemm_splitk_config with any
 * configuration) needs for this call: written to *bytes, 0 when no split
 * would be launched.  Pure host function.
 * Errors: TG_ERR_NULL_POINTER (bytes NULL), TG_ERR_BAD_DTYPE,
 *   TG_ERR_BAD_SHAPE (as tg_gemm, or splits < 0).
 */
tg_status tg_gemm_splitk_workspace_size(int64_t M, int64_t N, int64_t K, tg_dtype dtype,
                                        int splits, size_t* bytes);

/*
 * Split-K GEMM that allocates nothing, for callers that cannot allocate device
 * memory or pass a workspace (code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc).  Same arguments, numerics and
 * results as tg_gemm_splitk, without the workspace: the arrival counters and
 * fp32 partial tiles live in a fixed static device array of
 * TG_SPLITK_SCRATCH_BYTES, one per GPU, held from the library's first use on
 * that GPU until the process ends.  The array's device address is looked up
 * once per device (the calling thread's current device, which must be the
 * stream's).  Each call that splits first zeroes the counters it uses with a
 * small fill kernel on `stream` (no memset node, so it can be captured), then
 * launches the GEMM; nothing is allocated or freed.
 * Every call on one GPU shares the array: calls that overlap in time on one
 * GPU (other streams, other threads) race and give wrong results; issue them
 * on one stream.
 * Errors: as tg_gemm_splitk (never TG_ERR_WORKSPACE); TG_ERR_SCRATCH when the
 *   split launched would need more than TG_SPLITK_SCRATCH_BYTES
 *   (tg_gemm_splitk_workspace_size gives the bytes; lower `splits` or use
 *   tg_gemm_splitk); TG_ERR_HIP also when the array's address lookup fails.
 */
#define TG_SPLITK_SCRATCH_BYTES (16 * 1024 * 1024)
tg_status tg_gemm_splitk_noalloc(int64_t M, int64_t N, int64_t K, tg_dtype dtype,
                                 const void* A, const void* B, void* C, tg_epilogue epi,
                                 int splits, tg_stream_t stream);

/*
 * Weight-only 4-bit dequant GEMM: C = epilogue(A x W^T).
 *   A : bf16 [M][K] row-major activations.
 *   Wq: uint8 [N][K/2]: weight row n holds its K E2M1 codes (OCP MX v1.0 FP4:
 *       sign, 2-bit exponent with bias 1, 1-bit mantissa) two per byte, even k
 *       in bits 3:0 and odd k in bits 7:4.
 *   Ws: uint8 [N][K/32]: one E8M0 scale byte E per 32 consecutive k of a row,
 *       scale 2^(E - 127).
 *   W[n][k] = e2m1(code(n, k)) * 2^(Ws[n][k/32] - 127); C[m][n] = sum_k A[m][k] * W[n][k].
 *   C : bf16 [M][N].  The weights are expanded to bf16 on chip (exact for
 *       E in [2, 252]; other scale bytes follow the hardware conversion) and
 *       multiplied on the bf16 matrix cores with fp32 accumulation.
 *   The pages name this workload ("WFP4" GEMM, "Dequant GEMM") but not its
 *   format; the format above is the workload statement's.
 * Errors: as tg_gemm; TG_ERR_BAD_SHAPE also when K % 32 != 0.
 */
tg_status tg_dequant_gemm_w4(int64_t M, int64_t N, int64_t K, const void* A, const uint8_t* Wq,
                             const uint8_t* Ws, void* C, tg_epilogue epi, tg_stream_t stream);

/*
 * MX-format GEMM: C = epilogue(A x W^T) with the activations, too, in OCP
 * microscaling blocks (the pages' "WFP4" GEMM of "TileLang架构深度剖析", the
 * performance section, run natively in the block formats instead of
 * dequantised: the matrix cores of gfx950 multiply E2M1 / E4M3 elements and
 * apply the E8M0 block scales themselves).
 *   Aq: activation element codes, format a_fmt:
 *       TG_MX_E2M1: uint8 [M][K/2], two E2M1 codes per byte as in Wq below;
 *       TG_MX_E4M3: uint8 [M][K], one OCP E4M3 code per byte (sign, 4-bit
 *                   exponent with bias 7, 3-bit mantissa; no infinities;
 *                   S.1111.111 is NaN; largest finite value 448).
 *   As: uint8 [M][K/32]: one E8M0 scale byte per 32 consecutive k of a row.
 *   Wq: uint8 [N][K/2] E2M1 weight codes, Ws: uint8 [N][K/32] E8M0 scales,
 *       laid out as for tg_dequant_gemm_w4.
 *   a(m, k) = elem(Aq, m, k) * 2^(As[m][k/32] - 127),
 *   w(n, k) = e2m1(Wq, n, k) * 2^(Ws[n][k/32] - 127),
 *   C[m][n] = sum_k a(m, k) * w(n, k), rounded once to bf16; C: bf16 [M][N].
 *   Scale byte 255 is NaN: every result that takes a product of that block is
 *   NaN (as is every one that takes an E4M3 NaN).
 *   Arithmetic: the gfx950 scaled matrix instruction adds each group of 8
 *   consecutive products (within one 32-k block) in fixed point whose last
 *   bit is 2^(e - 13), e being the group's largest exponent sum E(a) + E(w)
 *   of the unscaled elements (subnormal and zero elements count with their
 *   format's smallest normal exponent), each product truncated toward zero;
 *   group sums are scaled and accumulated in fp32.  E2M1 x E2M1 products
 *   never reach that window (exact up to the fp32 accumulation); E4M3
 *   products more than 2^13 below their group's largest lose their low bits.
 *   (Measured on MI355X with in-bounds probes; the reference is the exact
 *   sum.)
 *   The pages give no format for this workload; the one above is the OCP MX
 *   v1.0 definition.
 * Requirements: K % 128 == 0 (else TG_ERR_BAD_SHAPE); Aq and Wq 16-byte
 *   aligned, As and Ws 4-byte aligned (else TG_ERR_NO_CONFIG).  (Forced
 *   configurations whose name ends in _sc8 also need K % 512 == 0 and 16-byte
 *   aligned As and Ws.)
 * Errors: as tg_gemm; TG_ERR_BAD_DTYPE when a_fmt is not a tg_mx_format.
 */
tg_status tg_gemm_mx(int64_t M, int64_t N, int64_t K, tg_mx_format a_fmt, const uint8_t* Aq,
                     const uint8_t* As, const uint8_t* Wq, const uint8_t* Ws, void* C,
                     tg_epilogue epi, tg_stream_t stream);

/*
 * 2:4 structured-sparse GEMM: C = epilogue(A x B) with A [M][K] keeping at
 * most two values in every group of four consecutive k, given compressed
 * (the 2:4 sparse GEMM of "使用 Tilelang DSL 开发 GPU/CPU/加速器高性能内核",
 * its monitoring-and-debugging paragraph, which skips the dense work):
 *   Ac: [M][K/2] of `dtype`: group j (k = 4j .. 4j + 3) of row m keeps
 *       Ac[m][2j] and Ac[m][2j + 1];
 *   Ai: uint8 [M][K/8]: group j's positions as the nibble
 *       (Ai[m][j/2] >> (4 * (j % 2))) & 0xF = p0 | p1 << 2 (p0, p1 in 0..3;
 *       a repeated position adds both values);
 *   B : [K][N] row-major of `dtype`; C: [M][N] of `dtype`.
 *   C[m][n] = sum_j (Ac[m][2j] * B[4j + p0][n] + Ac[m][2j + 1] * B[4j + p1][n]),
 *   fp32 accumulation on the sparse matrix instruction, one RNE rounding;
 *   TG_EPI_RELU as for tg_gemm.  The pages give no storage format; this one
 *   is the library's (two values per group in k order, 4-bit position pairs).
 * Requirements: dtype TG_F16 or TG_BF16 (else TG_ERR_BAD_DTYPE); K % 32 == 0
 *   (else TG_ERR_BAD_SHAPE); Ac and B 16-byte aligned, N % 8 == 0, Ai 4-byte
 *   aligned (else TG_ERR_NO_CONFIG).
 * Errors: as tg_gemm.
 */
tg_status tg_gemm_sp24(int64_t M, int64_t N, int64_t K, tg_dtype dtype, const void* Ac,
                       const uint8_t* Ai, const void* B, void* C, tg_epilogue epi,
                       tg_stream_t stream);

/*
 * Quantisation of activations to 8-bit integers, one scale for each row
 * (token): for row m with a = max(max_k |X[m][k]|, 127 * 2^-126),
 *   Q[m][k] = round(127 X[m][k] / a), ties to even;  s[m] = a / 127 (fp32),
 * so that X[m][k] is Q[m][k] s[m] to half a level.  (The lower bound on a
 * keeps s normal: a row of zeros gets zero levels and the scale 2^-126.)
 * A row that holds an infinity or NaN gets zero levels and the scale NaN:
 * every product taken from it is NaN (with TG_EPI_RELU zero: this library's ReLU
 * takes NaN to 0, so a program that has to see such a row looks at s).
 *   X: [M][K] of `dtype`, row stride ldx; Q: int8 [M][K], row stride ldq;
 *   s: fp32 [M].  Strides in elements, at least K.  Any alignment.
 *   The levels are the exact ones for fp32, fp16 and bf16 inputs.
 * Errors: TG_ERR_BAD_DTYPE, TG_ERR_BAD_SHAPE (negative or above 2^31 - 1, or a
 *   stride below K), TG_ERR_NULL_POINTER, TG_ERR_ALIAS (Q or s overlaps X or
 *   each other), TG_ERR_HIP.
 */
tg_status tg_quant_i8(int64_t M, int64_t K, tg_dtype dtype, const void* X, int64_t ldx, int8_t* Q,
                      int64_t ldq, float* s, tg_stream_t stream);

/*
 * 8-bit integer GEMM with a scale for each token and channel:
 *   C[m][n] = epilogue(sa[m] sw[n] sum_k A[m][k] W[n][k] + bias[n]).
 *   A: int8 [M][K], row stride lda, with fp32 scales sa [M];
 *   W: int8 [N][K], row stride ldw, with fp32 scales sw [N];
 *   bias: fp32 [N] or NULL; C: [M][N] of `dtype`, row stride ldc.
 *   Strides in elements.  All 256 levels are valid.  The sum is exact (32-bit
 *   integers, hence K <= 131071); it is converted to fp32, scaled by sa, then
 *   sw with the bias added, the ReLU applied as in tg_gemm, and rounded once to `dtype`.
 *   Any sizes and alignment; rows of A and W that start at 16-byte boundaries
 *   with K % 16 == 0 take the fast kernels.  K == 0: C = epilogue(bias); A and
 *   W may be NULL then.
 * The pages name low-bit GEMM workloads ("TileLang架构深度剖析", the performance
 * section) but not this format.
 * Errors: TG_ERR_BAD_DTYPE, TG_ERR_BAD_EPILOGUE, TG_ERR_BAD_SHAPE (also a
 *   stride below its row length, K > 131071, lda or ldw > 8388607),
 *   TG_ERR_NULL_POINTER,
 *   TG_ERR_ALIAS (C overlaps an input), TG_ERR_HIP.
 */
tg_status tg_gemm_i8(int64_t M, int64_t N, int64_t K, const int8_t* A, int64_t lda,
                     const float* sa, const int8_t* W, int64_t ldw, const float* sw,
                     const float* bias, tg_dtype dtype, void* C, int64_t ldc, tg_epilogue epi,
                     tg_stream_t stream);

/*
 * The two above in one call: C = epilogue(X W^T + bias) with the rows of X
 * quantised as by tg_quant_i8 and W in 8 bits as in tg_gemm_i8.
 *   X: [M][K] of `dtype`, row stride ldx; C: [M][N] of `dtype`, row stride ldc.
 *   workspace: device memory, 16-byte aligned, of at least the size
 *     tg_linear_i8_workspace_size reports for these sizes (it holds the levels
 *     and scales and, for some sizes with K % 16 != 0, W with its rows at
 *     16-byte boundaries; 0 bytes, and NULL, where the call needs none).  Its
 *     contents need not be kept between calls; calls that share it must not
 *     run concurrently.
 *   The result has the bits of tg_quant_i8 followed by tg_gemm_i8.
 * Errors: as for those; TG_ERR_WORKSPACE when the workspace is NULL, smaller
 *   than needed or not 16-byte aligned; TG_ERR_ALIAS also when it overlaps an
 *   operand.
 */
tg_status tg_linear_i8(int64_t M, int64_t N, int64_t K, tg_dtype dtype, const void* X, int64_t ldx,
                       const int8_t* W, int64_t ldw, const float* sw, const float* bias, void* C,
                       int64_t ldc, tg_epilogue epi, void* workspace, size_t workspace_bytes,
                       tg_stream_t stream);
tg_status tg_linear_i8_workspace_size(int64_t M, int64_t N, int64_t K, tg_dtype dtype,
                                      size_t* bytes);

/*
 * The norms, gate and residual between two blocks of a transformer, in one
 * pass.  For each token t (row of D values), with norm(v) = v r and
 * r = 1 / sqrt(mean(v^2) + eps):
 *   x_out[t] = alpha x[t] + gate[t / gate_rows] * norm(y[t]) * w_post
 *   h[t]     = norm(x_out[t]) * w_pre
 * y is the output of the block before, x the residual stream beside it, h the
 * input of the block after.
 *   x, x_out: [T][D] of `xtype`; y, h: [T][D] of `btype`; gate: [ceil(T /
 *     gate_rows)][D], w_post, w_pre: [D], of `btype`, dense.  (xtype, btype):
 *     equal, or TG_F32 with TG_F16 or TG_BF16.  Row strides in elements.
 *   y NULL: there is no block before; x_out must be NULL, h = norm(x) * w_pre
 *     (alpha has no part in it).
 *   post_norm 0: y[t] stands in place of norm(y[t]) * w_post (w_post NULL).
 *   gate, w_post, w_pre NULL: ones.
 *   h, hq: either, both or (x_out not NULL) neither.  hq: int8 [T][D] with
 *     fp32 scales hs [T], as tg_gemm_i8 takes them as A and sa: h quantised as
 *     by tg_quant_i8.  The levels are the exact ones of norm(x_out) * w_pre, ties
 *     to even: r is one factor of the row and has no part in them, nor has any
 *     rounding of h.  (Only where x_out and w_pre are both fp32 may a value
 *     within a 64-bit rounding of the border between two levels get either, and in
 *     a row whose scale is the least one a value within an fp32 rounding of it.)
 *   r_post, r_pre: fp32 [T] or NULL: the norms' r, for the gradients.
 *   x_out may be x itself (same address and stride).
 * Sums and intermediate values are fp32; x_out is rounded to xtype, and h is
 * computed from the rounded x_out, so that the call equals one that computes
 * x_out and one that computes h from it, bit for bit.
 * D <= 32768, T <= 2^30.  T == 0 or D == 0: nothing is launched (with D == 0, hs,
 * r_post and r_pre are not written).  A row of zeros with eps 0 has no norm (NaN).
 * Errors: TG_ERR_BAD_DTYPE, TG_ERR_BAD_SHAPE (sizes, strides below D,
 *   gate_rows < 1 with a gate), TG_ERR_NULL_POINTER (x, or nothing to write,
 *   or hq without hs or the reverse, x_out NULL with y), TG_ERR_BAD_LAYOUT (x_out, gate, w_post
 *   or r_post without y; w_post or r_post without post_norm; r_pre or w_pre
 *   without h or hq), TG_ERR_ALIAS (an output overlaps an input, except x_out
 *   being x, or another output), TG_ERR_HIP.
 */
typedef struct {
    int64_t T, D;
    tg_dtype xtype, btype;
    const void* x;
    int64_t ldx;
    const void* y;
    int64_t ldy;
    const void* gate;
    int64_t gate_rows;
    const void* w_post;
    const void* w_pre;
    float alpha, eps;
    int post_norm;
    void* x_out;
    int64_t ldx_out;
    void* h;
    int64_t ldh;
    int8_t* hq;
    int64_t ldhq;
    float* hs;
    float* r_post;
    float* r_pre;
} tg_block_norm_args;

tg_status tg_block_norm(const tg_block_norm_args* args, tg_stream_t stream);

/*
 * Gradients of tg_block_norm (h as h; the 8-bit h has none).  In: x_new, the
 * x_out of the forward call (its x when y is NULL: dx is then the gradient at
 * x_new, whatever alpha is), y, gate, gate_rows,
 * w_post, w_pre, alpha, post_norm and the saved r_post, r_pre; the gradients
 * dx_new at x_out and dh at h (either may be NULL: zeros).  Out, each NULL if
 * not wanted:
 *   dx [T][D] of xtype, dy [T][D] of btype,
 *   dgate [ceil(T / gate_rows)][D], dw_post [D], dw_pre [D] in fp32: sums over
 *     the tokens that share them.
 *   Sums are fp32 in a fixed order: the same call gives the same bits.
 *   workspace: device memory, 16-byte aligned, of at least the size
 *     tg_block_norm_backward_workspace_size reports for the same arguments; it
 *     holds partial sums.  Its contents need not be kept; calls that share it must not run
 *     concurrently.
 * D <= 32768, T <= 2^30.  T == 0: dgate, dw_post and dw_pre are not written.
 * Above D = 8192 a row's sums do not fit the registers: right, but at 1.7 to 3
 * TB/s up to D = 16384 and 0.8 to 1 TB/s beyond, where shorter rows reach 4.2 to 5.
 * Errors: as tg_block_norm; TG_ERR_NULL_POINTER also when an input that an
 *   output needs is NULL (x_new and r_pre with dh, r_post with post_norm) or
 *   when nothing is to be written; TG_ERR_BAD_LAYOUT also for dy, dgate, dw_post without
 *   their y, gate, w_post, and dw_pre without w_pre and dh; TG_ERR_ALIAS (an
 *   output or the workspace overlaps an input or another output);
 *   TG_ERR_WORKSPACE.
 */
typedef struct {
    int64_t T, D;
    tg_dtype xtype, btype;
    const void* x_new;
    int64_t ldx_new;
    const void* y;
    int64_t ldy;
    const void* gate;
    int64_t gate_rows;
    const void* w_post;
    const void* w_pre;
    float alpha;
    int post_norm;
    const float* r_post;
    const float* r_pre;
    const void* dx_new;
    int64_t lddx_new;
    const void* dh;
    int64_t lddh;
    void* dx;
    int64_t lddx;
    void* dy;
    int64_t lddy;
    float* dgate;
    float* dw_post;
    float* dw_pre;
} tg_block_norm_grad_args;

tg_status tg_block_norm_backward(const tg_block_norm_grad_args* args, void* workspace,
                                 size_t workspace_bytes, tg_stream_t stream);
tg_status tg_block_norm_backward_workspace_size(const tg_block_norm_grad_args* args,
                                                size_t* bytes);

/*
 * Microscaled blocks (OCP MX v1.0): 32 consecutive elements of 4 bits (E2M1) or
 * 8 bits (E4M3) share one power of two P.  For a block with the largest
 * magnitude a,
 *   P = 2^(floor(log2 a) - emax), at least 2^-127   (emax: 2 for E2M1, 8 for E4M3),
 *   element = x / P rounded to the format, ties to even, at most its largest
 *     magnitude (6; 448),
 * and the scale byte is P's exponent + 127.  A block that holds an infinity or
 * NaN gets the scale byte 255 (NaN) and zero elements: every product taken from
 * it is NaN (with TG_EPI_RELU zero).  A block of zeros gets the scale byte 0.
 *
 * tg_quant_mx writes X's blocks along its rows (Q, S), along its columns as rows
 * of the transpose (Qt, St), or both in one launch (NULL: not wanted).
 *   X: [M][K] of `dtype`, row stride ldx in elements, any alignment.
 *   Q: codes of [M][Kp] elements, Kp = K rounded up to a multiple of 128, zeros
 *     past K: uint8 [M][Kp / 2], two E2M1 codes to a byte (even k in bits 3:0),
 *     or uint8 [M][Kp] of E4M3;  S: uint8 [M][Kp / 32].
 *   Qt: codes of [K][Mp] elements, Mp = M rounded up likewise, zeros past M;
 *     St: uint8 [K][Mp / 32].
 *   These are the operands of tg_gemm_mx (Aq, As or Wq, Ws, with its K the Kp
 *   here) and the weights of tg_linear_mx.
 * tg_dequant_mx writes the values that Q and S stand for, rounded once to `dtype`:
 *   X: [M][K], row stride ldx.
 * M or K == 0: nothing is launched.
 * Errors: TG_ERR_BAD_DTYPE (also fmt), TG_ERR_BAD_SHAPE (negative, above 2^29 - 1,
 *   a stride below K, or M Kp of 2^36 and more, in fp32 2^35), TG_ERR_NULL_POINTER
 *   (X, neither Q nor Qt, or codes without scales or the reverse),
 *   TG_ERR_NO_CONFIG (codes not 16-byte or scales not 4-byte aligned),
 *   TG_ERR_ALIAS (an output overlaps X or another), TG_ERR_HIP.
 */
tg_status tg_quant_mx(int64_t M, int64_t K, tg_dtype dtype, const void* X, int64_t ldx,
                      tg_mx_format fmt, uint8_t* Q, uint8_t* S, uint8_t* Qt, uint8_t* St,
                      tg_stream_t stream);
tg_status tg_dequant_mx(int64_t M, int64_t K, tg_mx_format fmt, const uint8_t* Q, const uint8_t* S,
                        tg_dtype dtype, void* X, int64_t ldx, tg_stream_t stream);

/*
 * Linear layer with 4-bit weights: C = epilogue(Q(X) W^T + bias), the rows of X
 * brought to blocks of format `fmt` within the call, as by tg_quant_mx.
 *   X: [M][K] of `dtype`, row stride ldx; bias: fp32 [N] or NULL; C: [M][N] of
 *   `dtype`, row stride ldc.  Strides in elements, any alignment.
 *   Wq, Ws: E2M1 weights [N][Kp] as tg_quant_mx writes them (Kp: K rounded up to
 *     a multiple of 128); what they hold past K has no part in C as long as its
 *     scale bytes are not 255.
 *   Products are exact and summed in fp32, the bias is added in fp32 and C rounded
 *   once; sums are taken in an order that depends on the sizes only.  Only a 16-bit
 *   C of more than 16 tokens with E4M3 activations may take the arithmetic that
 *   tg_gemm_mx states for them, which cuts the products of each eight k at 2^-13 of
 *   their largest (measured: 7e-6 of the result; rounding to fp16 alone is 2.1e-4).
 *   workspace: device memory, 16-byte aligned, of at least the size
 *     tg_linear_mx_workspace_size reports for these sizes (it holds X's codes
 *     and scales; 0 bytes, and NULL, where the call needs none).  Its contents
 *     need not be kept between calls; calls that share it must not run
 *     concurrently.
 *   K == 0: C = epilogue(bias); X, Wq and Ws may be NULL then.
 * Errors: TG_ERR_BAD_DTYPE (also fmt), TG_ERR_BAD_EPILOGUE, TG_ERR_BAD_SHAPE
 *   (also a stride below its row length, K > 8388479, M above 2^29 - 1, N above
 *   2^27 - 16, or an X that tg_quant_mx does not take),
 *   TG_ERR_NULL_POINTER, TG_ERR_NO_CONFIG (Wq not 16-byte or Ws not 4-byte aligned),
 *   TG_ERR_WORKSPACE, TG_ERR_ALIAS (C or the workspace overlaps an operand or
 *   each other), TG_ERR_HIP.
 */
tg_status tg_linear_mx(int64_t M, int64_t N, int64_t K, tg_dtype dtype, const void* X, int64_t ldx,
                       tg_mx_format fmt, const uint8_t* Wq, const uint8_t* Ws, const float* bias,
                       void* C, int64_t ldc, tg_epilogue epi, void* workspace,
                       size_t workspace_bytes, tg_stream_t stream);
tg_status tg_linear_mx_workspace_size(int64_t M, int64_t N, int64_t K, tg_dtype dtype,
                                      tg_mx_format fmt, size_t* bytes);

/*
 * Gradients of the linear layer Y = X W^T + bias with both products in blocks, each
 * operand quantised along the axis that is summed (Q(.) to `fmt`, Q4(.) to E2M1):
 *   dX[M][K] = Q(dY) Q4(W)       blocks along N,
 *   dW[N][K] = Q(dY)^T Q4(X)     blocks along M,
 *   dbias[N] = sum_m dY[m][n]    from dY as given, fp32, in a fixed order.
 * X and W are in 4 bits here whatever `fmt` is: a layer whose forward pass took X in
 * E4M3 gets dW from X in E2M1.
 * The roundings of the quantisation are passed over (their gradient is taken to be
 * that of the value itself).  dY is the gradient before the ReLU, if there is one.
 * Products and sums are those of tg_linear_mx.
 *   dY: [M][N], X, dX: [M][K] of `dtype`; W, dW: [N][K] of `wtype`, which is
 *   `dtype` or TG_F32 (W as the optimiser holds it, not in 4 bits).  Row strides in
 *   elements, any alignment.  dX, dW, dbias: NULL if not wanted; dX needs W, dW
 *   needs X.
 *   workspace: as for tg_linear_mx, of the size that
 *     tg_linear_mx_backward_workspace_size reports for the same arguments.
 * With no tokens dW and dbias are zero, with N == 0 dX is.  Outputs without elements
 * may be NULL.
 * Errors: TG_ERR_NULL_POINTER (an input that an output needs, or no output),
 *   TG_ERR_BAD_DTYPE, TG_ERR_BAD_SHAPE (also a size above 8388479),
 *   TG_ERR_WORKSPACE, TG_ERR_ALIAS (an output or the workspace overlaps an input
 *   or another output), TG_ERR_HIP.
 */
typedef struct {
    int64_t M, N, K;
    tg_dtype dtype, wtype;
    tg_mx_format fmt;
    const void* dY;
    int64_t lddy;
    const void* X;
    int64_t ldx;
    const void* W;
    int64_t ldw;
    void* dX;
    int64_t lddx;
    void* dW;
    int64_t lddw;
    float* dbias;
} tg_linear_mx_grad_args;

tg_status tg_linear_mx_backward(const tg_linear_mx_grad_args* args, void* workspace,
                                size_t workspace_bytes, tg_stream_t stream);
tg_status tg_linear_mx_backward_workspace_size(const tg_linear_mx_grad_args* args,
                                               size_t* bytes);

/*
 * Norm of every query and key head with the rotation to its token's position, in
 * one pass.  For a head x of D values at position t,
 *   y = x r * w,  r = 1 / sqrt(mean(x^2) + eps),
 *   out = y with pair i of its first R values (a, b) turned to
 *     (a cos[t][i] - b sin[t][i], a sin[t][i] + b cos[t][i]);
 * pair i is (i, i + R / 2), or (2 i, 2 i + 1) with `interleaved`; values past R
 * are not turned.
 *   q: Hq heads of T tokens: values of token t, head h at q + t q_t + h q_h
 *     (strides in elements; slices of one projection's output, or heads that
 *     hold their tokens); k: Hk heads, likewise.  No heads of a kind: its
 *     pointers may be NULL.
 *   w_q, w_k: [D] of `dtype`, or NULL: ones.
 *   cos, sin: fp32 [P][R / 2], dense; positions: int64 [T], or NULL: token t is at
 *     position t.  Values turned by a position outside [0, P) are NaN; tables are
 *     not read out of range.
 *   q_out, k_out: of `dtype`; may be q and k themselves (same address and strides).
 *   Heads of queries and keys may lie between each other (the same strides, other
 *   places); of other strides, ranges that overlap count as overlapping.
 * Sums and intermediate values are fp32, one rounding to `dtype`.
 * D <= 1024, T <= 2^30, Hq and Hk <= 65536.
 * Errors: TG_ERR_BAD_DTYPE, TG_ERR_BAD_SHAPE (sizes, R odd or above D, strides
 *   negative, heads of an output that overlap, P < T without positions, P < 1
 *   with R), TG_ERR_NULL_POINTER, TG_ERR_ALIAS (an output overlaps an input,
 *   except in place, or the other output), TG_ERR_HIP.
 */
typedef struct {
    int64_t T, Hq, Hk, D, R;
    tg_dtype dtype;
    const void* q;
    int64_t q_t, q_h;
    const void* k;
    int64_t k_t, k_h;
    const void* w_q;
    const void* w_k;
    const float* cos;
    const float* sin;
    int64_t P;
    const int64_t* positions;
    float eps;
    int interleaved;
    void* q_out;
    int64_t q_out_t, q_out_h;
    void* k_out;
    int64_t k_out_t, k_out_h;
} tg_head_norm_rope_args;

tg_status tg_head_norm_rope(const tg_head_norm_rope_args* args, tg_stream_t stream);

/*
 * Gradients of tg_head_norm_rope.  In: its inputs, q and k as they were, and the
 * gradients dq_out and dk_out at its outputs.  Out: dq, dk of `dtype`; dw_q, dw_k
 * [D] in fp32, sums over all tokens and heads in a fixed order (NULL: not wanted;
 * zero for no tokens).
 *   workspace: device memory, 16-byte aligned, of at least the size
 *     tg_head_norm_rope_backward_workspace_size reports for the same arguments; it
 *     holds partial sums.  Its contents need not be kept; calls that share it must
 *     not run concurrently.
 * Errors: as tg_head_norm_rope; TG_ERR_BAD_LAYOUT (dw_q, dw_k without w_q, w_k);
 *   TG_ERR_ALIAS (an output or the workspace overlaps an input or another output;
 *   there is no in-place form); TG_ERR_WORKSPACE.
 */
typedef struct {
    int64_t T, Hq, Hk, D, R;
    tg_dtype dtype;
    const void* q;
    int64_t q_t, q_h;
    const void* k;
    int64_t k_t, k_h;
    const void* w_q;
    const void* w_k;
    const float* cos;
    const float* sin;
    int64_t P;
    const int64_t* positions;
    float eps;
    int interleaved;
    const void* dq_out;
    int64_t dq_out_t, dq_out_h;
    const void* dk_out;
    int64_t dk_out_t, dk_out_h;
    void* dq;
    int64_t dq_t, dq_h;
    void* dk;
    int64_t dk_t, dk_h;
    float* dw_q;
    float* dw_k;
} tg_head_norm_rope_grad_args;

tg_status tg_head_norm_rope_backward(const tg_head_norm_rope_grad_args* args, void* workspace,
                                     size_t workspace_bytes, tg_stream_t stream);
tg_status tg_head_norm_rope_backward_workspace_size(const tg_head_norm_rope_grad_args* args,
                                                    size_t* bytes);

/* Static, NUL-terminated description of a status code (never NULL). */
const char* tg_status_str(tg_status s);

/*
 * Which compiled kernel configuration the library would launch for this call.
 * Writes a NUL-terminated description (tile sizes, waves, stages, swizzle
 * group, launch grid) into buf[0 .. len-1], truncating if needed.
 * op: TG_OP_GEMM, TG_OP_DEQUANT_W4 (dtype ignored), TG_OP_MX (dtype
 * carries the tg_mx_format of the activations), TG_OP_SP24 or TG_OP_I8 (dtype
 * is C's; rows at 16-byte boundaries assumed).
 * Errors: TG_ERR_NULL_POINTER (buf NULL or len 0), TG_ERR_BAD_SHAPE,
 *   TG_ERR_BAD_DTYPE, TG_ERR_NO_CONFIG (op unknown).
 */
tg_status tg_query_config(int op, int64_t M, int64_t N, int64_t K, tg_dtype dtype, char* buf,
                          size_t len);

/* As tg_query_config, for the operand layouts of tg_gemm_ex (dequant, MX and
 * sparse: 0, 0; TG_ERR_BAD_LAYOUT otherwise). */
tg_status tg_query_config_ex(int op, int64_t M, int64_t N, int64_t K, tg_dtype dtype, int trans_a,
                             int trans_b, char* buf, size_t len);

/*
 * Offline sweep support: the compiled configurations, listed per (op, dtype),
 * can be launched by index instead of by the built-in selection table.  The
 * dequant list ignores dtype; the MX list holds both activation formats and
 * ignores dtype too (a configuration runs calls of its own format only).
 *   tg_config_count: number of configurations for (op, dtype); 0 if none.
 *   tg_config_name : description of configuration `index` (as tg_query_config).
 *   tg_gemm_config / tg_gemm_ex_config / tg_dequant_gemm_w4_config /
 *     tg_gemm_mx_config / tg_gemm_sp24_config / tg_gemm_splitk_config: same
 *     contract as tg_gemm / tg_gemm_ex / tg_dequant_gemm_w4 / tg_gemm_mx /
 *     tg_gemm_sp24 / tg_gemm_splitk, launching configuration `index`;
 *     TG_ERR_NO_CONFIG if `index` is out of range or the configuration cannot
 *     run the call (operand layout, alignment, a K multiple it needs, another
 *     activation format, or, for split K, a configuration without k-slice
 *     wave groups: names with three wave counts, "_w1x1x4_").
 */
int tg_config_count(int op, tg_dtype dtype);
tg_status tg_config_name(int op, tg_dtype dtype, int index, char* buf, size_t len);
tg_status tg_gemm_config(int index, int64_t M, int64_t N, int64_t K, tg_dtype dtype,
                         const void* A, const void* B, void* C, tg_epilogue epi,
                         tg_stream_t stream);
tg_status tg_gemm_ex_config(int index, int64_t M, int64_t N, int64_t K, tg_dtype dtype,
                            const void* A, int trans_a, const void* B, int trans_b, void* C,
                            tg_epilogue epi, tg_stream_t stream);
tg_status tg_dequant_gemm_w4_config(int index, int64_t M, int64_t N, int64_t K, const void* A,
                                    const uint8_t* Wq, const uint8_t* Ws, void* C,
                                    tg_epilogue epi, tg_stream_t stream);
tg_status tg_gemm_mx_config(int index, int64_t M, int64_t N, int64_t K, tg_mx_format a_fmt,
                            const uint8_t* Aq, const uint8_t* As, const uint8_t* Wq,
                            const uint8_t* Ws, void* C, tg_epilogue epi, tg_stream_t stream);
tg_status tg_gemm_sp24_config(int index, int64_t M, int64_t N, int64_t K, tg_dtype dtype,
                              const void* Ac, const uint8_t* Ai, const void* B, void* C,
                              tg_epilogue epi, tg_stream_t stream);
tg_status tg_gemm_splitk_config(int index, int64_t M, int64_t N, int64_t K, tg_dtype dtype,
                                const void* A, const void* B, void* C, tg_epilogue epi,
                                int splits, void* workspace, size_t workspace_bytes,
                                tg_stream_t stream);

/*
 * The block-swizzled tile order, for host-side checking.  For a grid of
 * tiles_m x tiles_n output tiles and a swizzle group of `group_m` tile rows,
 * writes for every workgroup id w in [0, tiles_m * tiles_n) the tile it
 * computes: out_m[w], out_n[w].  Workgroup ids are first regrouped so that
 * the ids the hardware dispatches to one XCD (w mod 8) form a contiguous run,
 * then walked in groups of `group_m` tile rows, column by column.
 * Pure host function; touches no device.  Errors: TG_ERR_NULL_POINTER,
 * TG_ERR_BAD_SHAPE (tiles_m, tiles_n < 1, product above 2^31 - 1, group_m < 1).
 */
tg_status tg_tile_map(int64_t tiles_m, int64_t tiles_n, int group_m, int32_t* out_m,
                      int32_t* out_n);

/*
 * Clock record, a measurement aid.  The mhpq.cn page (section 4.2) reads a
 * GEMM's speed against the theoretical ceiling first; on a power-limited card
 * that ceiling moves with the shader clock, so a benchmark needs the clock the
 * kernel actually ran at.  With `stamps` set (a DEVICE pointer to 32 uint64,
 * caller-owned, NULL to switch off), every matrix-product kernel launched
 * afterwards by any entry point has wave 0 of its workgroups 0..7 (one per XCD) write
 * stamps[4 b + 0..3] = shader-clock counter and 100 MHz reference counter at
 * its start, then the same at its end (workgroups b < 8 only; a grid of fewer
 * workgroups leaves the rest untouched).  Each launch overwrites the previous
 * one's record, so read it after synchronising.  Clock of workgroup b:
 * (t1 - t0) / ((r1 - r0) / 100 MHz).  Process-wide setting for benchmarks;
 * calls on several threads or streams while it is set write the same buffer.
 */
void tg_set_clock_stamps(uint64_t* stamps);

/*
 * Tuning aids for the offline sweep (tiled_dense_gemm_07_amd/sweep.py), which
 * follows the mhpq.cn page's tuning advice (sections 4.2 and 4.3: measure
 * candidate tilings on the target GPU, check occupancy, keep the best).
 *   tg_set_swizzle_override: every launch afterwards, by any entry point, uses
 *     swizzle group `group_m` (tile rows per group of the block-swizzled tile
 *     order, a pure reordering: results are unchanged); 0 restores the
 *     selection's own group.  Process-wide, for timing runs.
 *   tg_config_occupancy: workgroups of compiled configuration `index` of
 *     (op, dtype) that one compute unit holds at once (registers, LDS and
 *     waves), from the HIP occupancy query on the current device.
 *     Errors: TG_ERR_NULL_POINTER, TG_ERR_NO_CONFIG (index out of range),
 *     TG_ERR_HIP (no device or the query failed).
 */
void tg_set_swizzle_override(int group_m);
tg_status tg_config_occupancy(int op, tg_dtype dtype, int index, int* workgroups_per_cu);

#ifdef __cplusplus
}
#endif

#endif /* TILEGEMM_H */
