/*
 * nvfp4.h -- C ABI of the MI355X (gfx950) NVFP4 block-scaled GEMM library.
 *
 * Operation (kernelindex, "NVFP4 linear layer", description): y = x @ W^T,
 * where x [M, K] and W [N, K] are both FP4 (E2M1) values, each run of 16
 * consecutive K-elements of a row carrying one FP8 E4M3FN scale factor.
 * Layout (same page, workload line: in_features_half = K/2, sf_k = K/16,
 * sf_vec_size = 16; magik.net "The 3.7 PFLOPS Revelation", "Input Knowledge",
 * item 2: two FP4 values per byte, data K//2 wide, scales K//16 wide):
 *   q  uint8 [rows, K/2]   element 2j in the low nibble of byte j,
 *                          nibble = sign(bit 3) | E2M1 magnitude code (bits 0-2)
 *   s  uint8 [rows, K/16]  E4M3FN bit patterns, row-major, no swizzle
 *   g  fp32                per-tensor global scale; a row element decodes as
 *                          E2M1(nibble) * E4M3(s[row, k/16]) * g
 * Quantisation may run ahead of the GEMM and is timed apart from it
 * (leverageai "blackwell-nvfp4-gemm-optimization", "What is this?").
 *
 * Conventions for every call:
 *   - All array pointers are DEVICE pointers (HBM of the current HIP device),
 *     allocated and owned by the caller.  The library allocates, frees and
 *     synchronises nothing; it keeps no state between calls.
 *   - Work is enqueued on `stream` (a hipStream_t; NULL = the null stream).
 *     Results are valid once the stream reaches that point.
 *   - Arguments are validated on the host before anything is enqueued; an
 *     invalid call returns a negative status and touches no memory.  A
 *     failed kernel launch returns NVFP4_ERR_HIP.  No call aborts or throws.
 *   - Sizes of 0 are valid and enqueue nothing (NVFP4_OK).
 *   - Inputs must be finite and scale bytes must not be NaN (0x7F, 0xFF);
 *     this is documented, not checked (checking would cost a device pass).
 */
#ifndef NVFP4_H_
#define NVFP4_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  NVFP4_OK = 0,
  NVFP4_ERR_INVALID_ARG = -1, /* bad size, null pointer, bad stride / dtype  */
  NVFP4_ERR_UNSUPPORTED = -2, /* valid but unsupported (alignment, sizes)    */
  NVFP4_ERR_HIP = -3          /* a HIP runtime call or kernel launch failed */
} nvfp4_status;

typedef enum {
  NVFP4_F32 = 0,  /* IEEE binary32                                         */
  NVFP4_BF16 = 1  /* bfloat16, written round-to-nearest-even from the fp32
                     result; y_bf16 == RNE(y_f32) bit for bit              */
} nvfp4_dtype;

/* nvfp4_quantize flag: read *global_scale instead of computing it from the
 * data (static, ahead-of-time scale); the amax pass is skipped. */
#define NVFP4_GLOBAL_SCALE_GIVEN 1u

/* Human-readable name of a status code (static string, never NULL). */
const char* nvfp4_status_string(int status);

/* Library version as "major.minor.patch" (static string). */
const char* nvfp4_version(void);

/* Bytes of device workspace nvfp4_quantize needs for x of [rows, cols]
 * (partial maxima of the amax pass).  0 when rows*cols == 0. */
size_t nvfp4_quantize_workspace_bytes(int64_t rows, int64_t cols);

/*
 * Quantise x [rows, cols] (row stride ld_x elements, dtype F32 or BF16) to
 * NVFP4: q [rows, cols/2], s [rows, cols/16] (both dense), *global_scale.
 *
 * Steps (exact reals, each stored quantity rounded once):
 *   g      = fl32(max|x| / 2688)                       (2688 = 448 * 6)
 *   s_b    = E4M3 nearest-even, saturating at 448, of max_{i in b}|x_i| / (6 g)
 *   code_i = E2M1 nearest-even, saturating at 6, of |x_i| / (E4M3(s_b) g)
 *   nibble = signbit(x_i) << 3 | code_i
 * A zero tensor gives g = 0, all scale bytes 0 and magnitude codes 0; a
 * block whose scale byte is 0 gets magnitude codes 0.  Output is unique:
 * the bytes equal the CPU definition exactly.
 *
 * Requirements: cols % 16 == 0; ld_x >= cols; x 16-byte aligned and
 * ld_x * sizeof(elem) % 16 == 0 (else NVFP4_ERR_UNSUPPORTED); q 8-byte
 * aligned.  workspace >= nvfp4_quantize_workspace_bytes(rows, cols) bytes,
 * 4-byte aligned (may be NULL when flags has NVFP4_GLOBAL_SCALE_GIVEN).
 * flags & NVFP4_GLOBAL_SCALE_GIVEN: *global_scale (device) is read, not
 * written; it must be finite and >= 0.
 */
int nvfp4_quantize(const void* x, nvfp4_dtype x_dtype, int64_t rows, int64_t cols,
                   int64_t ld_x, uint8_t* q, uint8_t* s, float* global_scale,
                   unsigned flags, void* workspace, size_t workspace_bytes,
                   void* stream);

/*
 * nvfp4_quantize for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments, results and errors as nvfp4_quantize, without the
 * workspace: the amax pass keeps its partial maxima (at most 4 KB) in a
 * device array of the library's own, one per GPU, held until the process
 * ends; the call allocates nothing.  Every call on one GPU shares that
 * array, so calls that overlap on a GPU (concurrent streams, other host
 * threads) race and must be ordered by the caller.  Shapes whose partial
 * maxima would not fit return NVFP4_ERR_UNSUPPORTED (none do: the amax
 * pass runs at most 1024 workgroups).  The first call on a device looks up
 * the array's address there (no allocation); a failure of that lookup
 * returns NVFP4_ERR_HIP.
 */
int nvfp4_quantize_noalloc(const void* x, nvfp4_dtype x_dtype, int64_t rows, int64_t cols,
                           int64_t ld_x, uint8_t* q, uint8_t* s, float* global_scale,
                           unsigned flags, void* stream);

/*
 * Dense NVFP4 GEMM (kernelindex, "NVFP4 linear layer"): for m < M, n < N
 *   y[m, n] = fl32(a_g * b_g) * sum_{k<K} A(m, k) * B(n, k)
 * with A(m, k) = E2M1(a_q nibble (m, k)) * E4M3(a_s[m, k/16]) and B the same
 * for b = W [N, K].  Products are formed exactly and accumulated in fp32;
 * |y - y_exact| <= 1e-5 * sum_k |x_k w_k| per element (plus one bf16 ulp for
 * BF16 output).  a_g and b_g are DEVICE pointers to one fp32 each, so a
 * quantise -> GEMM chain needs no host round-trip.
 *
 * a_q [M, K/2], a_s [M, K/16], b_q [N, K/2], b_s [N, K/16] are dense.
 * y [M, N] has row stride ld_y >= N elements of y_dtype.
 * Any M, N >= 0; K % 16 == 0.  Shapes are dispatched to a decode kernel
 * (M <= 128), an MFMA tile kernel, or a general kernel for unaligned K.
 */
int nvfp4_gemm(int64_t M, int64_t N, int64_t K,
               const uint8_t* a_q, const uint8_t* a_s, const float* a_g,
               const uint8_t* b_q, const uint8_t* b_s, const float* b_g,
               void* y, nvfp4_dtype y_dtype, int64_t ld_y, void* stream);

/*
 * Dense NVFP4 GEMM whose output is NVFP4 again: the next layer's input
 * quantisation done in this GEMM's epilogue with a static global scale fixed
 * ahead of time (leverageai "blackwell-nvfp4-gemm-optimization", "What is
 * this?": quantisation may happen before execution), so y never makes a
 * round trip through HBM in a wide type.
 *   y[m, n] = the fp32 value nvfp4_gemm stores with y_dtype NVFP4_F32
 *   (y_q, y_s) = the encoding of y by nvfp4_quantize's steps with g = *y_g
 *                (the bytes nvfp4_quantize with NVFP4_GLOBAL_SCALE_GIVEN
 *                would write from that fp32 y, exactly)
 * y_q [M, N/2] and y_s [M, N/16] are dense (row strides N/2 and N/16
 * bytes); y_q is 8-byte aligned.  y_g is a DEVICE fp32 scalar, read only;
 * it must be finite and >= 0 (0 gives scale bytes 0 and magnitude codes 0).
 * Values whose magnitude exceeds 2688 * g saturate (scale 448, code 6).
 * N % 16 == 0 (NVFP4_ERR_INVALID_ARG otherwise); the other requirements and
 * the kernel dispatch are those of nvfp4_gemm.
 */
int nvfp4_gemm_nvfp4_out(int64_t M, int64_t N, int64_t K,
                         const uint8_t* a_q, const uint8_t* a_s, const float* a_g,
                         const uint8_t* b_q, const uint8_t* b_s, const float* b_g,
                         uint8_t* y_q, uint8_t* y_s, const float* y_g, void* stream);

/*
 * Grouped (per-expert) NVFP4 GEMM for mixture-of-experts layers whose
 * experts each see a small, uneven number of tokens (magik.net "The Moment
 * of Synthesis", "The Reasoning Process": grouped GEMM is the lever for tiny
 * per-expert batches).  Rows of A are sorted by group: group e owns rows
 * [m_offsets[e], m_offsets[e+1]) and multiplies them by its own weight
 *   B_e = (b_q + e*N*K/2 [N, K/2], b_s + e*N*K/16 [N, K/16], b_g[e]).
 *   y[r, n] = fl32(*a_g * b_g[e]) * sum_k A(r, k) * B_e(n, k)
 * m_offsets: DEVICE int32 [G+1], non-decreasing, m_offsets[0] = 0,
 * m_offsets[G] = total_m (the host copy of the last entry).  Empty groups
 * are allowed.  b_g: DEVICE fp32 [G]; a_g: DEVICE fp32 scalar.
 * y [total_m, N] with row stride ld_y, rows in A's order.  K % 16 == 0.
 * Monotonicity of m_offsets is a documented precondition: rows outside
 * [0, total_m) are never read or written even if it is violated.
 */
int nvfp4_grouped_gemm(int32_t G, const int32_t* m_offsets, int64_t total_m,
                       int64_t N, int64_t K,
                       const uint8_t* a_q, const uint8_t* a_s, const float* a_g,
                       const uint8_t* b_q, const uint8_t* b_s, const float* b_g,
                       void* y, nvfp4_dtype y_dtype, int64_t ld_y, void* stream);

/*
 * The same grouped GEMM reading its activation rows through an index list
 * instead of a pre-gathered copy (the routing step of a mixture-of-experts
 * layer, "The Moment of Synthesis", "The Reasoning Process": tokens are sent
 * to their experts before the grouped GEMM).  Grouped row r (expert-sorted,
 * m_offsets as above) multiplies activation row row_index[r] of
 * a [a_rows, K/2] / [a_rows, K/16]; y [total_m, N] keeps the grouped order.
 * row_index: DEVICE int32 [total_m]; an index outside [0, a_rows) reads as a
 * row of zeros.  Indices may repeat (a token routed to several experts).
 * Otherwise as nvfp4_grouped_gemm (a_rows = total_m and row_index[r] = r give
 * the same result).  Errors: NVFP4_ERR_INVALID_ARG also for a_rows < 0 or a
 * null row_index with total_m > 0.
 */
int nvfp4_grouped_gemm_gather(int32_t G, const int32_t* m_offsets, const int32_t* row_index,
                              int64_t total_m, int64_t a_rows, int64_t N, int64_t K,
                              const uint8_t* a_q, const uint8_t* a_s, const float* a_g,
                              const uint8_t* b_q, const uint8_t* b_s, const float* b_g,
                              void* y, nvfp4_dtype y_dtype, int64_t ld_y, void* stream);

/*
 * Several independent grouped GEMMs in one launch.  A mixture-of-experts
 * layer runs its gate_up and down projections as grouped GEMMs over the
 * same routing ("The Moment of Synthesis", "The Reasoning Process":
 * grouping is the lever for tiny per-expert batches; "The Moment of
 * Recalibration", "The Broader Narrative Arc": persistent grouped kernels);
 * one persistent launch over the union of their (expert, weight tile) work
 * shares the launch ramp, the per-CU fill and the tail.  The projections
 * are independent here (each has its own activation; the operation between
 * them is outside this library).
 *
 * Each element of `problems` (a HOST array of `count` entries, 0 <= count
 * <= NVFP4_GROUPED_MAX_PROBLEMS) describes one call with exactly the
 * meaning of nvfp4_grouped_gemm (row_index == NULL) or
 * nvfp4_grouped_gemm_gather (row_index != NULL, a_rows = rows of a); with
 * row_index == NULL, a_rows must be 0 or total_m.  Results are those of
 * the separate calls, bit for bit.  Outputs of different problems must not
 * overlap.  Every problem is validated before anything is enqueued; any
 * error leaves all outputs untouched.  Problems the streaming kernel cannot
 * take (K % 512 != 0, unaligned rows, operands of 4 GiB or more) make the
 * call run each problem on its own.
 */
#define NVFP4_GROUPED_MAX_PROBLEMS 4

typedef struct {
  int32_t G;                  /* groups (experts)                                */
  const int32_t* m_offsets;   /* DEVICE int32 [G+1]                              */
  const int32_t* row_index;   /* DEVICE int32 [total_m], or NULL                 */
  int64_t total_m;            /* m_offsets[G]                                    */
  int64_t a_rows;             /* rows of a when row_index != NULL                */
  int64_t N, K;
  const uint8_t* a_q;         /* [a_rows, K/2]  (total_m rows without row_index) */
  const uint8_t* a_s;         /* [a_rows, K/16]                                  */
  const float* a_g;           /* DEVICE fp32 scalar                              */
  const uint8_t* b_q;         /* [G, N, K/2]                                     */
  const uint8_t* b_s;         /* [G, N, K/16]                                    */
  const float* b_g;           /* DEVICE fp32 [G]                                 */
  void* y;                    /* [total_m, N], row stride ld_y                   */
  nvfp4_dtype y_dtype;
  int64_t ld_y;
} nvfp4_grouped_problem;

int nvfp4_grouped_gemm_multi(int32_t count, const nvfp4_grouped_problem* problems,
                             void* stream);

/*
 * MXFP4 variant: 32-element blocks with power-of-two (E8M0) scales, the
 * block shape the gfx950 scaled FP4 matrix instruction consumes natively,
 * so the products need no dequantisation.  The pages define NVFP4 only
 * (FP4 packs twice the values of FP8 and four times those of FP16: magik.net
 * "The 3.7 PFLOPS Revelation", "Input Knowledge", item 2); this format
 * follows the microscaling definition and shows the 4-bit format's compute
 * ceiling on this hardware.
 *
 * nvfp4_mxfp4_quantize: x (fp32 | bf16) [rows, cols], row stride ld_x
 * elements -> q [rows, cols/2] (element 2j in the low nibble of byte j) and
 * s [rows, cols/32] E8M0 bytes (value 2^(b - 127); 255 is NaN), all DEVICE.
 * Per 32-element block: E = floor(log2(amax)) - 2 clamped to [-127, 127]
 * (-127 for a zero block), s = E + 127, each element the E2M1 rounding
 * (nearest, ties to the even code, saturating at 6, sign kept) of x / 2^E;
 * a block holding a NaN or an infinity gets s = 255 and zero nibbles.  One
 * pass, no workspace, deterministic.
 * Errors: NVFP4_ERR_INVALID_ARG for cols % 32 != 0, negative sizes, a bad
 * dtype, ld_x < cols or a null pointer with rows, cols > 0;
 * NVFP4_ERR_UNSUPPORTED for x or its rows not 16-byte aligned, q not
 * 16-byte aligned, or a dimension above 2^30.
 */
int nvfp4_mxfp4_quantize(const void* x, nvfp4_dtype x_dtype, int64_t rows, int64_t cols,
                         int64_t ld_x, uint8_t* q, uint8_t* s, void* stream);

/*
 * y[m, n] = sum_k A(m, k) * B(n, k) with MXFP4 operands A = (a_q [M, K/2],
 * a_s [M, K/32]) and B = W = (b_q [N, K/2], b_s [N, K/32]), all DEVICE; no
 * per-tensor scale.  y [M, N] (fp32 or bf16, round to nearest even), row
 * stride ld_y.  fp32 accumulation; a NaN scale byte gives NaN outputs; terms
 * below fp32's subnormal range are lost.  K % 128 == 0 with 16-byte aligned
 * nibble rows and 4-byte aligned scale rows runs on the scaled FP4 matrix
 * instruction; other shapes run a general kernel.  K == 0 writes zeros.
 * Errors: NVFP4_ERR_INVALID_ARG for K % 32 != 0, negative sizes, a bad
 * y_dtype, ld_y < N or a null pointer; NVFP4_ERR_UNSUPPORTED for a
 * dimension above 2^30.
 */
int nvfp4_mxfp4_gemm(int64_t M, int64_t N, int64_t K, const uint8_t* a_q, const uint8_t* a_s,
                     const uint8_t* b_q, const uint8_t* b_s, void* y, nvfp4_dtype y_dtype,
                     int64_t ld_y, void* stream);

/*
 * FP8 operands: E4M3FN bytes with one fp32 scale per block of 128 elements
 * of K, for the layers a 4-bit format is too coarse for and for training.
 *   q  uint8 [rows, K]   E4M3FN bit patterns, dense rows
 *   s  fp32  [ceil(K/128), ceil(rows/block_rows)]
 *      block_rows 1: a scale per row and block; block_rows 128: per 128 x 128
 *   an element decodes as E4M3(q[r, k]) * s[k / 128, r / block_rows]
 * The last block of a row (of 128 rows) may be shorter.
 *
 * nvfp4_fp8_quantize: x [batch, rows, cols] (matrix b starts at row b * rows,
 * row stride ld_x elements, F32 or BF16) -> either or both of
 *   rows layout  q [batch, rows, cols], s of blocks along the rows: the
 *                operand of a product over cols;
 *   transposed   qt [batch, cols, rows_t], st of blocks along the columns,
 *                rows_t = rows rounded up to 16 (bytes past rows are zero):
 *                the operand of a product over rows, as the gradients need.
 * Per block: A = max(max|x|, 2^-100), s = fl32(A / 448), and each byte is the
 * E4M3 rounding (nearest, ties to even) of fl32(x * fl32(448 / A)).  A block
 * holding a NaN or an infinity gets a NaN scale and zero bytes.  With
 * block_rows 128 both layouts hold the same values.  One pass over x, no
 * workspace, deterministic.
 * Errors: NVFP4_ERR_INVALID_ARG for cols % 16 != 0, block_rows not 1 or 128,
 * negative sizes, a bad dtype, ld_x < cols, one pointer of a pair (q, s) or
 * (qt, st) without the other, both pairs null, or a null x;
 * NVFP4_ERR_UNSUPPORTED for x, its rows, q or qt not 16-byte aligned, a
 * dimension above 2^30, or sizes whose launch would pass 2^32 threads (here
 * and in the products below: from about 2^22 blocks or tiles of outputs on).
 */
int nvfp4_fp8_quantize(const void* x, nvfp4_dtype x_dtype, int64_t batch, int64_t rows,
                       int64_t cols, int64_t ld_x, int block_rows, uint8_t* q, float* s,
                       uint8_t* qt, float* st, void* stream);

/* Columns P of an expert-wise transposed operand of total_m tokens in G
 * groups (below): 128 * floor((total_m + 127 * min(G, total_m)) / 128). */
int64_t nvfp4_fp8_grouped_columns(int64_t total_m, int32_t G);

/*
 * The same quantisation (block_rows 1) of rows sorted by group, m_offsets as
 * in nvfp4_grouped_gemm (here m_offsets[G] <= total_m; rows of no group are
 * not read, and q, s are left as they were there):
 *   rows layout  q [total_m, cols], s [ceil(cols/128), total_m]
 *   transposed   qt [cols, P], st [P/128, cols]: each group's tokens start at
 *                the next multiple of 128 columns, so that no block mixes
 *                groups; columns of no token are zero.
 * row_index (or NULL): grouped row r is row row_index[r] of x [x_rows, cols];
 * an index outside [0, x_rows) is a row of zeros.  Without it x has total_m
 * rows and x_rows is not read.  Errors as above, and NVFP4_ERR_UNSUPPORTED for
 * G > 2^31 - 65.
 */
int nvfp4_fp8_grouped_quantize(const void* x, nvfp4_dtype x_dtype, int32_t G,
                               const int32_t* m_offsets, const int32_t* row_index,
                               int64_t total_m, int64_t x_rows, int64_t cols, int64_t ld_x,
                               uint8_t* q, float* s, uint8_t* qt, float* st, void* stream);

/* nvfp4_fp8_gemm / nvfp4_fp8_grouped_wgrad flag: y += product (F32 y). */
#define NVFP4_ACCUMULATE 1u

/*
 * y[m, n] (+)= sum_k A(m, k) * B(n, k) of FP8 operands a [M, K] (block_rows 1)
 * and b [N, K] (b_block_rows 1 or 128).  A linear layer's three products:
 *   y  = x . W^T       a = x (rows),           b = W (128, rows)
 *   dx = dy . W        a = dy (rows),          b = W (128, transposed)
 *   dW = dy^T . x      a = dy (transposed),    b = x (transposed)
 * Each block's products are summed, and the block's sum is multiplied by
 * sa * sb (rounded to fp32 first: it must be finite, and below 2^-126 it is
 * a multiple of 2^-149) as it is added to the result in fp32.  With an F32 y
 * a block's own sum is fp32 as well.  With a BF16 y it may come from the 8-bit
 * matrix instructions, which align a block's products to the largest of their
 * running sums and cut each 2^-16 below it: a block is then off by at most
 * 2^-9 of the sum of its |A B|.  For data without outliers that is about
 * 1.5e-5 of the result, far below the rounding to BF16; where large products
 * cancel it can be all of it.  A caller who needs fp32 sums there asks for an
 * F32 y.
 * y [M, N] has row stride ld_y >= N elements.  A NaN scale gives NaN in the
 * rows (columns) it scales.  K == 0 writes zeros (adds nothing).
 * Errors: NVFP4_ERR_INVALID_ARG for K % 16 != 0, b_block_rows not 1 or 128,
 * negative sizes, a bad dtype or flag, NVFP4_ACCUMULATE with a BF16 y,
 * ld_y < N or a null pointer; NVFP4_ERR_UNSUPPORTED for q not 16-byte
 * aligned, s or y not aligned to their elements, K > 2^22, another dimension
 * above 2^30, or sizes whose launch would pass 2^32 threads.
 */
int nvfp4_fp8_gemm(int64_t M, int64_t N, int64_t K, const uint8_t* a_q, const float* a_s,
                   const uint8_t* b_q, const float* b_s, int b_block_rows, void* y,
                   nvfp4_dtype y_dtype, int64_t ld_y, unsigned flags, void* stream);

/*
 * Experts' products: group e's rows of a times its own weight
 * (b_q + e*N*K, b_s [G, ceil(K/128), ceil(N/128)]), as nvfp4_grouped_gemm and
 * (with row_index, a [a_rows, K]) nvfp4_grouped_gemm_gather; here
 * m_offsets[G] <= total_m is allowed, and rows of y of no group are left as
 * they were.  Without row_index a has total_m rows and a_rows must be 0 or
 * total_m.  The input gradient is the same call with dy and the transposed
 * weights.  Sums and errors as nvfp4_fp8_gemm, and NVFP4_ERR_UNSUPPORTED for
 * G > 2^31 - 65, or a_rows * K >= 2^31 with row_index.
 */
int nvfp4_fp8_grouped_gemm(int32_t G, const int32_t* m_offsets, const int32_t* row_index,
                           int64_t total_m, int64_t a_rows, int64_t N, int64_t K,
                           const uint8_t* a_q, const float* a_s, const uint8_t* b_q,
                           const float* b_s, void* y, nvfp4_dtype y_dtype, int64_t ld_y,
                           void* stream);

/*
 * Experts' weight gradients: dw[e, n, k] (+)= sum over group e's tokens of
 * dy[r, n] * x[r, k], from the transposed operands of
 * nvfp4_fp8_grouped_quantize: a = dy (a_q [N, P], a_s [P/128, N]) and b = x
 * (b_q [K, P], b_s [P/128, K]), P = nvfp4_fp8_grouped_columns(total_m, G).
 * dw [G, N, K] is dense; a group without tokens gets zeros (is left alone
 * with NVFP4_ACCUMULATE).  N, K >= 0 of any size.  Sums and errors as
 * nvfp4_fp8_gemm (P in the place of K).
 */
int nvfp4_fp8_grouped_wgrad(int32_t G, const int32_t* m_offsets, int64_t total_m, int64_t N,
                            int64_t K, const uint8_t* a_q, const float* a_s, const uint8_t* b_q,
                            const float* b_s, void* dw, nvfp4_dtype dw_dtype, unsigned flags,
                            void* stream);

/* Activation of a gated block: act(g) = g sigma(z), with z = g (SILU) or
 * z = 2 sqrt(2/pi) (g + 0.044715 g^3) (GELU, the tanh form), in fp32: sigma has
 * the bits of a subnormal number below 2^-126 and is 0 from 2^-150 on.  Of an
 * infinite g act is g or (-infinity) NaN, and act' NaN. */
typedef enum {
  NVFP4_SILU = 0,
  NVFP4_GELU = 1
} nvfp4_act;

/*
 * Gated feed-forward block, first half: h = act(x Wg^T) * (x Wu^T) [M, F] in one
 * product of the FP8 operands a = x [M, K] (block_rows 1) and w = [Wg; Wu]
 * [2F, K] (gate rows first; w_block_rows 1 or 128; F of any size, though a
 * block of 128 rows that ends inside the gate's last 32 costs some time).
 * Both products are summed as in nvfp4_fp8_gemm with an output of h's type: an
 * F32 h has fp32 sums; with a BF16 h either factor may be off by what that call
 * states of the 8-bit instructions, before act and the product, and by up to 16 rows
 * (which keep fp32 sums) a row of h can differ from its value in a larger batch.
 * They stay in fp32 up to h, which is rounded once.  gate_up (or NULL): bf16
 * [M, 2F], the two products for the backward, which is that of the rounded ones.
 * h (F32 or BF16) has row stride ld_h >= F, gate_up ld_gate_up >= 2F elements.
 * K == 0 writes zeros.
 * Errors as nvfp4_fp8_gemm (2F in the place of N), and
 * NVFP4_ERR_INVALID_ARG for a bad act, NVFP4_ERR_UNSUPPORTED for F > 2^27.
 */
int nvfp4_fp8_gated_gemm(int64_t M, int64_t F, int64_t K, const uint8_t* a_q, const float* a_s,
                         const uint8_t* w_q, const float* w_s, int w_block_rows, nvfp4_act act,
                         void* h, nvfp4_dtype h_dtype, int64_t ld_h, void* gate_up,
                         int64_t ld_gate_up, void* stream);

/*
 * The same per expert: group e's rows of a times w_q + e*2F*K,
 * w_s [G, ceil(K/128), ceil(2F/128)] (block_rows 128), with m_offsets, row_index
 * and a_rows as in nvfp4_fp8_grouped_gemm.  Rows of h and gate_up of no group
 * are left as they were.  NVFP4_ERR_UNSUPPORTED for G > 2^30 too.
 */
int nvfp4_fp8_grouped_gated_gemm(int32_t G, const int32_t* m_offsets, const int32_t* row_index,
                                 int64_t total_m, int64_t a_rows, int64_t F, int64_t K,
                                 const uint8_t* a_q, const float* a_s, const uint8_t* w_q,
                                 const float* w_s, nvfp4_act act, void* h, nvfp4_dtype h_dtype,
                                 int64_t ld_h, void* gate_up, int64_t ld_gate_up, void* stream);

/*
 * Its backward: from dh [rows, F] and gate_up = [g, u] [rows, 2F] (F32 or BF16
 * each)
 *   dg = dh u act'(g),   du = dh act(g)
 * as the FP8 operand [dg, du] [rows, 2F] of the products that follow, in either
 * or both layouts of nvfp4_fp8_quantize (block_rows 1):
 *   dx = [dg, du] . W       a = rows layout, b = W (128, transposed [K, 2F])
 *   dW = [dg, du]^T . x     a = transposed,  b = x (transposed)
 * dg and du are fp32 up to that quantisation.
 * Errors: NVFP4_ERR_INVALID_ARG for F % 8 != 0, negative sizes, a bad dtype or
 * act, a row stride below the row, one pointer of a pair without the other,
 * both pairs null, or a null input; NVFP4_ERR_UNSUPPORTED for inputs, their
 * rows, q or qt not 16-byte aligned, F > 2^27, rows above 2^30, or sizes whose
 * launch would pass 2^32 threads.
 */
int nvfp4_fp8_gated_backward(const void* dh, nvfp4_dtype dh_dtype, int64_t ld_dh,
                             const void* gate_up, nvfp4_dtype gate_up_dtype, int64_t ld_gate_up,
                             nvfp4_act act, int64_t rows, int64_t F, uint8_t* q, float* s,
                             uint8_t* qt, float* st, void* stream);

/*
 * The same for rows sorted by group: layouts, padding columns and rows of no
 * group as in nvfp4_fp8_grouped_quantize (cols = 2F), for
 * nvfp4_fp8_grouped_gemm and nvfp4_fp8_grouped_wgrad.  NVFP4_ERR_UNSUPPORTED
 * for G > 2^30 too.
 */
int nvfp4_fp8_grouped_gated_backward(int32_t G, const int32_t* m_offsets, const void* dh,
                                     nvfp4_dtype dh_dtype, int64_t ld_dh, const void* gate_up,
                                     nvfp4_dtype gate_up_dtype, int64_t ld_gate_up, nvfp4_act act,
                                     int64_t total_m, int64_t F, uint8_t* q, float* s, uint8_t* qt,
                                     float* st, void* stream);

/*
 * 8-bit integers with one fp32 scale per row, for serving: exact sums, and a
 * scale for each token and each output channel.
 *   q  int8 [rows, K]  dense rows
 *   s  fp32 [rows]     an element decodes as q[r, k] * s[r]
 *
 * nvfp4_int8_quantize: x [rows, cols] (F32 or BF16, row stride ld_x) -> q, s.
 * Per row: A = max(max|x|, 2^-100), s = fl32(A / 127), each q is
 * fl32(x * fl32(127 / A)) rounded to the nearest integer, ties to even.  A row
 * holding a NaN or an infinity gets a NaN scale and zeros; a row of no columns
 * has the scale of a zero row.  Deterministic.
 * Errors: NVFP4_ERR_INVALID_ARG for cols % 16 != 0, negative sizes, a bad
 * dtype, ld_x < cols or a null pointer; NVFP4_ERR_UNSUPPORTED for x, its rows
 * or q not 16-byte aligned, s not 4-byte aligned, a dimension above 2^30, or
 * sizes whose launch would pass 2^32 threads.
 */
int nvfp4_int8_quantize(const void* x, nvfp4_dtype x_dtype, int64_t rows, int64_t cols,
                        int64_t ld_x, int8_t* q, float* s, void* stream);

/*
 * y[m, n] = fl32(sum_k a_q[m, k] b_q[n, k]) * a_s[m] * b_s[n] (in this order) of
 * INT8 operands a [M, K] and b = W [N, K].  The sum is an exact 32-bit integer.
 * y [M, N] (F32 or BF16) has row stride ld_y >= N.  A NaN scale gives NaN in
 * its row (column), for K == 0 too, whose sums are 0.
 * Errors: NVFP4_ERR_INVALID_ARG for K % 16 != 0, negative sizes, a bad dtype,
 * ld_y < N or a null pointer; NVFP4_ERR_UNSUPPORTED for q not 16-byte aligned,
 * s or y not aligned to their elements, K >= 2^17 (where a sum could pass 32
 * bits), another dimension above 2^30, or sizes whose launch would pass 2^32
 * threads.
 */
int nvfp4_int8_gemm(int64_t M, int64_t N, int64_t K, const int8_t* a_q, const float* a_s,
                    const int8_t* b_q, const float* b_s, void* y, nvfp4_dtype y_dtype,
                    int64_t ld_y, void* stream);

/* One gradient of a list: n dense elements at g, and where its clipped values
 * go (out NULL or g: in place, out_dtype then being g_dtype). */
typedef struct nvfp4_grad {
  void* g;   /* DEVICE */
  void* out; /* DEVICE */
  int64_t n;
  nvfp4_dtype g_dtype;
  nvfp4_dtype out_dtype;
} nvfp4_grad;

/* Bytes of device workspace of the two calls below for a list of `count`. */
size_t nvfp4_grad_workspace_bytes(int64_t count);

/*
 * Sum of the squares of all elements of a list of gradients -> norm_sq (DEVICE,
 * one IEEE binary64).  `grads` is a HOST array, read before the call returns;
 * `out` is not read.  Squares and sums are binary64, so nothing finite
 * overflows; their order depends on the list's sizes, types and addresses
 * alone; a tensor listed twice counts twice.  A caller whose gradients are
 * spread over processes adds their sums before it clips.  workspace:
 * nvfp4_grad_workspace_bytes(count) bytes or more, 8-byte aligned, not shared by
 * calls that may overlap.  count == 0 writes 0.
 * Errors: NVFP4_ERR_INVALID_ARG for count < 0, n < 0, a bad dtype, a null
 * pointer (g only where n > 0), or a workspace that is too small or overlaps a
 * gradient;
 * NVFP4_ERR_UNSUPPORTED for pointers not aligned to their elements, or more
 * than 2^42 elements or 2^20 tensors.
 */
int nvfp4_grad_norm_sq(int64_t count, const nvfp4_grad* grads, double* norm_sq, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * out = g * c with c = max_norm / norm where norm > max_norm, else 1, and
 * norm = sqrt(norm_sq).  norm_sq (DEVICE, or NULL: it is computed from the list)
 * may be a sum over several processes.  norm (DEVICE fp32, or NULL) receives the
 * norm before clipping.  c and the product are binary64, rounded to fp32 (and
 * from there to bf16) as out is written.  With c == 1 gradients in place are not
 * touched, others are copied; a norm_sq that is not finite counts as c == 1, so
 * that a step can be dropped by looking at norm.  max_norm >= 0 (infinity: never
 * clips).
 * Errors: as above, and NVFP4_ERR_INVALID_ARG for max_norm < 0 or NaN, types
 * that differ in place (of n > 0), a written tensor that overlaps another of the
 * list; for norm or the workspace overlapping a tensor of the list, norm_sq one
 * that is written, or norm overlapping the workspace or norm_sq.  workspace may be
 * NULL where norm_sq is given, and is not used then.
 */
int nvfp4_clip_grads(int64_t count, const nvfp4_grad* grads, double max_norm,
                     const double* norm_sq, float* norm, void* workspace, size_t workspace_bytes,
                     void* stream);

/* nvfp4_moe_route flag: weights are the softmax over the chosen experts. */
#define NVFP4_ROUTE_RENORMALIZE 1u

/* Bytes of device workspace of nvfp4_moe_route. */
size_t nvfp4_moe_route_workspace_bytes(int64_t T, int64_t E);

/*
 * Router of a mixture of experts: logits [T, E] (F32 or BF16, row stride
 * ld_logits elements) -> for each token its topk experts, and what the
 * grouped GEMMs take.
 *   p[t, :]      = softmax(logits[t, :])
 *   expert_index int32 [T, topk]  experts of the largest logits, descending,
 *                ties (-0 and +0 too) to the lowest expert
 *   weights      fp32 [T, topk]   p at those (or, renormalised, their softmax)
 *   counts       int32 [E]        tokens of each expert
 *   m_offsets    int32 [E + 1]    their running sums
 *   row_index    int32 [T * topk] token of each grouped row, sorted by
 *                (expert, token); -1 behind m_offsets[E]
 *   pair_row     int32 [T, topk]  grouped row of each choice
 *   routed       int32 [1]        n, tokens that chose any expert
 *   loss         fp32 [1]         E * sum_e (counts_e / (n topk)) (1/n sum_t p[t, e]),
 *                1 for an even load; 0 when n == 0
 * token_mask (uint8 [T], or NULL): a token with 0 chooses nothing and counts
 * nowhere.  An expert at -inf is never chosen; choices that are left over
 * are expert -1, weight 0, pair_row -1.  Other logits must be finite.
 * Probabilities and sums are fp32 or wider, in an order that does not change
 * between calls.  T == 0 writes counts, m_offsets, routed and loss.
 * workspace >= nvfp4_moe_route_workspace_bytes(T, E) bytes, 4-byte aligned,
 * not shared by calls that may overlap.
 * Errors: NVFP4_ERR_INVALID_ARG for T < 0, E < 1, topk < 1 or > E, a bad
 * dtype or flag, ld_logits < E, a null pointer or a workspace too small;
 * NVFP4_ERR_UNSUPPORTED for E > 1024, topk > 16, T * topk >= 2^31, or
 * pointers not aligned to their elements.
 */
int nvfp4_moe_route(int64_t T, int64_t E, int32_t topk, const void* logits,
                    nvfp4_dtype logits_dtype, int64_t ld_logits, const uint8_t* token_mask,
                    unsigned flags, int32_t* expert_index, float* weights, int32_t* counts,
                    int32_t* m_offsets, int32_t* row_index, int32_t* pair_row, int32_t* routed,
                    float* loss, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradient of the logits of nvfp4_moe_route (same logits, mask and flags, and
 * its expert_index, counts and routed) from d_weights fp32 [T, topk] and
 * d_loss fp32 [1] (device; either may be NULL for none).  counts are
 * constants of the loss.  d_logits [T, E] has the logits' dtype and row
 * stride ld_d >= E; rows of tokens that chose nothing are zero.  d_weights
 * of left-over choices are not read.  T == 0 enqueues nothing.
 */
int nvfp4_moe_route_backward(int64_t T, int64_t E, int32_t topk, const void* logits,
                             nvfp4_dtype logits_dtype, int64_t ld_logits,
                             const uint8_t* token_mask, unsigned flags,
                             const int32_t* expert_index, const int32_t* counts,
                             const int32_t* routed, const float* d_weights, const float* d_loss,
                             void* d_logits, int64_t ld_d, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_H_ */
