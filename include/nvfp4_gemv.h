/*
 * nvfp4_gemv.h -- C ABI of the MI355X (gfx950) NVFP4 block-scaled batched GEMV,
 * of the FP4 linear layers and routed experts around it, and of attention over a
 * paged NVFP4 key/value cache (last parts).
 *
 * Operation (kernelbot NVFP4 GEMV, submission 103289, `cute_kernel`: each k
 * contributes a * sfa * b * sfb, the contributions of one output row are
 * accumulated in float32 and the sum is cast to float16):
 *
 *   c[l][m] = fp16( sum_{k<K} e2m1(A[l][m][k]) * e4m3(SFA[l][m][k/16])
 *                            * e2m1(B[l][k])    * e4m3(SFB[l][k/16]) )
 *
 * for m < M, l < L (N = 1). Element format: E2M1 (Float4E2M1FN), packed two per
 * byte along k, the even k in the low nibble. Scale format: E4M3 (Float8E4M3FN),
 * one scale per 16 consecutive k. Accumulation is float32; the cast to float16
 * rounds to nearest even and overflows to +-inf. Summation order inside a row
 * is the library's own (all products are exact; partial sums round in float32),
 * and it does not depend on the scale layout.
 *
 * Memory order of every operand is batch-outermost and dense (the CuTe layouts
 * of submission 103289 `cute_jit_kernel`: A stride (K, 1, M*K), C stride
 * (1, 1, M)):
 *
 *   a    uint8  [L][M][K/2]     packed E2M1 codes of A
 *   b    uint8  [L][K/2]        packed E2M1 codes of the vector B
 *   c    fp16   [L][M]          output (IEEE binary16 bits), written
 *   sfa, sfb in one of two layouts, chosen by sf_layout for both:
 *     NVFP4_SF_PLAIN:   sfa uint8 [L][M][K/16], sfb uint8 [L][K/16]
 *     NVFP4_SF_BLOCKED: the 128x4 blocked ("permuted") layout of submission
 *       69953 `to_blocked_batch` (equivalently submission 69575
 *       `blocked_transform_kernel`, and the 6-D tensor of submission 103289
 *       `permuted_to_blocked`), per batch, batches back to back:
 *         scale (r, kb) of a rows x (K/16) matrix is at byte
 *           ((r/128)*ceil(K/64) + kb/4)*512 + (r%32)*16 + ((r%128)/32)*4 + kb%4
 *         sfa: rows = M, ceil(M/128)*ceil(K/64)*512 bytes per batch
 *         sfb: rows = 1, ceil(K/64)*512 bytes per batch (B padded to 128 rows)
 *       Padding bytes (rows >= M, columns >= K/16) are never read.
 *
 * Conventions shared by all entry points:
 *   - a, b, sfa, sfb, c and workspace are DEVICE pointers owned by the caller;
 *     the library keeps no reference to them after the call returns.
 *   - Calls only enqueue work on `stream` (a hipStream_t; NULL = the null
 *     stream) and never synchronise. Faults inside the kernel surface later on
 *     the stream.
 *   - Every argument is validated before any HIP call; on failure nothing is
 *     launched and a nonzero nvfp4_status_t is returned.
 *   - Requirements: M, K, L >= 1; K % 32 == 0; L*M*K/2 < 2^62; a, b and sfa
 *     16-byte aligned; sfb 4-byte aligned; c 2-byte aligned.
 */
#ifndef NVFP4_GEMV_H
#define NVFP4_GEMV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    NVFP4_SF_PLAIN = 0,
    NVFP4_SF_BLOCKED = 1
} nvfp4_sf_layout_t;

typedef enum {
    NVFP4_OK = 0,
    NVFP4_ERR_NULL_POINTER = 1,     /* a required pointer is NULL                 */
    NVFP4_ERR_INVALID_SHAPE = 2,    /* M, K or L out of range, or K % 32 != 0      */
    NVFP4_ERR_MISALIGNED = 3,       /* a pointer misses its required alignment     */
    NVFP4_ERR_INVALID_LAYOUT = 4,   /* sf_layout is not an nvfp4_sf_layout_t       */
    NVFP4_ERR_WORKSPACE = 5,        /* workspace missing, misaligned or too small  */
    NVFP4_ERR_HIP = 6,              /* a HIP call failed; see nvfp4_last_hip_error */
    NVFP4_ERR_INVALID_SCALE = 7,    /* the global scale alpha is NaN or infinite   */
    NVFP4_ERR_INVALID_STRIDE = 8,   /* an operand stride is out of range or misaligned */
    NVFP4_ERR_INVALID_TYPE = 9,     /* not an nvfp4_dtype_t                       */
    NVFP4_ERR_INVALID_ROUTING = 10, /* a router option is out of range            */
    NVFP4_ERR_INVALID_ROTATION = 11, /* a rope layout or scaling is out of range   */
    NVFP4_ERR_INVALID_CACHE = 12    /* a cache's or attention's option is out of range */
} nvfp4_status_t;

/* Element types of activations, results and logits. */
typedef enum {
    NVFP4_F16 = 0,
    NVFP4_BF16 = 1,
    NVFP4_F32 = 2
} nvfp4_dtype_t;

/*
 * Batched GEMV as defined above. If the problem is split along K (small M*L),
 * float32 partial sums go to a workspace that the library allocates on first
 * need, per device, grows on demand (with a device synchronisation) and keeps
 * until the process ends. Calls that overlap in time on one device therefore
 * must not use this entry point concurrently from two streams; use
 * nvfp4_gemv_ex with separate workspaces instead. Under HIP graph capture:
 * make the first call of the largest split shape eagerly, before capturing
 * (allocation is not capturable), and note that a captured graph keeps the
 * workspace address, which a later call needing a larger workspace frees;
 * nvfp4_gemv_ex with a caller-owned workspace, or nvfp4_gemv_noalloc, has
 * neither concern.
 */
nvfp4_status_t nvfp4_gemv(const void *a, const void *b, const void *sfa, const void *sfb,
                          void *c, int64_t M, int64_t K, int64_t L, int sf_layout,
                          void *stream);

/*
 * As nvfp4_gemv, for callers that cannot allocate: code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation. It calls no
 * hipMalloc, hipFree or allocating routine. The split-K workspace comes from a
 * fixed scratch array of nvfp4_gemv_noalloc_scratch_bytes() bytes that the
 * library holds in device memory, one copy per GPU it runs on, until the
 * process ends. The first call on a device looks up that copy's address and
 * enqueues one small kernel on `stream` that zeroes its ticket region; every
 * completed call leaves the tickets zero again. All calls on one GPU share its
 * copy, so calls that overlap in time on one GPU (two streams, or two host
 * threads) race and must not be made. A shape whose workspace
 * (nvfp4_gemv_workspace_bytes) exceeds the array returns NVFP4_ERR_WORKSPACE
 * with nothing launched; the library's own plans split K only for small M*L,
 * whose workspace stays far below it.
 */
nvfp4_status_t nvfp4_gemv_noalloc(const void *a, const void *b, const void *sfa, const void *sfb,
                                  void *c, int64_t M, int64_t K, int64_t L, int sf_layout,
                                  void *stream);

/* Bytes of nvfp4_gemv_noalloc's fixed scratch array (the workspace limit). */
size_t nvfp4_gemv_noalloc_scratch_bytes(void);

/*
 * Workspace bytes nvfp4_gemv_ex needs for this shape (0 when the shape is not
 * split along K). The value depends only on M, K and L.
 */
size_t nvfp4_gemv_workspace_bytes(int64_t M, int64_t K, int64_t L);

/*
 * As nvfp4_gemv, with a caller-owned device workspace of at least
 * nvfp4_gemv_workspace_bytes(M, K, L) bytes, 256-byte aligned (may be NULL
 * when that size is 0). The workspace must be zero-filled before its first use;
 * every completed call leaves its counter region zero again, so it can be reused
 * for any later shape without clearing. Two calls may share a workspace only
 * if they are ordered on one stream.
 */
nvfp4_status_t nvfp4_gemv_ex(const void *a, const void *b, const void *sfa, const void *sfb,
                             void *c, int64_t M, int64_t K, int64_t L, int sf_layout,
                             void *workspace, size_t workspace_bytes, void *stream);

/*
 * Batched GEMV with NVFP4's second scaling level: one float32 scale per tensor
 * pair on top of the per-16-element E4M3 scales (the "dual scaling" that
 * kernelbot NVFP4 GEMV submission 69575 lists among its notes on the format;
 * none of the pages' kernels applies it, so its placement is this library's
 * reading: it multiplies the finished float32 row sum once, before the cast):
 *
 *   c[l][m] = fp16( alpha * sum_{k<K} e2m1(A) * e4m3(SFA) * e2m1(B) * e4m3(SFB) )
 *
 * A caller whose A and B carry global scales ga and gb passes alpha = ga * gb.
 * alpha must be finite (else NVFP4_ERR_INVALID_SCALE, nothing launched); with
 * alpha = 1 the result is bit-identical to nvfp4_gemv. The product alpha * sum
 * is rounded to float32 and then to float16 (two roundings, within the
 * library's float32-accumulation error). Layouts, alignment and the other
 * arguments are as for nvfp4_gemv.
 * Workspace: NULL with workspace_bytes = 0 uses the library-owned workspace as
 * nvfp4_gemv does; otherwise it is a caller-owned workspace with the
 * requirements of nvfp4_gemv_ex (NVFP4_ERR_WORKSPACE if too small or
 * misaligned when the shape needs one).
 */
nvfp4_status_t nvfp4_gemv_scaled(const void *a, const void *b, const void *sfa, const void *sfb,
                                 void *c, int64_t M, int64_t K, int64_t L, int sf_layout,
                                 float alpha, void *workspace, size_t workspace_bytes,
                                 void *stream);

/*
 * Operand strides, for callers whose tensors are not densely packed (the
 * pages' harness, kernelbot NVFP4 GEMV submission 103289, hands B over with
 * its N dimension padded to 128 rows, so B's batch stride is 128*K/2 bytes;
 * submission 69575 reads plain scales through arbitrary row and batch
 * strides). Inside a row everything stays contiguous. Byte strides except
 * c_batch, which counts float16 elements:
 *   a_row      between rows m, m+1 of A        >= K/2, multiple of 16
 *   a_batch    between batches of A            >= 0,   multiple of 16
 *   b_batch    between batches of B            >= 0,   multiple of 16
 *   sfa_row    between rows of SFA (plain layout only; ignored for blocked,
 *              whose tiles fix it)             >= K/16, even
 *   sfa_batch  between batches of SFA          >= 0, even (plain) / multiple of 16 (blocked)
 *   sfb_batch  between batches of SFB          >= 0, even (plain) / multiple of 16 (blocked)
 *   c_batch    between batches of C, elements  >= M when L > 1 (outputs must not overlap)
 * A batch stride of 0 broadcasts one input to every batch. All strides are
 * below 2^40, and the rows of A that one workgroup reads must lie within 2^31
 * bytes: (ceil(rows_per_wg/128) + 1) * 128 * a_row + K/2 < 2^31, with
 * rows_per_wg from nvfp4_gemv_plan (about a_row <= 2^21 for any shape).
 */
typedef struct {
    int64_t a_row, a_batch;
    int64_t b_batch;
    int64_t sfa_row, sfa_batch;
    int64_t sfb_batch;
    int64_t c_batch;
} nvfp4_strides_t;

/* The dense strides of the layouts above (what nvfp4_gemv assumes). */
void nvfp4_gemv_dense_strides(int64_t M, int64_t K, int64_t L, int sf_layout,
                              nvfp4_strides_t *strides);

/*
 * nvfp4_gemv_scaled with operand strides (`strides` must not be NULL):
 * pointers, alignment, alpha and workspace as for nvfp4_gemv_scaled;
 * NVFP4_ERR_INVALID_STRIDE, nothing launched, for strides outside the rules
 * above. Results are bit-identical to the dense call on the same values.
 */
nvfp4_status_t nvfp4_gemv_strided(const void *a, const void *b, const void *sfa, const void *sfb,
                                  void *c, int64_t M, int64_t K, int64_t L, int sf_layout,
                                  const nvfp4_strides_t *strides, float alpha, void *workspace,
                                  size_t workspace_bytes, void *stream);

/*
 * Launch plan chosen for a shape (for tests and reports). Returns NVFP4_OK and
 * fills the fields, or an error status for an invalid shape.
 *   lanes_per_row  lanes that share one output row (1..256)
 *   rows_per_wg    output rows per workgroup (at most; 4 per 16-byte scale slot)
 *   k_splits       number of K-slices (1 = no split)
 *   k_per_split    K-elements per slice
 *   workgroups     grid size; threads_per_wg threads each (the first 64 of
 *                  them stage the scales, the others compute)
 *   lds_bytes      dynamic LDS per workgroup
 */
typedef struct {
    int32_t lanes_per_row;
    int32_t rows_per_wg;
    int32_t k_splits;
    int32_t k_per_split;
    int64_t workgroups;
    int32_t threads_per_wg;
    int32_t lds_bytes;
} nvfp4_plan_t;

nvfp4_status_t nvfp4_gemv_plan(int64_t M, int64_t K, int64_t L, nvfp4_plan_t *plan);

/*
 * Launch plan of the GEMV kernel with two right-hand vectors, which
 * nvfp4_gemm_small_n runs for N = 2 where no matrix-core kernel applies and
 * the GEMV's plan needs no K-split (for tests and reports; fields as for
 * nvfp4_gemv_plan). NVFP4_ERR_INVALID_SHAPE where that kernel does not run.
 */
nvfp4_status_t nvfp4_gemv_two_vectors_plan(int64_t M, int64_t K, int64_t L, nvfp4_plan_t *plan);

/*
 * Block-scaled skinny GEMM with N = 1..8 right-hand vectors (the general
 * product kernelbot NVFP4 GEMV submission 103289 hands to torch._scaled_mm,
 * a @ b^T with block scales and a float16 result; the GEMV is N = 1):
 *
 *   c[l][n][m] = fp16( alpha * sum_{k<K} e2m1(A[l][m][k]) * e4m3(SFA[l][m][k/16])
 *                                      * e2m1(B[l][n][k]) * e4m3(SFB[l][n][k/16]) )
 *
 *   a    uint8 [L][M][K/2]      as for nvfp4_gemv
 *   b    uint8 [L][N][K/2]      N packed vectors per batch
 *   sfa  as for nvfp4_gemv (layout sf_layout)
 *   sfb  plain uint8 [L][N][K/16]; blocked: the 128x4 layout of the N x K/16
 *        matrix (rows padded to 128), ceil(K/64)*512 bytes per batch
 *   c    fp16 [L][N][M]          written (column n of batch l contiguous)
 * Requirements and alignment as for nvfp4_gemv, 1 <= N <= 8, alpha finite.
 * Accumulation is float32 per row and vector (summation order the library's
 * own); no K-split and no workspace: small M*L leaves the GPU partly idle.
 * N = 1 runs the GEMV kernel (nvfp4_gemv_scaled), and N = 2 the GEMV kernel
 * with two vectors, whenever the GEMV's plan needs no split-K workspace; else
 * a dot-product kernel. From N = 3 a matrix-core kernel runs (and for N = 2
 * with blocked scales, K >= 4096 and at least 128 of its workgroups): a' =
 * e2m1 * e4m3 and b' are exact in float16, so the product is a float16 MFMA
 * with float32 accumulation. Either way nothing is allocated.
 */
nvfp4_status_t nvfp4_gemm_small_n(const void *a, const void *b, const void *sfa, const void *sfb,
                                  void *c, int64_t M, int64_t N, int64_t K, int64_t L, int sf_layout,
                                  float alpha, void *stream);

/* Launch plan of nvfp4_gemm_small_n's own kernels for a shape and scale
 * layout: rows per workgroup, workgroups and dynamic LDS bytes (for N = 1 or
 * 2 where the GEMV's kernel runs instead, the plan of the dot-product kernel
 * that would run otherwise). The matrix-core kernels (N >= 3, and N = 2 on
 * large blocked shapes) give each workgroup 32 rows, 4 workgroups per 128-row
 * block. With blocked scales they stage B, the SFB dwords and the workgroup's
 * SFA lines in LDS: grids of more than 256 workgroups stage all of K at once
 * where that fits in 150 KiB (about (3N/4 + 2) * K bytes; 256 threads per
 * workgroup), other grids stream K through three slots of 32 K-steps (52 KiB
 * for N <= 4, 78 KiB up to N = 8; 320 threads per workgroup). Plain scales:
 * no LDS. Any output pointer may be NULL. Returns NVFP4_ERR_INVALID_SHAPE for
 * shapes it does not take, NVFP4_ERR_INVALID_LAYOUT for an unknown layout. */
nvfp4_status_t nvfp4_gemm_small_n_plan(int64_t M, int64_t N, int64_t K, int64_t L, int sf_layout,
                                       int32_t *rows_per_wg, int64_t *workgroups, int32_t *lds_bytes);

/*
 * Device-side reblocking of plain scale factors into the 128x4 blocked layout
 * (the transformation kernelbot NVFP4 GEMV submission 69953 performs with
 * `to_blocked_batch` and submission 69575 with `blocked_transform_kernel`,
 * here as one HIP kernel for all batches), so that callers holding plain
 * scales can produce what nvfp4_gemv reads with sf_layout = NVFP4_SF_BLOCKED.
 *
 *   plain    uint8 [L][rows][K/16] E4M3 codes (rows = M for SFA, 1 for SFB)
 *   blocked  uint8, nvfp4_blocked_scales_bytes(rows, K, L) bytes, written:
 *            per batch ceil(rows/128)*ceil(K/64)*512 bytes, scale (r, kb) at
 *            ((r/128)*ceil(K/64) + kb/4)*512 + (r%32)*16 + ((r%128)/32)*4 + kb%4;
 *            padding bytes (r >= rows or kb >= K/16) are written as 0.
 * Both are DEVICE pointers owned by the caller; blocked must be 16-byte
 * aligned (plain has no alignment requirement) and the two must not overlap.
 * Requirements: rows, L >= 1; K >= 32, K % 32 == 0. Errors are reported before
 * any HIP call (nothing launched); the call only enqueues work on `stream`.
 */
nvfp4_status_t nvfp4_scales_to_blocked(const void *plain, void *blocked, int64_t rows, int64_t K,
                                       int64_t L, void *stream);

/* Bytes of the blocked layout for (rows, K, L); 0 for an invalid shape. */
size_t nvfp4_blocked_scales_bytes(int64_t rows, int64_t K, int64_t L);

/*
 * ---------------------------------------------------------------------------
 * FP4 linear layers: activations to NVFP4, products with any number of rows,
 * routed experts. Conventions as above (device pointers, nothing synchronised,
 * nothing allocated, every argument validated before any HIP call). No call
 * of this part keeps state between calls, so all may be captured into HIP
 * graphs and run on several streams at once; a workspace belongs to one call
 * at a time. Global scales are float32 values on the DEVICE, so that a layer
 * runs from activations to result without the host.
 *
 * Workspaces of this part: device memory of at least the bytes that the
 * matching _workspace_bytes function gives, 256-byte aligned, zero-filled
 * before its first use. Every completed call leaves its counters zero, so one
 * workspace serves any later call of this part without clearing, on one stream,
 * if it is large enough for that call. A product's size does not rise with its
 * rows N (or slots S): fewer rows may be split along K and then need more. No
 * call of this part needs more than NVFP4_WORKSPACE_MAX_BYTES, so a program that
 * does not know its row counts beforehand takes one workspace of that size. A
 * size of 0 means none is needed (NULL is then accepted).
 */
#define NVFP4_WORKSPACE_MAX_BYTES 67174400  /* 64 KiB of counters, 64 MiB of partial sums */

/*
 * Global scale of a tensor for nvfp4_quantize: the largest block of x then
 * gets the largest scale, E4M3's 448, and its largest value the largest code, 6:
 *
 *   *scale = max over finite x of |x|, times the float32 nearest to 1 / 2688
 *            (one rounding to float32), at least 2^-100; 1 if every finite x is zero
 *
 *   x       dtype (nvfp4_dtype_t) [L][rows][K], strides in elements: row_stride
 *           between rows (>= K, or anything >= 0 if rows == 1), batch_stride
 *           between batches (>= 0); a value contiguous in k; aligned to its type
 *   scale   float32, written
 * NaN and infinite values are passed over. Requirements: rows, L >= 1; K >= 1.
 */
size_t nvfp4_global_scale_workspace_bytes(void);
nvfp4_status_t nvfp4_global_scale(const void *x, int dtype, float *scale, int64_t rows, int64_t K,
                                  int64_t L, int64_t row_stride, int64_t batch_stride,
                                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * Quantisation to NVFP4. Per row and block b of 16 consecutive k, with the
 * global scale g = *global_scale (NULL: g = 1):
 *
 *   s[b]  = E4M3 nearest to  max_{k in b} |x[k]| / (6 g)   (at most 448)
 *   q[k]  = E2M1 nearest to  x[k] / (s[b] g)               (at most 6 in size)
 *
 * Ties go to the even code. Both roundings are those of the exact quotients:
 * no intermediate rounding decides a code. The sign of x[k] is kept (a value
 * that rounds to zero keeps it too). s[b] = 0 gives codes of 0. A block with
 * a NaN gets the scale code 0x7F (NaN), so that products with it are NaN; an
 * infinite x[k] saturates to code 6 of its block, whose scale is then 448. A g
 * that is not finite or below 2^-100 makes every scale 0x7F.
 *
 *   x       as for nvfp4_global_scale
 *   codes   uint8 [L][rows][K/2], written (8-byte aligned)
 *   scales  uint8, written in sf_layout: plain [L][rows][K/16]; blocked: the
 *           128x4 layout, nvfp4_blocked_scales_bytes(rows, K, L) bytes, padding
 *           written as 0 (4-byte aligned)
 * The outputs are operands of nvfp4_gemv (rows = 1 or M), nvfp4_gemm_small_n
 * and nvfp4_gemm: those want 16-byte aligned codes. Requirements: rows, L >= 1;
 * K % 32 == 0; codes and scales do not overlap x; and at most 2^24 - 1
 * workgroups, which are L * ceil(rows * K / 4096) for plain scales and
 * L * 8 * ceil(rows / 128) * ceil(K / 256) for blocked ones.
 */
nvfp4_status_t nvfp4_quantize(const void *x, int dtype, const float *global_scale, void *codes,
                              void *scales, int64_t rows, int64_t K, int64_t L, int64_t row_stride,
                              int64_t batch_stride, int sf_layout, void *stream);

/*
 * The values that codes and scales stand for: out[l][r][k] = q * s * g, out
 * of type dtype, dense [L][rows][K]. q * s is exact; the product with g is
 * rounded to float32 and then to dtype (so at most half a step and 2^-24 off).
 * Requirements: rows, L >= 1; K % 32 == 0; L * rows * K <= 4096 * (2^24 - 1).
 */
nvfp4_status_t nvfp4_dequantize(const void *codes, const void *scales, const float *global_scale,
                                void *out, int dtype, int64_t rows, int64_t K, int64_t L,
                                int sf_layout, void *stream);

/*
 * Product of NVFP4 matrices with any number of rows N (prompts and batches;
 * nvfp4_gemm_small_n's operation without its limit on N):
 *
 *   c[l][n][m] = alpha * ga * gb * sum_{k<K} e2m1(A[l][m][k]) * e4m3(SFA[l][m][k/16])
 *                                          * e2m1(B[l][n][k]) * e4m3(SFB[l][n][k/16])
 *
 *   a, b, sfa, sfb, sf_layout  as for nvfp4_gemm_small_n, N >= 1
 *   scale_a, scale_b           float32 on the device, ga and gb (NULL: 1)
 *   c      dtype [L][N][M], written; aligned to its type
 * Accumulation is float32 (the products are exact), one rounding of the scaled
 * sum to float32 and one to dtype; float16 overflows to +-inf. The product
 * alpha * ga * gb itself may leave float32's range. The order of
 * summation is fixed for a shape, so equal calls give equal bits.
 * Requirements: M, N, L >= 1; K % 32 == 0; M, N <= 2^30; K <= 2^22; a, b, sfa
 * and sfb 16-byte aligned; alpha finite; at most 2^23 - 1 workgroups (a shape
 * that needs more is refused by nvfp4_gemm_plan too).
 */
size_t nvfp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t L);
nvfp4_status_t nvfp4_gemm(const void *a, const void *b, const void *sfa, const void *sfb, void *c,
                          int dtype, int64_t M, int64_t N, int64_t K, int64_t L, int sf_layout,
                          float alpha, const float *scale_a, const float *scale_b, void *workspace,
                          size_t workspace_bytes, void *stream);

/* What nvfp4_gemm launches for a shape (for tests and reports): rows of A and
 * of B per workgroup, slices of K, K-elements per slice, workgroups. */
typedef struct {
    int32_t tile_m, tile_n;
    int32_t k_splits, k_per_split;
    int64_t workgroups;
} nvfp4_gemm_plan_t;

nvfp4_status_t nvfp4_gemm_plan(int64_t M, int64_t N, int64_t K, int64_t L, nvfp4_gemm_plan_t *plan);

/*
 * Router of a mixture of experts: the k experts of each of T tokens, their
 * weights, and the experts' lists that nvfp4_gemm_experts takes.
 *
 *   score[t][e]  softmax over e of logits[t] (NVFP4_SCORE_SOFTMAX) or
 *                1 / (1 + exp(-logits[t][e])) (NVFP4_SCORE_SIGMOID)
 *   pick[t][e]   score + bias[e] (bias NULL: score)
 *   groups       the E experts form n_group runs of E / n_group; a group's
 *                value is the sum of its group_top largest picks (of those not
 *                masked); only experts of the topk_group groups of largest
 *                value are left
 *   ids[t][j]    the k left experts of largest pick, largest first
 *   weights[t][j] score (without bias) of expert ids[t][j]; if renormalize,
 *                divided by the token's sum of them; times scaling
 *
 * Scores and picks are compared in float64 (ties, also between groups, go to
 * the lower index), weights are rounded once more to float32 at the end and are
 * within a few float32 steps.
 * A logit of -inf or NaN masks its expert: score 0, never picked; so does a
 * bias of -inf or NaN, which leaves the scores as they are. Where fewer
 * than k experts are left, the rest of ids is -1 with weight 0; a token whose
 * mask leaves none gets only those. Logits of +inf share a softmax equally.
 * If the sum of a token's scores is 0, renormalised weights are 0.
 *
 * The experts' lists hold the slots t * k + j with ids[t][j] >= 0, sorted by
 * expert and then by slot:
 *   offsets int32 [E + 1]   expert e's slots are order[offsets[e] .. offsets[e+1])
 *   order   int32 [T * k]   entries from offsets[E] on are not written
 *
 *   logits dtype [T][E] dense, bias float32 [E], ids int32 [T][k], weights
 *   float32 [T][k]; all aligned to their types.
 * Requirements: T >= 1, T * k <= 2^30, T <= 16 * (2^24 - 1) where k < 16 and
 * E <= 256, T <= 4 * (2^24 - 1) elsewhere; 1 <= E <= 1024; 1 <= k <= min(E, 64);
 * n_group divides E and is at most 64; 1 <= topk_group <= n_group; 1 <= group_top
 * <= E / n_group, at most 2; scaling finite.
 */
typedef enum {
    NVFP4_SCORE_SOFTMAX = 0,
    NVFP4_SCORE_SIGMOID = 1
} nvfp4_score_t;

typedef struct {
    int32_t score;          /* nvfp4_score_t */
    int32_t n_group, topk_group, group_top;
    int32_t renormalize;    /* 0 or 1 */
    float scaling;
} nvfp4_routing_t;

size_t nvfp4_moe_route_workspace_bytes(int64_t T, int64_t E, int64_t k);
nvfp4_status_t nvfp4_moe_route(const void *logits, int dtype, const float *bias, int32_t *ids,
                               float *weights, int32_t *offsets, int32_t *order, int64_t T,
                               int64_t E, int64_t k, const nvfp4_routing_t *routing,
                               void *workspace, size_t workspace_bytes, void *stream);

/*
 * Products of routed rows with their experts' NVFP4 weights. Slot s has row
 * s / slots_per_row of B (slots_per_row = k: the tokens' rows, each taken for
 * k slots; 1: a row for each slot) and the expert e whose list holds s:
 *
 *   c[s][m] = alpha * ga[e] * gb * sum_{k<K} e2m1(A[e][m][k]) * e4m3(SFA[e][m][k/16])
 *                * e2m1(B[s / slots_per_row][k]) * e4m3(SFB[s / slots_per_row][k/16])
 *
 *   a, sfa   the experts' weights: as nvfp4_gemm's with E batches
 *   b, sfb   rows x K, one batch
 *   offsets, order   as nvfp4_moe_route writes them (on the device): offsets
 *            rise from 0 to at most S = rows * slots_per_row, and order's
 *            entries are slots in [0, S), each once. Entries outside [0, S)
 *            are passed over, offsets are clamped to 0..S: nothing is read or
 *            written out of bounds whatever they hold.
 *   scale_a  float32 [E] on the device (NULL: 1), scale_b float32 (NULL: 1)
 *   c        dtype [S][M]; rows of slots in no list are not written
 * Rounding, order of summation and requirements as for nvfp4_gemm; E <= 1024,
 * rows, slots_per_row >= 1, S <= 2^30, rows * K / 2 <= 2^32 (B's rows are gathered
 * by 32-bit offsets); workgroups as for nvfp4_gemm, for the most tiles that any
 * lists of S slots have.
 */
size_t nvfp4_gemm_experts_workspace_bytes(int64_t M, int64_t K, int64_t E, int64_t S);
nvfp4_status_t nvfp4_gemm_experts(const void *a, const void *b, const void *sfa, const void *sfb,
                                  void *c, int dtype, int64_t M, int64_t K, int64_t E, int64_t rows,
                                  int64_t slots_per_row, int sf_layout, const int32_t *offsets,
                                  const int32_t *order, float alpha, const float *scale_a,
                                  const float *scale_b, void *workspace, size_t workspace_bytes,
                                  void *stream);

/*
 * Weighted sum of each token's slots:
 *   out[t][m] = sum_j weights[t][j] * y[t * k + j][m]   over j with ids[t][j] >= 0
 * in float32, j = 0, 1, .., rounded once to dtype; 0 for a token with no such
 * j. Slots with a negative id are not read (their rows may hold anything).
 *   y dtype [T * k][M], out dtype [T][M], ids int32 and weights float32 [T][k];
 * all aligned to their types. Requirements: T, k, M >= 1; k <= 64; T * k <= 2^30;
 * M <= 2^30; T * ceil(M / 8) (float32: M / 4) <= 256 * (2^24 - 1).
 */
nvfp4_status_t nvfp4_moe_combine(const void *y, int dtype, const int32_t *ids, const float *weights,
                                 void *out, int64_t T, int64_t k, int64_t M, void *stream);

/*
 * ---------------------------------------------------------------------------
 * Attention over a paged NVFP4 key/value cache. Conventions as in the part
 * before (device pointers, nothing synchronised, nothing allocated, no state
 * between calls, every argument validated before any HIP call; the workspace
 * of nvfp4_cache_attention is one of that part's, with the same rules and the
 * same largest size). A layer's step, for the q, k and v of T new tokens:
 * nvfp4_rope on the heads of q and k, nvfp4_cache_write of k and v,
 * nvfp4_cache_attention of q.
 */

/*
 * Rotary positions. Per token t and head, for the R / 2 pairs of the head's
 * first R values, with a = positions[t] * frequencies[j]:
 *
 *   out[i0] = factor * (x[i0] * cos a - x[i1] * sin a)
 *   out[i1] = factor * (x[i0] * sin a + x[i1] * cos a)
 *
 *   layout     NVFP4_ROPE_HALF: i0 = j, i1 = j + R / 2; NVFP4_ROPE_INTERLEAVED:
 *              i0 = 2 j, i1 = 2 j + 1. Values from R on are copied as they are.
 *   transpose  1: with -a for a. That is the gradient: the gradient of x is
 *              nvfp4_rope with transpose = 1 of the gradient of out.
 *   x, out     dtype (nvfp4_dtype_t) [T][H][D], strides in elements between
 *              tokens and between heads (x's may be 0; rows of out must not
 *              overlap); a row contiguous; aligned to their type. out may be x
 *              with the same strides; else the two do not overlap. The heads of
 *              q and k in one packed projection are one call.
 *   positions  int64 [T], frequencies float64 [R / 2], both 8-byte aligned
 * The angle is exact to 2^-24 while its size is below 2^40 (so are positions
 * up to 2^40 with frequencies up to 1), cos and sin to 2^-22, the sum is float32
 * and rounded once to dtype. Requirements: T, H >= 1; 2 <= R <= D, R even, at most 2048;
 * H, D <= 2^20; factor finite; at most 2^24 - 1 workgroups (about one per token
 * or more).
 */
typedef enum {
    NVFP4_ROPE_HALF = 0,
    NVFP4_ROPE_INTERLEAVED = 1
} nvfp4_rope_layout_t;

nvfp4_status_t nvfp4_rope(const void *x, int dtype, void *out, const int64_t *positions, const double *frequencies,
                          int64_t T, int64_t H, int64_t D, int64_t R, int64_t x_token_stride, int64_t x_head_stride,
                          int64_t out_token_stride, int64_t out_head_stride, int layout, float factor, int transpose,
                          void *stream);

/*
 * Frequencies for nvfp4_rope, on the HOST (float64 [R / 2], written): f[j] =
 * base^(-2 j / R), scaled for contexts longer than `length`, the positions that
 * a model was trained on (scaling NULL: NVFP4_ROPE_UNSCALED):
 *
 *   LINEAR  f / factor
 *   BASE    base * factor^(R / (R - 2)) in place of base
 *   BANDS   f * keep + f / factor * (1 - keep), keep rising from 0 to 1 with the
 *           turns length * f / (2 pi) from `low` to `high`, linear in the turns
 *   RAMP    the same with keep falling from 1 to 0 linearly in j, from the pair
 *           that turns `high` times (rounded down, at least 0) to the one that
 *           turns `low` times (rounded up, at most R - 1)
 * Requirements: R even, 2..2048 (BASE: not 2); base > 1; factor >= 1; BANDS and
 * RAMP: 0 < low < high, length > 0; all finite.
 */
typedef enum {
    NVFP4_ROPE_UNSCALED = 0,
    NVFP4_ROPE_LINEAR = 1,
    NVFP4_ROPE_BASE = 2,
    NVFP4_ROPE_BANDS = 3,
    NVFP4_ROPE_RAMP = 4
} nvfp4_rope_method_t;

typedef struct {
    int32_t method;                 /* nvfp4_rope_method_t */
    double factor, length, low, high;
} nvfp4_rope_scaling_t;

nvfp4_status_t nvfp4_rope_frequencies(double *frequencies, int64_t R, double base,
                                      const nvfp4_rope_scaling_t *scaling);

/*
 * A paged key/value cache in NVFP4 (the struct is read on the host, by each call):
 *
 *   k_codes, v_codes    uint8 [pages][heads][page_size][head_size / 2]
 *   k_scales, v_scales  uint8 [pages][heads][page_size][head_size / 16] (E4M3)
 * A page is dense; code_page_stride and scale_page_stride are the bytes between
 * pages (of keys and of values alike), so keys and values may share an
 * allocation. The value of a code is q * s * g with g = *k_scale (*v_scale),
 * float32 on the device, NULL: 1. The slot of a token is page * page_size + its
 * place in the page. Requirements: 1 <= pages < 2^31; page_size a power of two,
 * 16..4096; 1 <= heads <= 4096; head_size a multiple of 32, 32..256; a page's
 * codes below 2^31 bytes; codes and scales 16-byte aligned, page strides
 * multiples of 16, at least a page and below 2^32; k_scale, v_scale 4-byte aligned.
 */
typedef struct {
    void *k_codes, *k_scales, *v_codes, *v_scales;
    const float *k_scale, *v_scale;
    int64_t pages, page_size, heads, head_size;
    int64_t code_page_stride, scale_page_stride;
} nvfp4_cache_t;

/*
 * Keys and values of T tokens into the cache, quantised as by nvfp4_quantize
 * with the cache's global scales (blocks of 16 values along the head; a NaN
 * makes its block's scale NaN):
 *   k, v    dtype [T][heads][head_size], strides in elements between tokens and
 *           between heads (>= 0); a row contiguous; aligned to their type
 *   slots   int64 [T]; a token whose slot is outside the cache (negative, say)
 *           is not written. Each slot at most once: where two tokens have one slot,
 *           its blocks' codes and scales may stay from either, each by itself.
 * Nothing else of the cache changes. Requirements: T >= 1; (T + 64) * heads *
 * head_size / 16 <= 2^31 - 2048.
 */
nvfp4_status_t nvfp4_cache_write(const nvfp4_cache_t *cache, const void *k, const void *v, int dtype,
                                 const int64_t *slots, int64_t T, int64_t k_token_stride, int64_t k_head_stride,
                                 int64_t v_token_stride, int64_t v_head_stride, void *stream);

/*
 * Rows of the cache as values, rounded as by nvfp4_dequantize: k and v dtype
 * [T][heads][head_size] dense, written; slots as above, in any order and any
 * number of times; zeros for a slot outside the cache. Requirements as above.
 */
nvfp4_status_t nvfp4_cache_read(const nvfp4_cache_t *cache, void *k, void *v, int dtype, const int64_t *slots, int64_t T,
                                void *stream);

/*
 * Attention of the queries of B sequences over their pages of the cache. The
 * queries of sequence b are rows offsets[b] .. offsets[b + 1] of q, n_b of them:
 * the last n_b of its lengths[b] positions (decoding: 1; drafted tokens: a few;
 * prompts and their chunks: many; any mixture). Position t is in page
 * table[b][t / page_size], at place t % page_size. Query head h reads the
 * cache's head h / (H / heads). For query i of sequence b, at position
 * p = lengths[b] - n_b + i:
 *
 *   logit[t] = scale * q . K[t]      over the positions t that it sees:
 *              0 <= t < lengths[b]; causal: t <= p; window > 0: t > p - window;
 *              and the page of t is a page of the cache
 *   out      = sum_t softmax(logit)[t] * V[t]
 *   lse      = ln sum_t exp(logit[t])            (float32 [T][H], optional)
 *
 * A query that sees nothing gets zeros, and -inf. What it does not see does not
 * enter, whatever it holds: positions behind a sequence's length, NaN scales of keys or
 * values that the mask hides. (A NaN scale of a value makes NaN the block of every
 * query that sees it, whatever its probability.) A query with an infinite or
 * NaN value that sees something gets NaN.
 *
 *   q        dtype [T][H][head_size], strides in elements between tokens and
 *            between heads (>= 0); a row contiguous; aligned to its type
 *   out      dtype [T][H][head_size] dense; aligned to its type; does not overlap
 *            q. Rows of no sequence (behind offsets[B], say) are not written.
 *   offsets  int32 [B + 1], rising from 0 to at most T; lengths int32 [B]; table
 *            int32 [B][table_width]; on the device, where they may change
 *            between a captured graph's replays. Offsets are clamped to 0..T, lengths to
 *            0..max_length, and entries of the table outside the cache hide
 *            their positions: nothing is read or written out of bounds
 *            whatever they hold.
 *   max_q, max_length   bounds of the host on n_b and lengths[b], from which
 *            the grid is planned. Rows behind a sequence's first max_q are not
 *            written. max_length <= table_width * page_size.
 * Keys and values are exact in float16 and go to the matrix cores as that; q is
 * taken to float16 with a power of two of its row's own (float32: as two float16,
 * 22 bits), probabilities to float16 (float32: two; all to at least 2^-33 of the
 * query's largest), sums, maxima and norms are
 * float32 (logits past its range give NaN), out is rounded once to dtype. The order of summation is fixed for
 * given arguments and lengths, so equal calls give equal bits.
 * Requirements: T, B >= 1; T <= 2^30; B * max_q and H / heads * max_q <= 2^30; heads
 * divides H, H / heads <= 1024; head_size 64, 96, 128, 192 or 256; 1 <= max_q <= T; 1 <= max_length <=
 * table_width * page_size <= 2^30; scale finite; window >= 0 and below 2^31; at most 2^23 - 1
 * workgroups.
 */
typedef struct {
    int64_t q_token_stride, q_head_stride;
    int64_t max_q, max_length;
    int64_t window;                 /* 0: none */
    float scale;
    int32_t causal;                 /* 0 or 1 */
} nvfp4_attention_t;

size_t nvfp4_cache_attention_workspace_bytes(const nvfp4_cache_t *cache, int dtype, int64_t T, int64_t H, int64_t B,
                                             const nvfp4_attention_t *attention);
nvfp4_status_t nvfp4_cache_attention(const nvfp4_cache_t *cache, const void *q, int dtype, void *out, float *lse,
                                     const int32_t *offsets, const int32_t *lengths, const int32_t *table, int64_t T,
                                     int64_t H, int64_t B, int64_t table_width, const nvfp4_attention_t *attention,
                                     void *workspace, size_t workspace_bytes, void *stream);

/* Static description of a status code (never NULL). */
const char *nvfp4_status_string(int status);

/* The hipError_t of the last failed HIP call in this thread (0 if none). */
int nvfp4_last_hip_error(void);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_GEMV_H */
