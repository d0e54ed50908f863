/*
 * tgemm -- tiled GEMM  C = A * B^T  for AMD Instinct MI355X (gfx950).
 *
 * The operation is the one FlyDSL's preshuffle GEMM computes (FlyDSL "Kernel
 * authoring guide", section 11 "Complete example: Preshuffle GEMM"; FlyDSL
 * "Kernel Authoring" skill, section 6 "GEMM Pattern (Preshuffle)"):
 *
 *     C[m][n] = cvt( (sum_k A[m][k] * B[n][k]) * s_a * s_b )
 *
 * products of the input elements summed in fp32 (fp8: by the matrix unit, in
 * fewer bits; see GEMM_E4M3_OUT_BF16), the scale applied in fp32
 * as (acc * s_a) * s_b (the Kernel Authoring skill's section 3 shows that
 * order), then converted to the output type with round-to-nearest-even.
 *
 * Storage (all row-major, leading dimensions implicit):
 *   A  M x K    elements of the input type            (lda = K)
 *   B  N x K    elements of the input type            (ldb = K)
 *              or, for GEMM_LAYOUT_BT_PRESHUFFLED, the N*K-element image
 *              written by gemm_preshuffle_b (see there)
 *   C  M x N    elements of the output type           (ldc = N)
 *
 * GEMM_LAYOUT_BN stores B as K x N row-major (ldb = N), the layout of the
 * pages' naive GEMM template (FlyDSL "Kernel Authoring" skill, section 8
 * "Common Patterns and Recipes", the naive GEMM's (K, N):(N, 1) view of B),
 * so C = A * B with b(n,k) = B[k][n].  The kernel reads it through the
 * gfx950 LDS transpose load (ds_read_b64_tr_b16, the 16-lane copy atom of
 * FlyDSL's "add-target-atom-op" skill, section 1.5.2 "Shape-product
 * invariants"; for 8-bit elements its form ds_read_b64_tr_b8).  bf16, fp8
 * e4m3 or int8 inputs; K * N * elem_bytes < 2^31; no pre-shuffled image
 * (gemm_preshuffle_b rejects such plans); fp8 and int8 plans use 256 x 256
 * tiles.
 *
 * GEMM_LAYOUT_AT and GEMM_LAYOUT_AT_BN store A as K x M row-major (lda = M),
 * so a(m,k) = A[k][m]; B is N x K (AT) or K x N (AT_BN, b(n,k) = B[k][n]).
 * The other operand layout the same skill's naive template and transpose
 * atom describe, read through the same LDS transpose load (16-bit or 8-bit
 * form).  bf16, fp8 e4m3 or int8 inputs; M * elem_bytes % 16 == 0 (16-byte
 * pieces of A's K-rows); K * M * elem_bytes < 2^31; such plans always use
 * 256 x 256 tiles.  B is read as stored; only
 * GEMM_LAYOUT_BT_PRESHUFFLED plans read the pre-shuffled image.
 *
 * Every pointer passed to gemm_preshuffle_b / gemm_run is a DEVICE pointer
 * owned by the caller.  The library allocates no device memory, never
 * synchronises, and launches asynchronously on the given stream; a plan holds
 * only host metadata and may be destroyed as soon as gemm_run returns.
 * Calls on one plan from several streams or threads are safe.  C must not
 * overlap A or B.
 *
 * Errors: functions returning int give GEMM_OK (0) or a negative
 * gemm_status; functions returning a pointer give NULL.  The reason is kept
 * per thread and read with gemm_last_error().  Only errors detectable on the
 * host are reported (argument checks, launch failures via hipGetLastError);
 * a fault inside a kernel surfaces at the caller's next synchronisation.
 */
#ifndef TGEMM_H
#define TGEMM_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    GEMM_OK = 0,
    GEMM_ERR_INVALID_ARG = -1,   /* NULL or misaligned pointer, bad enum, negative size */
    GEMM_ERR_UNSUPPORTED = -2,   /* shape outside the supported set, wrong GPU       */
    GEMM_ERR_HIP = -3            /* a HIP runtime call or kernel launch failed        */
} gemm_status;

typedef enum {
    GEMM_BF16_OUT_F32 = 0,       /* A, B bf16; C fp32 (no rounding of the fp32 sum)   */
    GEMM_BF16_OUT_BF16 = 1,      /* A, B bf16; C bf16                                 */
    GEMM_E4M3_OUT_BF16 = 2,      /* A, B OCP fp8 e4m3fn (max 448); C bf16.  The matrix
                                    unit (also for MXFP8) adds 8 products along K at a
                                    time and drops what lies more than 13 binary places
                                    below the largest; the sums of 8 are added in fp32.
                                    Measured on N(0, 1) data against sum |a b|: at most
                                    2.1e-5 at K = 128, 3.1e-6 at 2048, 1.0e-6 at 8192.
                                    (e4m3 converts to bf16 exactly: a bf16 plan keeps fp32
                                    sums, at half the rate.)                          */
    GEMM_MXFP8_OUT_BF16 = 3,     /* A, B MX: e4m3fn elements + E8M0 scales; C bf16    */
    GEMM_MXFP4_OUT_BF16 = 4,     /* A, B MX: e2m1 elements (2 per byte) + E8M0; C bf16 */
    GEMM_I8_OUT_BF16 = 5,        /* A, B int8, exact int32 sums; C bf16               */
    GEMM_W4A8_OUT_BF16 = 6       /* A int8, B int4 (2 per byte), int32 sums; C bf16   */
} gemm_dtype;

typedef enum {
    GEMM_LAYOUT_BT = 0,               /* B is N x K row-major                        */
    GEMM_LAYOUT_BT_PRESHUFFLED = 1,   /* B is the image written by gemm_preshuffle_b */
    GEMM_LAYOUT_BN = 2,               /* B is K x N row-major: C = A * B (bf16, e4m3, int8) */
    GEMM_LAYOUT_AT = 3,               /* A is K x M row-major, B N x K (bf16, e4m3, int8)   */
    GEMM_LAYOUT_AT_BN = 4             /* A is K x M, B K x N row-major (bf16, e4m3, int8)   */
} gemm_layout;

typedef struct gemm_plan gemm_plan;   /* opaque, immutable after creation */

/*
 * gemm_plan_create -- validate a problem and pick its kernel and tiling.
 *   M, N, K  sizes in elements; M may be 0 (gemm_run then does nothing),
 *            K may be 0 (C is then all zeros).
 *   dtype    gemm_dtype; layout gemm_layout.
 * Requirements (else NULL with GEMM_ERR_UNSUPPORTED / GEMM_ERR_INVALID_ARG):
 *   0 <= M, N, K <= 2^30;  N % 16 == 0;
 *   K * elem_bytes % 64 == 0 -- the 64-byte K step of the pages' GEMM (Kernel
 *   Authoring skill, section 10 "Troubleshooting", tile_k rule);
 *   K * elem_bytes < 2^23 and N * out_bytes * 256 < 2^31 (a 256-row tile of
 *   any operand stays inside one 2^31-byte buffer range).
 * Host only: no device work, no allocation on the device.  Returns a plan the
 * caller frees with gemm_plan_destroy.
 */
gemm_plan *gemm_plan_create(int64_t M, int64_t N, int64_t K, int dtype, int layout);

/*
 * Kernel choice for gemm_plan_create_opt.  GEMM_KERNEL_AUTO is the planner's
 * own pick by shape, dtype and layout (what gemm_plan_create does); the others
 * force one kernel family for every shape, so that each family the planner
 * may pick can be checked and timed on any shape.  Every choice computes the
 * same C within the same bound; only speed differs.
 */
typedef enum {
    GEMM_KERNEL_AUTO = 0,         /* the planner's table                                      */
    GEMM_KERNEL_GENERIC_128 = 1,  /* generic tiled kernel, 128 x 128 tiles (bf16, e4m3)       */
    GEMM_KERNEL_GENERIC_256 = 2,  /* generic tiled kernel, 256 x 256 tiles (bf16, e4m3)       */
    GEMM_KERNEL_TILE256 = 3,      /* the planner's 256 x 256 kernel at any size (no skinny
                                     kernel, no 128 x 128 tiles)                              */
    GEMM_KERNEL_PIPE = 4,         /* 256 x 256, B straight to registers, 8 waves (bf16 and
                                     e4m3 with B N x K or pre-shuffled; integer operands)     */
    GEMM_KERNEL_PIPE4 = 5         /* the same with 4 waves and AGPR accumulators; for MX plans
                                     the 16x16x128 form of the scaled MFMA (block-scale image
                                     form 0)                                                   */
} gemm_kernel_choice;

typedef struct {
    int32_t kernel;               /* gemm_kernel_choice                                       */
    int32_t splits;               /* gemm_run_ws K slices: 0 the planner's choice, 1 never
                                     split, 2..64 that many (plans whose kernel can split)    */
} gemm_plan_options;

/*
 * gemm_plan_create_opt -- gemm_plan_create with an explicit kernel choice and
 * split count.  opt == NULL (or all fields 0) is exactly gemm_plan_create.
 * Errors as gemm_plan_create, plus GEMM_ERR_INVALID_ARG for an unknown choice
 * or a split count outside 0..64, and GEMM_ERR_UNSUPPORTED when the chosen
 * family has no kernel for the dtype and layout.  The library reads no
 * environment variables: a plan depends on these arguments only.
 */
gemm_plan *gemm_plan_create_opt(int64_t M, int64_t N, int64_t K, int dtype, int layout,
                                const gemm_plan_options *opt);

/* gemm_plan_destroy -- free a plan (NULL is ignored). */
void gemm_plan_destroy(gemm_plan *plan);

/*
 * gemm_preshuffled_b_bytes -- bytes of the pre-shuffled B image:
 * N * K * b_elem_bits / 8 (a pure permutation of B).  0 for a NULL plan.
 */
size_t gemm_preshuffled_b_bytes(const gemm_plan *plan);

/*
 * gemm_preshuffle_b -- write B (N x K row-major) in MFMA operand order.
 * The image is the 5-mode byte array (N/16, Kb/64, 4, 16, 16) taken in
 * row-major order, with Kb = K * b_elem_bits / 8 (B's row bytes): n-block, 64-byte k-block,
 * 16-byte k-quarter q, row r within the n-block, byte.  Each 1 KiB block is
 * therefore one wave's B operand for a 64-byte K step: lane 16*q + r loads
 * the 16 bytes of row 16*nb + r at k-bytes 64*kb + 16*q.  (Kernel Authoring
 * skill, section 6 "GEMM Pattern (Preshuffle)" step 1; K counted in bytes and
 * kpack = 16 bytes is this library's reading of that tuple.)
 *   B       device pointer, 16-byte aligned, N*K elements.
 *   B_shuf  device pointer, 16-byte aligned, gemm_preshuffled_b_bytes(plan)
 *           bytes, must not overlap B.
 *   stream  HIP stream (0 = default stream).
 * Any plan of the same (N, K, dtype) may be used; the image does not depend
 * on M or on the plan's layout.  Asynchronous; returns GEMM_OK or an error.
 */
int gemm_preshuffle_b(const gemm_plan *plan, const void *B, void *B_shuf, hipStream_t stream);

/*
 * gemm_run -- C = cvt((A * B^T) * s_a * s_b) on `stream`.
 *   A      device pointer, 16-byte aligned, M x K input elements (K x M
 *          for GEMM_LAYOUT_AT and GEMM_LAYOUT_AT_BN).
 *   B      device pointer, 16-byte aligned: N x K (GEMM_LAYOUT_BT,
 *          GEMM_LAYOUT_AT), the pre-shuffled image (GEMM_LAYOUT_BT_PRESHUFFLED)
 *          or K x N (GEMM_LAYOUT_BN, GEMM_LAYOUT_AT_BN).
 *   C      device pointer, 16-byte aligned, M x N output elements; overwritten.
 *   scale  device pointer to two floats {s_a, s_b}, or NULL for 1, 1.  Read
 *          on the device, so fp8 scales never force a host synchronisation.
 * Asynchronous; allocates nothing.  Returns GEMM_OK or an error code.
 */
int gemm_run(const gemm_plan *plan, const void *A, const void *B, void *C,
             const float *scale, hipStream_t stream);

/*
 * Fused epilogues.  The pages' GEMM takes scale_a, scale_b and bias tensors
 * and an epilogue choice of "none", "bias", "bias_relu", "bias_silu" or
 * "bias_gelu" (FlyDSL "Kernel authoring guide", section 11 "Complete
 * example: Preshuffle GEMM"), applying the scales as (acc * scale_a) *
 * scale_b in fp32 (FlyDSL "Kernel Authoring" skill, section 3).  This
 * library's reading of the shapes and formulas, all in fp32:
 *
 *   z[m][n] = (acc[m][n] * sa(m)) * sb(n)  (+ bias[n])
 *   C[m][n] = cvt( act(z[m][n]) )
 *
 *   sa(m) = scale_a[m] (per row of C) or scale_a[0], 1 when scale_a is NULL;
 *   sb(n) = scale_b[n] (per column of C) or scale_b[0], 1 when NULL;
 *   act:  none; ReLU z > 0 ? z : +0; SiLU z / (1 + e^-z);
 *         GELU by its definition z * Phi(z) = z / 2 * (1 + erf(z / sqrt 2)).
 */
typedef enum {
    GEMM_EPI_NONE = 0,           /* scales only; bias must be NULL            */
    GEMM_EPI_BIAS = 1,           /* + bias                                    */
    GEMM_EPI_BIAS_RELU = 2,      /* + bias, then ReLU                         */
    GEMM_EPI_BIAS_SILU = 3,      /* + bias, then SiLU                         */
    GEMM_EPI_BIAS_GELU = 4       /* + bias, then GELU (erf form)              */
} gemm_epilogue;

typedef struct {
    const float *scale_a;        /* device; NULL, 1 value, or M values; 4-byte aligned           */
    const float *scale_b;        /* device; NULL, 1 value, or N values; 4-byte aligned, 16-byte
                                    aligned when per column                                      */
    const float *bias;           /* device; N values, 16-byte aligned; required by the bias
                                    epilogues, NULL for GEMM_EPI_NONE                             */
    int32_t scale_a_per_row;     /* 0: scale_a[0] scales every row; 1: scale_a[m] scales row m
                                    (M below 2^30)                                                */
    int32_t scale_b_per_col;     /* 0: scale_b[0] scales every column; 1: scale_b[n] column n     */
    int32_t epilogue;            /* gemm_epilogue                                                 */
} gemm_epilogue_args;

/*
 * gemm_run_ex -- gemm_run with the fused epilogue above.
 *   A, B, C, stream  as for gemm_run.
 *   epi      host pointer to the description (read during the call only; the
 *            vectors it points to are read on the device, asynchronously, and
 *            must stay valid until the launch completes).  NULL = no scaling,
 *            no bias, no activation.
 * gemm_run(plan, A, B, C, scale, s) is gemm_run_ex with scale_a = scale,
 * scale_b = scale + 1 (per tensor) and GEMM_EPI_NONE.
 * Errors: GEMM_ERR_INVALID_ARG for an unknown epilogue, a per-row/column flag
 * other than 0 or 1, a missing bias (bias epilogues) or an unexpected one
 * (GEMM_EPI_NONE), or a misaligned vector; otherwise as gemm_run.
 */
int gemm_run_ex(const gemm_plan *plan, const void *A, const void *B, void *C,
                const gemm_epilogue_args *epi, hipStream_t stream);

/*
 * Split K with a caller-provided workspace.  When a problem has fewer
 * 256 x 256 output tiles than the chip has compute units (a few hundred rows
 * of A against a large B: batched decode, small prefill), each tile is
 * computed by s workgroups that take one K slice each and write fp32 partial
 * tiles to the workspace; a second kernel sums the s partials of every
 * element in slice order (deterministic) and applies the epilogue of
 * gemm_run_ex.  The plan decides s (gemm_plan_info.ws_splits); plans with
 * s == 1 need no workspace.  bf16, fp8 e4m3, int8 and W4A8 plans with
 * GEMM_LAYOUT_BT or GEMM_LAYOUT_BT_PRESHUFFLED split; MX plans and the other
 * layouts never do.  (The pages' GEMM
 * has no split K: this is this library's answer to shapes whose tile grid
 * leaves most of the chip idle.)
 *
 * gemm_workspace_bytes -- bytes gemm_run_ws needs to split K:
 *   ws_splits * M * N * 4, or 0 when the plan does not split (or NULL).
 */
size_t gemm_workspace_bytes(const gemm_plan *plan);

/*
 * gemm_run_ws -- gemm_run_ex, split over K when the workspace allows it.
 *   A, B, C, epi, stream  as for gemm_run_ex.
 *   workspace        device pointer, 16-byte aligned, not overlapping A, B
 *                    or C; owned by the caller, contents need not be
 *                    initialised and are undefined afterwards.
 *   workspace_bytes  its size.  With a NULL workspace or fewer than
 *                    gemm_workspace_bytes(plan) bytes the call is exactly
 *                    gemm_run_ex (no split).
 * Two launches on `stream` (tile kernel, then the reduction); asynchronous;
 * allocates nothing.  Calls that share one workspace must not overlap in time
 * (issue them on one stream).  Errors as gemm_run_ex, plus
 * GEMM_ERR_INVALID_ARG for a misaligned or overlapping workspace.
 */
int gemm_run_ws(const gemm_plan *plan, const void *A, const void *B, void *C,
                const gemm_epilogue_args *epi, void *workspace, size_t workspace_bytes,
                hipStream_t stream);

/*
 * gemm_run_res -- the fused epilogue with a residual and a saved
 * pre-activation, for layers whose output joins a residual stream and for
 * training:
 *
 *   z[m][n] = (acc[m][n] * sa(m)) * sb(n)  (+ bias[n])      as gemm_run_ex
 *   C[m][n] = cvt( act(z[m][n]) + residual[m][n] )          one rounding
 *   preact[m][n] = cvt( z[m][n] )
 *
 *   A, B, C, epi, stream  as for gemm_run_ex (MX plans: gemm_run_mx_res).
 *   residual  device pointer, M x N of C's type, 16-byte aligned, or NULL (0).
 *             It may be C itself (C is then updated in place); otherwise it
 *             must not overlap C.
 *   preact    device pointer, M x N of C's type, 16-byte aligned, or NULL.
 *             Must not overlap A, B, C, the residual or the workspace.
 *             gemm_act_grad takes it for the backward pass.
 *   workspace, workspace_bytes  as for gemm_run_ws (NULL, 0: no split).  It
 *             must not overlap the residual either.
 * SiLU: the tiled bf16, fp8 and integer kernels evaluate it with the hardware's
 * 2^x and reciprocal, the skinny ones, the split-K reduction, MX plans and the
 * transposed 8-bit layouts with expf and a division.  Both stay within
 * 2^-20 |z|, but the last bit of C may depend on the kernel, and so on M and
 * on whether a workspace is given (as the order of the sums does).
 * Every plan with GEMM_KERNEL_AUTO, GEMM_KERNEL_TILE256 or
 * GEMM_KERNEL_GENERIC_128, and GEMM_KERNEL_PIPE with a pre-shuffled B or
 * W4A8, has this epilogue; GEMM_KERNEL_GENERIC_256, GEMM_KERNEL_PIPE4 and
 * GEMM_KERNEL_PIPE otherwise give GEMM_ERR_UNSUPPORTED when a residual or
 * preact is given.  With neither, the call is gemm_run_ws.  Errors as
 * gemm_run_ws.
 */
int gemm_run_res(const gemm_plan *plan, const void *A, const void *B, void *C, const gemm_epilogue_args *epi,
                 const void *residual, void *preact, void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * gemm_run_ws_noalloc -- gemm_run_ws on the library's own static workspace,
 * for callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation).  The
 * library holds one GEMM_STATIC_WORKSPACE_BYTES array per GPU it runs on,
 * from first use until the process ends; this call allocates nothing and
 * calls no allocating routine.
 *   A, B, C, epi, stream  as for gemm_run_ex.
 * A plan that does not split runs exactly as gemm_run_ex.  A plan whose
 * partials (gemm_workspace_bytes) exceed GEMM_STATIC_WORKSPACE_BYTES is
 * refused with GEMM_ERR_UNSUPPORTED (gemm_run_ws takes any workspace).
 * Every call on one GPU shares that GPU's array, whose contents are whatever
 * the last call left (every element a split reads is written first by the
 * same call, so nothing needs clearing): calls that overlap in time on one
 * GPU race -- issue them on one stream.  Errors as gemm_run_ws.
 */
#define GEMM_STATIC_WORKSPACE_BYTES ((size_t)64 << 20)
int gemm_run_ws_noalloc(const gemm_plan *plan, const void *A, const void *B, void *C,
                        const gemm_epilogue_args *epi, hipStream_t stream);

/*
 * gemm_run_lora -- gemm_run_res with the low-rank adapters of many requests
 * beside the shared B.  Row m of A belongs to adapter a = adapter[m]:
 *
 *   v[m][r] = scale[a] * sum_k A[m][k] * down[a][r][k]                       (fp32)
 *   z[m][n] = sum_k A[m][k] * b(n,k)  +  sum_r v[m][r] * up[a][n][r]  (+ bias[n])
 *   C[m][n] = cvt( act(z[m][n])  (+ residual[m][n]) )          preact[m][n] = cvt( z[m][n] )
 *
 * Both sums over r and k are fp32; v is not rounded to bf16 (it enters the
 * second product as a sum of two bf16 numbers, within 2^-16 of it, or of three,
 * within 2^-24, where the output is fp32; an infinite v stays one).  A row whose
 * adapter is outside 0 .. adapters - 1 has none.  Rows of different adapters
 * may be mixed in any order (above 256 rows it is fast where the rows of one
 * lie together: 8192 x 4096 x 4096 takes 0.25 ms in six runs of rows, 1.8 ms with
 * 64 adapters in random order); an adapter's infinities and NaN reach its own
 * rows only.
 *   adapter  device pointer, M ints;
 *   down     adapters x rank x K bf16, up  adapters x N x rank bf16, 16-byte
 *            aligned (adapters of a lower rank are filled up with zeros);
 *   scale    device pointer, adapters floats, or NULL (1);
 *   adapters 1 .. GEMM_LORA_MAX_ADAPTERS;
 *   rank     a multiple of 8, 8 .. GEMM_LORA_MAX_RANK.
 * Plans: bf16 (either output type) with GEMM_LAYOUT_BT or
 * GEMM_LAYOUT_BT_PRESHUFFLED, M <= GEMM_GROUP_MAX_ROWS.  epi has no scales.
 *   residual, preact  as for gemm_run_res;
 *   workspace  gemm_lora_workspace_bytes(plan, rank) bytes, 16-byte aligned,
 *            contents undefined before and after (v, and the partial tiles
 *            where K is split: above 8192 where the plan splits, and where its
 *            options say so).  Calls that share one must not overlap
 *            in time.
 * The workspace, C and preact overlap no other operand, the bias among them
 * (but C may be the residual).
 * Asynchronous; allocates nothing; two launches (three with split K).  GEMM_OK
 * or an error.
 */
#define GEMM_LORA_MAX_ADAPTERS 65536
#define GEMM_LORA_MAX_RANK 256

typedef struct {
    const int32_t *adapter;
    const void *down;
    const void *up;
    const float *scale;
    int32_t adapters;
    int32_t rank;
} gemm_lora_args;

size_t gemm_lora_workspace_bytes(const gemm_plan *plan, int rank);
int gemm_run_lora(const gemm_plan *plan, const void *A, const void *B, void *C, const gemm_epilogue_args *epi,
                  const gemm_lora_args *lora, const void *residual, void *preact, void *workspace,
                  size_t workspace_bytes, hipStream_t stream);

/*
 * MX block-scaled operands (GEMM_MXFP8_OUT_BF16, GEMM_MXFP4_OUT_BF16).  The
 * pages' gfx950 scaled MFMA (FlyDSL "Kernel authoring guide", section 4.3
 * "ROCm intrinsics", MFMA instructions: mfma_scale_f32_16x16x128_f8f6f4)
 * takes E8M0 block scales per operand with block size 32 (FlyDSL "Kernel
 * Authoring" skill, section 6 "MFMA Integration", gfx1250 WMMA entry); the
 * element and scale formats are those of the OCP Microscaling formats:
 *
 *     C[m][n] = cvt( sum_k (a(m,k) * 2^(SA[m][k/32] - 127)) * (b(n,k) * 2^(SB[n][k/32] - 127)) )
 *
 *   A   M x K elements row-major (MXFP8: 1 byte each; MXFP4: 2 per byte,
 *       element 2t in the low nibble of byte t); B likewise N x K, or its
 *       pre-shuffled image (gemm_preshuffle_b on the bytes: for MXFP4 the
 *       64-byte k-blocks hold 128 elements);
 *   SA  M x K/32 E8M0 bytes row-major, SB N x K/32 (0xFF is NaN).
 * Requirements beyond gemm_plan_create's: K % 32 == 0; K * elem_bits / 8 % 64 == 0.
 * The scales go to the kernel as an image that lets each lane fetch the scales
 * of 4 row blocks for 4 MFMA K-slices (128 elements each) in one 16-byte load:
 * the bytes (ceil(R/64), G, 64, 4, 4), G = ceil(ceil(K/128)/4), row-major:
 * row quad, slice group g, lane l, 16-row block b, slice s holds
 * S[64 quad + 16 b + l % 16][4 (4 g + s) + l / 16] (127 past the rows or K).
 * That is form 0 (gemm_plan_info.scale_form), for the 16x16x128 MFMA.  MX
 * plans on 256 x 256 tiles run the 32x32x64 form of the instruction (twice
 * the e2m1 rate, 8 waves), whose lanes take the scale of row l % 32 and K
 * block 2 s' + l / 32 of 64-element slice s'; their image is form 1, with the
 * same size and record order: (quad, g, lane l, word w, byte b) holds
 * S[64 quad + 32 (w / 2) + l % 32][16 g + 2 (2 b + w % 2) + l / 32].
 * gemm_preshuffle_bscale writes the plan's form.
 */

/* gemm_bscale_image_bytes -- bytes of the image of A's (operand 0) or B's
 * (operand 1) block scales; 0 for a non-MX plan or another operand. */
size_t gemm_bscale_image_bytes(const gemm_plan *plan, int operand);

/*
 * gemm_preshuffle_bscale -- write the image above from R x K/32 E8M0 bytes
 * (R = M for operand 0, N for operand 1).
 *   scales  device pointer, R * K/32 bytes;  image  device pointer, 16-byte
 *   aligned, gemm_bscale_image_bytes(plan, operand) bytes, not overlapping.
 * Asynchronous on `stream`; GEMM_OK or an error (non-MX plan, bad operand,
 * NULL or misaligned pointers, overlap).
 */
int gemm_preshuffle_bscale(const gemm_plan *plan, int operand, const void *scales, void *image,
                           hipStream_t stream);

/*
 * gemm_run_mx -- C = cvt(epilogue(A * B^T)) for an MX plan.
 *   A, B, C    as for gemm_run (B plain or pre-shuffled per the plan's layout).
 *   A_bscale, B_bscale  device pointers to the images of SA and SB, 16-byte
 *              aligned (gemm_preshuffle_bscale).
 *   epi        the fused epilogue (see gemm_run_ex), or NULL.
 * gemm_run and gemm_run_ex reject MX plans.  Asynchronous; GEMM_OK or an error.
 */
int gemm_run_mx(const gemm_plan *plan, const void *A, const void *A_bscale, const void *B,
                const void *B_bscale, void *C, const gemm_epilogue_args *epi, hipStream_t stream);

/*
 * gemm_run_mx_res -- gemm_run_mx with the residual and pre-activation of
 * gemm_run_res (no split K).
 */
int gemm_run_mx_res(const gemm_plan *plan, const void *A, const void *A_bscale, const void *B,
                    const void *B_bscale, void *C, const gemm_epilogue_args *epi, const void *residual,
                    void *preact, hipStream_t stream);

/*
 * Integer operands (GEMM_I8_OUT_BF16, GEMM_W4A8_OUT_BF16).  The pages' int8
 * MFMA accumulates i8 x i8 products in int32 (FlyDSL "Kernel authoring
 * guide", section 4.3 "ROCm intrinsics", MFMA instructions; "Kernel
 * Authoring" skill, section 6 "MFMA Integration"), and their W4A8 GEMM takes
 * an int8 A with a B of packed int4 values unpacked to int8 inside the kernel
 * (the same skill, section 10 "Troubleshooting", INT4 item).  This library's
 * reading:
 *
 *     acc[m][n] = sum_k a(m,k) * b(n,k)            exact, in int32
 *     C[m][n]   = cvt( act( (float(acc) * sa(m)) * sb(n) (+ bias[n]) ) )
 *
 *   int8 two's complement (-128 .. 127); int4 two's complement (-8 .. 7), two
 *   per byte, element 2t in the low nibble of byte t.  float() rounds to
 *   nearest even (exact while |acc| < 2^24).  The scales and epilogue are
 *   those of gemm_run / gemm_run_ex, typically per-row and per-column
 *   dequantisation scales.
 *   A   M x K bytes row-major;  B  N x K bytes (int8) or N x K/2 bytes (int4)
 *       row-major, or the pre-shuffled image (gemm_preshuffle_b on B's bytes:
 *       for int4 a 64-byte k-block holds 128 values).
 * Requirements beyond gemm_plan_create's: K % 64 == 0 (int8) or K % 128 == 0
 * (W4A8), so every row of B is whole 64-byte K steps; K < 2^17, so no sum of
 * products (each at most 2^14 in magnitude) can leave the int32 range.
 * Run through gemm_run or gemm_run_ex.
 */

/* ------------------------------------------------------------------------
 * Products grouped by expert.  A mixture-of-experts layer sends every token to
 * a few of G experts; the rows that go to one expert form a group, and each
 * group is multiplied by its own B.  The groups' sizes are only known on the
 * device: they are given as G + 1 offsets in device memory, group g holding
 * the rows offsets[g] .. offsets[g + 1] - 1, and no call reads them on the host.
 * The usual chain is
 *
 *   gemm_group_sort     expert ids -> offsets, row_token, slot_row
 *   gemm_group_run      up projection (row_index = row_token gathers the tokens)
 *   gemm_group_run      down projection
 *   gemm_group_combine  the weighted sum of each token's rows (slot_row)
 *
 * and backwards gemm_group_combine_grad, gemm_act_grad, gemm_group_run with
 * GEMM_LAYOUT_BN (input gradients) and GEMM_LAYOUT_AT_BN (weight gradients),
 * and gemm_group_combine without weights (the gradient of the gather).  The
 * weight gradient has no row_index: for the up projection the caller gathers
 * the tokens' rows (row_token) into an array of their own first.
 * ------------------------------------------------------------------------ */
#define GEMM_GROUP_MAX 1024                 /* most groups                            */
#define GEMM_GROUP_MAX_ROWS ((int64_t)1 << 24)   /* most rows (or slots) of one call */

typedef enum {
    GEMM_TYPE_F32 = 0,
    GEMM_TYPE_BF16 = 1,
    GEMM_TYPE_E4M3 = 2          /* weights of gemm_group_mlp_run only */
} gemm_type;

typedef struct gemm_group_plan gemm_group_plan;   /* opaque, immutable after creation */

/*
 * gemm_group_plan_create -- validate a grouped product and pick its kernel.
 *   groups   G, 1 .. GEMM_GROUP_MAX.
 *   M, N, K, dtype, layout  as for gemm_plan_create, with:
 *     GEMM_LAYOUT_BT, GEMM_LAYOUT_BT_PRESHUFFLED, GEMM_LAYOUT_BN (bf16): the
 *       ROWS are grouped.  A is M x K and C is M x N, M being the number of
 *       rows they have room for (offsets[G] may be less); B is G matrices,
 *       N x K each (BN: K x N each), one behind the other.  Row r of group g:
 *           C[r] = cvt( epilogue( A[r] * B_g^T ) )     (BN: A[r] * B_g)
 *     GEMM_LAYOUT_AT_BN (bf16): the INNER size is grouped.  A is K x M and B
 *       is K x N, K being the number of rows they have room for; C is G
 *       matrices M x N.  Every matrix of C is written, zeros for an empty
 *       group:
 *           C_g = cvt( sum over rows r of group g of A[r]^T * B[r] )
 *       K may be any number here; M * 2 % 16 == 0; M < 2^24 (a step's 64
 *       rows of A stay inside one 2^31-byte buffer range).
 *   dtype    GEMM_BF16_OUT_F32, GEMM_BF16_OUT_BF16, GEMM_E4M3_OUT_BF16 (the
 *            last with GEMM_LAYOUT_BT and GEMM_LAYOUT_BT_PRESHUFFLED).
 * The other requirements are gemm_plan_create's (N % 16 == 0; K * elem_bytes
 * % 64 == 0 where rows are grouped; ...); grouped rows at most
 * GEMM_GROUP_MAX_ROWS; all tiles of one launch together fewer than 2^32
 * threads (gemm_group_plan_info: grid * threads).  Host only.  NULL on error;
 * freed with gemm_group_plan_destroy.
 */
gemm_group_plan *gemm_group_plan_create(int groups, int64_t M, int64_t N, int64_t K, int dtype, int layout);

/*
 * gemm_group_plan_create_opt -- the same with the kernel named by the rows of
 * its tiles: 32, 64, 128 (not GEMM_LAYOUT_AT_BN) or 256; 0 the planner's own
 * choice from M / groups.  Every choice computes the same C
 * within the same bound.  GEMM_ERR_UNSUPPORTED when the family has no kernel
 * for the dtype and layout.
 */
gemm_group_plan *gemm_group_plan_create_opt(int groups, int64_t M, int64_t N, int64_t K, int dtype, int layout,
                                            int tile_rows);
void gemm_group_plan_destroy(gemm_group_plan *plan);

typedef struct {
    int64_t M, N, K;
    int32_t groups, dtype, layout;
    int32_t tile_m, tile_n;
    int32_t threads, lds_bytes;
    int32_t grid;            /* workgroups of one launch (an upper bound on the tiles) */
} gemm_group_plan_info;
int gemm_group_plan_query(const gemm_group_plan *plan, gemm_group_plan_info *info);

/*
 * gemm_group_preshuffled_b_bytes, gemm_group_preshuffle_b -- the pre-shuffled
 * images of the G matrices B, one behind the other (gemm_preshuffle_b on
 * each).  Arguments and errors as there; 0 bytes for the layouts without an
 * image.
 */
size_t gemm_group_preshuffled_b_bytes(const gemm_group_plan *plan);
int gemm_group_preshuffle_b(const gemm_group_plan *plan, const void *B, void *B_shuf, hipStream_t stream);

/*
 * gemm_group_run -- the grouped product on `stream`.
 *   A, B, C    device pointers, 16-byte aligned, as described above.
 *   offsets    device pointer, G + 1 ints, not decreasing, 0 <= offsets[0],
 *              offsets[G] <= M (AT_BN: K).  Values outside are clamped to that
 *              range; rows of C outside every group are left as they were.
 *              Each row may belong to one group only.
 *   row_index  device pointer to M ints, or NULL.  Given, A has a_rows rows and
 *              row r of C is made from row row_index[r] of A (the gather of the
 *              tokens, without a copy); an index outside 0 .. a_rows - 1 stands
 *              for a row of zeros.  a_rows * K * elem_bytes < 2^31.  Not for
 *              GEMM_LAYOUT_AT_BN.
 *   a_rows     rows of A when row_index is given (ignored otherwise).
 *   epi        the fused epilogue, or NULL: scale_a one value or one per row of
 *              A; scale_b one value, or G x N values (per column of every
 *              group); bias G x N values.  AT_BN: NULL or scales of one value
 *              and GEMM_EPI_NONE.
 *   preact     device pointer, M x N of C's type, 16-byte aligned, or NULL: the
 *              pre-activation, as for gemm_run_res.  Not for AT_BN.
 * Asynchronous; allocates nothing; one launch.  Errors as gemm_run_ex.
 */
int gemm_group_run(const gemm_group_plan *plan, const void *A, const void *B, void *C, const int32_t *offsets,
                   const int32_t *row_index, int64_t a_rows, const gemm_epilogue_args *epi, void *preact,
                   hipStream_t stream);

/*
 * gemm_group_sort -- the tables of the grouped calls from the experts' ids.
 *   ids        device pointer, `slots` ints: slot s = token * topk + j holds
 *              the j-th expert of the token.  An id outside 0 .. groups - 1 is
 *              a slot that goes nowhere (an expert of another rank, padding).
 *   slots      number of ids, at most GEMM_GROUP_MAX_ROWS, a multiple of topk.
 *   offsets    groups + 1 ints out: where each group's rows start.
 *   row_token  `slots` ints out: the token (s / topk) of every sorted row; the
 *              entries from offsets[groups] on are left as they were.
 *   slot_row   `slots` ints out: the sorted row of every slot, -1 for a slot
 *              that goes nowhere.
 * The rows of a group keep the order of their slots (a stable sort, so the
 * result is the same on every run).
 *   workspace  gemm_group_sort_workspace_bytes(slots, groups) bytes of device
 *              memory, 4-byte aligned, contents undefined before and after;
 *              NULL when that is 0.  Calls that share one must not overlap in
 *              time.
 * The outputs overlap neither each other nor the ids or the workspace.
 * Asynchronous; allocates nothing.  GEMM_OK or an error.
 */
size_t gemm_group_sort_workspace_bytes(int64_t slots, int groups);
int gemm_group_sort(const int32_t *ids, int64_t slots, int topk, int groups, int32_t *offsets, int32_t *row_token,
                    int32_t *slot_row, void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * gemm_group_combine -- every token's rows brought back together:
 *
 *   out[t][n] = cvt( sum over j of weights[t][j] * src[slot_row[t][j]][n]  (+ residual[t][n]) )
 *
 * summed in fp32 in the order of j, the residual last.  A slot_row outside
 * 0 .. src_rows - 1 contributes nothing (its weight is not read as a factor:
 * an infinite or NaN weight of such a slot does not reach the output).
 *   tokens, topk  0 .. GEMM_GROUP_MAX_ROWS tokens, 1 .. 64 slots per token;
 *                 N % 16 == 0.
 *   type       gemm_type of src, residual and out.
 *   src        src_rows x N;  slot_row  tokens x topk ints;
 *   weights    tokens x topk floats, or NULL (1);
 *   residual   tokens x N or NULL; may be out itself, else no overlap;
 *   out        tokens x N, not overlapping src.
 * src, residual and out 16-byte aligned.  Asynchronous; GEMM_OK or an error.
 */
int gemm_group_combine(int64_t tokens, int topk, int64_t N, int type, const void *src, int64_t src_rows,
                       const int32_t *slot_row, const float *weights, const void *residual, void *out,
                       hipStream_t stream);

/*
 * gemm_group_combine_grad -- the gradient of that sum:
 *
 *   d_src[slot_row[t][j]][n] = cvt( weights[t][j] * d_out[t][n] )
 *   d_weights[t][j] = sum over n of d_out[t][n] * src[slot_row[t][j]][n]     (0 for a slot that goes nowhere)
 *
 * Every row may be named by one slot only (as gemm_group_sort's table does);
 * rows of d_src that no slot names are left as they were.  d_weights is fp32
 * or NULL (src may then be NULL too); weights NULL stands for 1.  d_src does
 * not overlap src or d_out.  The residual's gradient is d_out itself.
 * Otherwise as gemm_group_combine.
 */
int gemm_group_combine_grad(int64_t tokens, int topk, int64_t N, int type, const void *d_out, const void *src,
                            int64_t src_rows, const int32_t *slot_row, const float *weights, void *d_src,
                            float *d_weights, hipStream_t stream);

/*
 * gemm_group_mlp_* -- a whole mixture-of-experts layer for a few tokens
 * (decode), two launches without routing tables: slot s = t * topk + j holds
 * token t's j-th expert e = ids[s],
 *
 *   gated:  h[s][n] = cvt( act(g[s][n]) * u[s][n] )       else  h[s][n] = cvt( act(u[s][n]) )
 *   g[s][n] = (sum_k x[t][k] * up[e][n][k])     * up_scale[e][n]     + up_bias[e][n]
 *   u[s][n] = (sum_k x[t][k] * up[e][N + n][k]) * up_scale[e][N + n] + up_bias[e][N + n]      (not gated: n for N + n)
 *   o[s][k] = (sum_n h[s][n] * down[e][k][n])   * down_scale[e][k]   + down_bias[e][k]
 *   out[t][k] = cvt( sum over j of weights[t][j] * o[s][k]  (+ residual[t][k]) )
 *
 * sums, scales, biases and activations in fp32; h is rounded to bf16 (as the
 * chain of single products keeps it), o is not.  The sum over j runs in the
 * order of j, the residual last.  A slot whose id is outside 0 .. groups - 1
 * contributes nothing (nor is its weight read as a factor).  The result does
 * not depend on scheduling: every run gives the same bits.  For more tokens
 * there are gemm_group_sort, gemm_group_run and gemm_group_combine: without the
 * gate's product, which is the caller's between two runs, and with rows of the
 * weights' type (e4m3 beside e4m3 weights).
 *
 * gemm_group_mlp_plan_create
 *   groups   1 .. GEMM_GROUP_MAX;  tokens 0 .. GEMM_GROUP_MLP_MAX_TOKENS;
 *   topk     1 .. GEMM_GROUP_MLP_MAX_TOPK;
 *   K, N     the model's width and an expert's hidden width, 1 .. 2^20;
 *            multiples of 32 (bf16 weights) or 64 (e4m3);
 *            tokens * topk * N < 2^30.
 *   weight_type  GEMM_TYPE_BF16 or GEMM_TYPE_E4M3 (products exact, as bf16).
 *   layout   GEMM_LAYOUT_BT or GEMM_LAYOUT_BT_PRESHUFFLED, of both matrices.
 *   gated    1: up holds 2 N rows per expert (the N gate rows first); 0: N.
 *   epilogue a gemm_epilogue: which activation (NONE and BIAS: none).
 * Host only.  NULL on error; freed with gemm_group_mlp_plan_destroy.
 */
#define GEMM_GROUP_MLP_MAX_TOKENS 64
#define GEMM_GROUP_MLP_MAX_TOPK 64

typedef struct gemm_group_mlp_plan gemm_group_mlp_plan;   /* opaque, immutable after creation */

gemm_group_mlp_plan *gemm_group_mlp_plan_create(int groups, int64_t tokens, int topk, int64_t K, int64_t N,
                                                int weight_type, int layout, int gated, int epilogue);
void gemm_group_mlp_plan_destroy(gemm_group_mlp_plan *plan);

typedef struct {
    int64_t tokens, K, N;
    int32_t groups, topk, weight_type, layout, gated, epilogue;
} gemm_group_mlp_plan_info;
int gemm_group_mlp_plan_query(const gemm_group_mlp_plan *plan, gemm_group_mlp_plan_info *info);

/* gemm_group_mlp_workspace_bytes -- bytes gemm_group_mlp_run needs (0: no tokens, or NULL). */
size_t gemm_group_mlp_workspace_bytes(const gemm_group_mlp_plan *plan);

/*
 * gemm_group_mlp_preshuffle -- the pre-shuffled images of both matrices (each
 * as large as its source; gemm_group_preshuffle_b on each).  All four are
 * 16-byte aligned, the images overlap neither a matrix nor each other, and
 * nothing is launched where one is refused.  For plans with
 * GEMM_LAYOUT_BT_PRESHUFFLED.
 */
int gemm_group_mlp_preshuffle(const gemm_group_mlp_plan *plan, const void *up, void *up_image, const void *down,
                              void *down_image, hipStream_t stream);

/*
 * gemm_group_mlp_weights -- the experts' matrices (device pointers).
 *   up    groups x (gated ? 2 N : N) x K;  down  groups x K x N; each as is or
 *         its image, as the plan's layout says; 16-byte aligned.
 *   up_scale, up_bias      groups x (gated ? 2 N : N) floats, or NULL (1, 0);
 *   down_scale, down_bias  groups x K floats, or NULL (1, 0).
 */
typedef struct {
    const void *up;
    const void *down;
    const float *up_scale;
    const float *down_scale;
    const float *up_bias;
    const float *down_bias;
} gemm_group_mlp_weights;

/*
 * gemm_group_mlp_run -- the layer on `stream`.
 *   x         tokens x K bf16, 16-byte aligned;  ids  tokens x topk ints;
 *   weights   tokens x topk floats (the router's), or NULL (1);
 *   mats      host pointer, read during the call only;
 *   residual  tokens x K bf16, 16-byte aligned, or NULL; may be out itself;
 *   out       tokens x K bf16, 16-byte aligned, overlapping no other operand;
 *   workspace gemm_group_mlp_workspace_bytes(plan) bytes, 16-byte aligned,
 *             contents undefined before and after.  Calls that share one must
 *             not overlap in time.
 * Asynchronous; allocates nothing; two launches.  GEMM_OK or an error.
 */
int gemm_group_mlp_run(const gemm_group_mlp_plan *plan, const void *x, const int32_t *ids, const float *weights,
                       const gemm_group_mlp_weights *mats, const void *residual, void *out, void *workspace,
                       size_t workspace_bytes, hipStream_t stream);

/*
 * gemm_act_grad -- the gradient of the fused epilogue, from the saved
 * pre-activation z (gemm_run_res, gemm_group_run):
 *
 *   d_z[m][n] = cvt( d_c[m][n] * act'(z[m][n]) )
 *   d_bias[g][n] = sum over the rows m of group g of d_c[m][n] * act'(z[m][n])     (fp32, before the rounding)
 *
 *   act': 1; ReLU z > 0; SiLU s(z) (1 + z (1 - s(z))), s the logistic function;
 *   GELU Phi(z) + z phi(z).  0 is taken where z is -inf (SiLU, GELU).
 *   M, N       rows and columns (N % 16 == 0, M <= GEMM_GROUP_MAX_ROWS).
 *   type       gemm_type of d_c, z and d_z (16-byte aligned).
 *   epilogue   gemm_epilogue: which activation (NONE and BIAS: none).
 *   z          M x N; may be NULL without an activation.
 *   d_z        M x N; may be d_c or z itself, else no overlap with them.
 *   d_bias     groups x N floats, 16-byte aligned, or NULL.
 *   groups, offsets  the row groups (G + 1 device ints, as for
 *              gemm_group_run); offsets NULL: one group of M rows (groups is
 *              then 1).  Rows outside every group: d_z is left as it was.
 *   workspace  gemm_act_grad_workspace_bytes(M, N, groups) bytes when d_bias is
 *              given (16-byte aligned, contents undefined before and after);
 *              not read otherwise.  Calls that share one must not overlap in
 *              time.
 * d_bias is summed in a fixed order (no atomics): the same on every run.
 * Asynchronous; allocates nothing.  GEMM_OK or an error.
 */
size_t gemm_act_grad_workspace_bytes(int64_t M, int64_t N, int groups);
int gemm_act_grad(int64_t M, int64_t N, int type, int epilogue, const void *d_c, const void *z, void *d_z,
                  float *d_bias, int groups, const int32_t *offsets, void *workspace, size_t workspace_bytes,
                  hipStream_t stream);

/* ------------------------------------------------------------------------
 * Activations kept in 8 bits between the forward and the backward pass.  Of a
 * row's every 32 columns (the last block of a row may have 16) the checkpoint
 * holds e4m3 elements and one power of two:
 *
 *   s[m][b] = the smallest power of two, 2^-127 or more, with |x| <= 448 s for every finite x of the block
 *   q[m][n] = e4m3( x[m][n] / s )        (nearest even; no element is clipped; Inf and NaN become NaN)
 *   value   = q[m][n] * s[m][n / 32]
 *
 *   q       M x N bytes row-major, 16-byte aligned;
 *   scales  M x ceil(N / 32) bytes row-major, E8M0: s = 2^(byte - 127), 255 NaN.
 * 33 / 32 bytes per element instead of 2 or 4, each within 2^-4 of itself (and
 * within 2^-10 s near zero); a finite |x| of 2^128 (1 - 2^-5) or more is rounded
 * to 2^128, which fp32 and bf16 hold as infinity.  With N a multiple of 64 the pair is an operand of
 * the MXFP8 products (q as A or B, scales through gemm_preshuffle_bscale).
 *
 * The usual use: gemm_run_res or gemm_group_run saves the pre-activation z,
 * gemm_ckpt_pack keeps it; backwards gemm_act_grad_ckpt makes d_z from it, and
 * gemm_ckpt_unpack with the activation makes the layer's output again, the
 * operand of the next layer's weight gradient (GEMM_LAYOUT_AT_BN).
 *   M, N    rows and columns: 0 .. GEMM_GROUP_MAX_ROWS; N % 16 == 0, N < 2^21.
 *   type    gemm_type of src, out, d_c and d_z (GEMM_TYPE_F32 or GEMM_TYPE_BF16).
 * ------------------------------------------------------------------------ */

/*
 * gemm_ckpt_pack -- src (M x N, 16-byte aligned) into q and scales.  None of
 * the three overlap.  Asynchronous; one launch; GEMM_OK or an error.
 */
int gemm_ckpt_pack(int64_t M, int64_t N, int type, const void *src, void *q, void *scales, hipStream_t stream);

/*
 * gemm_ckpt_unpack -- out[m][n] = cvt( act(value) ), act the activation of
 * `epilogue` (a gemm_epilogue; NONE and BIAS: none).  out is 16-byte aligned and
 * overlaps neither q nor scales.  Asynchronous; one launch; GEMM_OK or an error.
 */
int gemm_ckpt_unpack(int64_t M, int64_t N, int type, int epilogue, const void *q, const void *scales, void *out,
                     hipStream_t stream);

/*
 * gemm_act_grad_ckpt -- gemm_act_grad with z read from its checkpoint (q and
 * scales may be NULL without an activation).  GELU's normal distribution is
 * within 2^-23 in fp32 and, here and in gemm_ckpt_unpack, within 2^-21 (before
 * the result's rounding; d_bias sums it as it is) in bf16.  d_z may be d_c, and overlaps
 * neither q nor scales.  The workspace is gemm_act_grad_workspace_bytes.
 */
int gemm_act_grad_ckpt(int64_t M, int64_t N, int type, int epilogue, const void *d_c, const void *q,
                       const void *scales, void *d_z, float *d_bias, int groups, const int32_t *offsets,
                       void *workspace, size_t workspace_bytes, hipStream_t stream);

/* gemm_last_error -- message for the calling thread's last failure ("" if none). */
const char *gemm_last_error(void);

/* ------------------------------------------------------------------------
 * Planner introspection (host only).  A layout is (shape, stride) of up to
 * GEMM_MAX_RANK modes; a coordinate maps to sum(c_i * stride_i) (Kernel
 * Authoring skill, section 2 "Layout System", "Coordinate Mapping").
 * ------------------------------------------------------------------------ */
#define GEMM_MAX_RANK 8

typedef struct {
    int64_t M, N, K;
    int32_t dtype, layout;
    int32_t elem_bytes, out_bytes;
    int32_t kernel;          /* 0 tiled, 1 skinny (M <= 64, B N x K or pre-shuffled)  */
    int32_t tile_m, tile_n;  /* output tile of one workgroup                          */
    int32_t tile_k_bytes;    /* K bytes consumed per main-loop step (multiple of 64)  */
    int32_t threads;         /* threads per workgroup                                 */
    int32_t lds_stages;      /* LDS buffers in the software pipeline                  */
    int32_t lds_bytes;       /* static LDS per workgroup (<= 160 KiB on gfx950)       */
    int32_t grid;            /* workgroups per gemm_run launch                        */
    int32_t tiles_m, tiles_n;
    int32_t group_m;         /* tile rows per raster group within one XCD             */
    int32_t split_k;         /* K slices reduced inside a workgroup (skinny kernel)   */
    int32_t elem_bits;       /* bits per input element of A (16, 8 or 4); elem_bytes
                                is elem_bits / 8, so 0 for MXFP4                       */
    int32_t b_elem_bits;     /* bits per input element of B (4 for W4A8, else elem_bits) */
    int32_t ws_splits;       /* K slices gemm_run_ws uses with a large enough
                                workspace (1: it runs as gemm_run_ex)                 */
    int32_t ws_grid;         /* workgroups of gemm_run_ws's tile launch               */
    int32_t scale_form;      /* MX plans: form of the block-scale image (0 or 1, see
                                gemm_preshuffle_bscale); 0 for other plans            */
} gemm_plan_info;

/* gemm_plan_query -- copy the plan's decisions into *info. */
int gemm_plan_query(const gemm_plan *plan, gemm_plan_info *info);

typedef enum {
    GEMM_VIEW_A = 0,          /* A bytes:       (M, Ka):(Ka, 1), Ka = K * elem_bits / 8;
                                 A stored K x M: (K, 2M):(2M, 1)                            */
    GEMM_VIEW_B = 1,          /* B bytes:       (N, Kb):(Kb, 1), Kb = K * b_elem_bits / 8    */
    GEMM_VIEW_B_SHUF = 2,     /* pre-shuffled:  (N/16, Kb/64, 4, 16, 16):(16Kb, 1024, 256, 16, 1) */
    GEMM_VIEW_B_SRC = 3,      /* B bytes seen through the same 5 coordinates:
                                 (N/16, Kb/64, 4, 16, 16):(16Kb, 64, 16, Kb, 1)           */
    GEMM_VIEW_C = 4,          /* C bytes:       (M, N):(N*out_bytes, out_bytes)              */
    GEMM_VIEW_LDS_A = 5,      /* one LDS stage of A, before the XOR swizzle:
                                 (tile_m, tile_k_bytes/16, 16):(tile_k_bytes, 16, 1)     */
    GEMM_VIEW_TILE = 6        /* C tile grid:   (tiles_m, tiles_n):(tile_m*N*ob, tile_n*ob) */
} gemm_view;

/* gemm_plan_layout -- the byte layout of one view; rank and GEMM_MAX_RANK-long arrays out. */
int gemm_plan_layout(const gemm_plan *plan, int view, int32_t *rank, int64_t *shape, int64_t *stride);

/* gemm_layout_crd2idx -- sum(crd_i * stride_i); -1 and GEMM_ERR_INVALID_ARG
 * in gemm_last_error when a coordinate lies outside its mode. */
int64_t gemm_layout_crd2idx(int32_t rank, const int64_t *shape, const int64_t *stride, const int64_t *crd);

/* gemm_layout_idx2crd -- c_i = (idx / stride_i) % shape_i (the inverse of
 * crd2idx on an injective layout whose modes do not overlap). */
int gemm_layout_idx2crd(int32_t rank, const int64_t *shape, const int64_t *stride, int64_t idx, int64_t *crd);

/* gemm_lds_swizzle -- physical 16-byte chunk of logical chunk `chunk` of row
 * `row` in an LDS tile of `chunks_per_row` chunks (the XOR-16 swizzle the
 * pages name in section 6 of the Kernel Authoring skill; the function is this
 * library's choice).  -1 on bad arguments. */
int32_t gemm_lds_swizzle(int32_t row, int32_t chunk, int32_t chunks_per_row);

/* gemm_tile_of_workgroup -- the (tile_m index, tile_n index) the plan's
 * XCD-aware raster assigns to workgroup `wg` (0 <= wg < grid). */
int gemm_tile_of_workgroup(const gemm_plan *plan, int32_t wg, int32_t *tm, int32_t *tn);

#ifdef __cplusplus
}
#endif

#endif /* TGEMM_H */
