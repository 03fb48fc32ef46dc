/*
 * gemm_bt.h -- C = A * B^T on one AMD Instinct MI355X (gfx950).
 *
 * The operation.  C[i][j] = sum_k A[i][k] * B[j][k] for 0 <= i < M, 0 <= j < N,
 * with A stored M x K row-major and B stored N x K row-major, i.e. B is kept
 * transposed so both operands are read along K ("Optimizing Blackwell matrix
 * multiplication in Mojo (part 2)", sections "Starting from the 4-line kernel"
 * and "Kernel 2: TMA and Tensor Core", where B is laid out row_major(N, K) so
 * its loads coalesce).  Inputs are bf16, f16 or one of the OCP 8-bit float
 * formats E4M3 / E5M2 (both operands the same type, as the MMA contract of
 * "Writing Mosaic GPU kernels with Pallas", section "MMA (TensorCore)",
 * requires; the pages list 8-bit floats among the supported MMA element
 * types); products are accumulated in fp32 and the
 * result is rounded once, to nearest even, into the output type ("Chapter 7:
 * Writing custom kernels with Pallas", section 4.1': fp32 accumulator, cast
 * only after the last K step).  8-bit integer inputs (two's complement) are
 * the integer MMA operand type of the same Mosaic GPU section, with an int32
 * accumulator: there C is the exact int32 sum, and int8 in requires int32
 * out (and int32 out requires int8 in).  C is overwritten: there is no
 * alpha/beta.
 *
 * Layout.  Dense and contiguous: lda = ldb = K elements, ldc = N elements.
 * For 16-bit inputs pointers need only element alignment (2 bytes, 4 bytes for
 * fp32 output); 16-byte alignment together with K % 8 == 0 selects the
 * widest loads and is a performance matter only.  8-bit inputs (float or
 * integer) need whole 16-byte rows: K % 16 == 0 and A, B 16-byte aligned
 * (else UNSUPPORTED).  int8 inputs also need K <= 131071, so that no sum can
 * leave the int32 range (|A[i][k] * B[j][k]| <= 2^14).
 *
 * Ownership.  The caller owns A, B and C (device memory, e.g. from PyTorch),
 * and the workspace of gemm_bt_ws.  The library allocates nothing per call,
 * keeps no pointer after it returns and holds no state beyond a per-device
 * cache of device attributes.
 *
 * Asynchrony and errors.  gemm_bt enqueues its kernel on `stream` (two
 * kernels in stream order for a plan with split_rows or split_items) and
 * returns without waiting.  Argument errors are reported before anything is
 * enqueued.  A launch failure is reported as GEMM_BT_ERR_LAUNCH; a fault
 * inside the kernel shows at the caller's next synchronisation.  No call
 * throws, exits or aborts.  Calls are thread-safe.  C must not overlap A or B.
 */
#ifndef GEMM_BT_H
#define GEMM_BT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
typedef enum {
    GEMM_BT_F32 = 0,      /* IEEE binary32 (output only) */
    GEMM_BT_F16 = 1,      /* IEEE binary16 */
    GEMM_BT_BF16 = 2,     /* bfloat16: the upper 16 bits of a binary32 */
    GEMM_BT_FP8_E4M3 = 3, /* OCP 8-bit E4M3 (input only): bias 7, no infinities, max 448 */
    GEMM_BT_FP8_E5M2 = 4, /* OCP 8-bit E5M2 (input only): bias 15, IEEE-style infinities */
    GEMM_BT_INT8 = 5,     /* two's-complement 8-bit integer (input only; output GEMM_BT_INT32) */
    GEMM_BT_INT32 = 6     /* two's-complement 32-bit integer (output only; input GEMM_BT_INT8) */
} gemm_bt_dtype;

/* Operand layouts for gemm_bt_layout. */
typedef enum {
    GEMM_BT_K_INNER = 0, /* A stored M x K, B stored N x K (K contiguous): the gemm_bt layout */
    GEMM_BT_K_OUTER = 1  /* A stored K x M (M contiguous), B stored K x N (N contiguous) */
} gemm_bt_layout_t;

/* Status codes returned by every entry point. */
typedef enum {
    GEMM_BT_OK = 0,
    GEMM_BT_ERR_INVALID_VALUE = 1, /* negative size, null pointer with data, bad plan pointer */
    GEMM_BT_ERR_UNSUPPORTED = 2,   /* dtype combination or size outside the supported range */
    GEMM_BT_ERR_NO_DEVICE = 3,     /* no HIP device, or it is not a gfx950 */
    GEMM_BT_ERR_LAUNCH = 4         /* the kernel launch failed */
} gemm_bt_status;

/*
 * C = A * B^T.
 *   A          device pointer, M x K elements of in_dtype, row-major
 *   B          device pointer, N x K elements of in_dtype, row-major (B^T stored)
 *   C          device pointer, M x N elements of out_dtype, row-major; overwritten
 *   M, N, K    sizes, each in [0, 2^31 - 1]; M*K, N*K and M*N elements must each
 *              fit below 2^31 bytes per 256-row panel (checked: UNSUPPORTED);
 *              8-bit inputs: K % 16 == 0 and A, B 16-byte aligned (UNSUPPORTED);
 *              int8 inputs: K <= 131071 (UNSUPPORTED)
 *   in_dtype   GEMM_BT_BF16, GEMM_BT_F16, GEMM_BT_FP8_E4M3, GEMM_BT_FP8_E5M2 or GEMM_BT_INT8
 *   out_dtype  GEMM_BT_F32, GEMM_BT_BF16 or GEMM_BT_F16 for float inputs; GEMM_BT_INT32
 *              for GEMM_BT_INT8 inputs (any other pairing: UNSUPPORTED)
 *   stream     hipStream_t to enqueue on; NULL means the default stream
 * M == 0 or N == 0: nothing is enqueued, returns GEMM_BT_OK.
 * K == 0: C is filled with zeros (the empty sum) on `stream`.
 * The device is the caller's current HIP device.
 */
int gemm_bt(const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K,
            int in_dtype, int out_dtype, void* stream);

/*
 * Batched product: C_z = A_z * B_z^T for z = 0 .. batch-1, every item with
 * the same sizes and types ("Chapter 7: Writing custom kernels with Pallas",
 * section 5.2: batching a kernel adds a leading grid dimension and runs the
 * unchanged kernel once per item; an operand mapped with in_axes=None is
 * shared by all items rather than copied).  One launch covers all items.
 *   A, B, C    base device pointers; item z uses A + z*stride_a, B + z*stride_b
 *              and C + z*stride_c (strides in elements of the operand's type)
 *   batch      number of items, 0 .. 65535 (0: nothing enqueued; more: UNSUPPORTED)
 *   stride_a   >= 0; 0 shares one A between all items (likewise stride_b for B)
 *   stride_c   >= M*N when batch > 1, so items of C never overlap (INVALID_VALUE)
 * Strides are ignored when batch == 1.  Alignment rules apply to every item's
 * pointers (the base pointers and the strides in bytes): e.g. 8-bit inputs
 * need 16-byte aligned A and B items.  Everything else is as for gemm_bt,
 * which is the batch == 1 case of this call.  Negative sizes or strides:
 * INVALID_VALUE.
 */
int gemm_bt_batched(const void* A, const void* B, void* C, int64_t batch, int64_t M, int64_t N, int64_t K,
                    int64_t stride_a, int64_t stride_b, int64_t stride_c, int in_dtype, int out_dtype,
                    void* stream);

/*
 * C = op(A) * op(B)^T with either operand stored K-outer ("Writing Mosaic GPU
 * kernels with Pallas", section "MMA (TensorCore)", transposed operands: for
 * 16-bit operands an A of shape (K, M), and likewise a B of shape (K, N), is
 * accepted and transposed by the hardware).  a_layout = GEMM_BT_K_OUTER: A is
 * K x M row-major; b_layout = GEMM_BT_K_OUTER: B is K x N row-major, so
 * (K_INNER, K_OUTER) is the plain C = A * B.  Both K_INNER is exactly gemm_bt.
 * Operands stored K-outer are transposed inside the kernel (LDS transpose
 * reads); nothing is copied.  Requirements (else UNSUPPORTED): bf16 or f16
 * inputs; every operand row in whole 16-byte chunks (M % 8 == 0 for a K-outer
 * A, N % 8 == 0 for a K-outer B, K % 8 == 0 for a K-inner operand) and A, B
 * 16-byte aligned; a K-outer operand below 2 GiB.  An unknown layout value is
 * INVALID_VALUE.  Everything else (C, sizes, K == 0, streams, errors) is as
 * for gemm_bt.
 */
int gemm_bt_layout(const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K, int a_layout,
                   int b_layout, int in_dtype, int out_dtype, void* stream);

/*
 * Batched products with operand layouts: gemm_bt_batched's items (item z at
 * A + z*stride_a, B + z*stride_b, C + z*stride_c elements; a stride of 0
 * shares an operand; stride_c >= M*N when batch > 1) with each operand stored
 * as gemm_bt_layout's a_layout / b_layout say.  An item of a K-outer A is a
 * K x M matrix, of a K-outer B a K x N one.  The rules of both calls apply, to
 * every item's pointers; gemm_bt_layout is the batch == 1 case and
 * gemm_bt_batched the (K_INNER, K_INNER) one.
 */
int gemm_bt_batched_layout(const void* A, const void* B, void* C, int64_t batch, int64_t M, int64_t N, int64_t K,
                           int64_t stride_a, int64_t stride_b, int64_t stride_c, int a_layout, int b_layout,
                           int in_dtype, int out_dtype, void* stream);

/*
 * C = A * B^T with a caller-provided workspace that lets the library split
 * the K range of output tiles over workgroups (the work split of stream-K:
 * "Writing Mosaic GPU kernels with Pallas", section "Cluster launch
 * control", a grid that keeps every core busy to the end).  Where a 16-bit
 * product would leave at least half the compute units without an output
 * tile and K is long, each of its T tiles is split into S pieces of
 * consecutive K steps (at least 32 steps of 64 each), one piece per
 * workgroup.  The tiles: 32 x 64 for M <= 32, 64 x 64 for M <= 64 (thin
 * products, in K steps of 128, e.g. 64 x 8192 x 8192: 128 tiles, S = 2),
 * else 128 x 128 (e.g.
 * 1024 x 1024 x 16384: 64 tiles, S = 4); S = floor(CUs / T), for thin
 * products at most K / 2048 (then S >= 2 is required), and for 128 x 128 tiles
 * no split when M fills less than 3/4 of their rows while narrower tiles
 * already give every compute unit a workgroup.  The last of a tile's
 * workgroups to finish adds the pieces in K
 * order (piece 0 + 1 + ...), whatever the order of arrival, so the result
 * is the same bits on every run with the same sizes on the same device.
 * The sum of each output is then formed in a different order than gemm_bt's
 * (pieces summed in fp32, then added), with the same accuracy bound.  Where
 * no split is planned (every other shape, batches, 8-bit inputs, operands
 * stored K-outer) the call is exactly gemm_bt.
 *   A, B, C, M, N, K, in_dtype, out_dtype, stream: as for gemm_bt
 *   workspace        device memory of at least workspace_bytes, 16-byte
 *                    aligned, owned by the caller, or NULL (then the call is
 *                    gemm_bt).  Its first 16 KiB must hold zeros before the
 *                    first call that uses it (e.g. hipMemset once after
 *                    allocation); every call leaves them zero again, so one
 *                    workspace serves any number of later calls with no
 *                    clearing.  Calls that share a workspace must not run
 *                    concurrently (one stream, or ordered by events).
 *   workspace_bytes  its size; smaller than gemm_bt_workspace_size reports for
 *                    these sizes: INVALID_VALUE (nothing enqueued)
 * Everything else (sizes, dtypes, K == 0, alignment, errors) is as for gemm_bt.
 */
int gemm_bt_ws(const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K, int in_dtype,
               int out_dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * gemm_bt_ws without a workspace argument, for callers that cannot allocate
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the split plan's counters and partial sums live in a scratch
 * array of the library's own in device memory, 16 KiB + 16 MiB (the largest
 * split plan on a GPU of up to 256 compute units), one copy per GPU, held
 * until the process ends.  The call allocates nothing (no hipMalloc, no
 * allocating library routine).  Same arguments, plan, kernels and results as
 * gemm_bt_ws with a large enough workspace (bit for bit); where no split is
 * planned it is gemm_bt.  A plan that would need more scratch than that
 * (more than 256 compute units): UNSUPPORTED, nothing enqueued.  All calls on
 * one GPU share its scratch, whose counters are zero when the library is
 * loaded and are left zero by every call: calls that overlap in time on one
 * GPU (different streams, or concurrent host threads without ordering) race
 * on it and must not be issued.
 */
int gemm_bt_noalloc(const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K, int in_dtype,
                    int out_dtype, void* stream);

/* Activations of an epilogue; Phi is the normal distribution's function. */
typedef enum {
    GEMM_BT_ACT_NONE = 0,      /* z */
    GEMM_BT_ACT_RELU = 1,      /* max(z, 0) */
    GEMM_BT_ACT_GELU = 2,      /* z Phi(z) */
    GEMM_BT_ACT_GELU_TANH = 3, /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2 */
    GEMM_BT_ACT_SILU = 4       /* z / (1 + exp(-z)) */
} gemm_bt_activation;

/* What gemm_bt_epi does to the sums before they are stored; a NULL pointer
   leaves its term out. */
typedef struct {
    const float* row_scale; /* M fp32 factors, one per row of A (8-bit rows with scales) */
    const float* col_scale; /* N fp32 factors, one per row of B */
    const void* bias;       /* N elements of bias_dtype */
    const void* residual;   /* M x N elements of residual_dtype, row-major; may be C itself if its type is C's */
    void* preact;           /* M x N elements of preact_dtype, row-major: receives Z (for a backward pass) */
    int bias_dtype, residual_dtype, preact_dtype; /* GEMM_BT_F32, _F16 or _BF16, read where the pointer is not NULL */
    int activation;                               /* gemm_bt_activation */
} gemm_bt_epilogue_t;

/*
 * The product with its epilogue in the same kernel:
 *   Z[i][j] = row_scale[i] * col_scale[j] * sum_k A[i][k] B[j][k] + bias[j]
 *   C[i][j] = act(Z[i][j]) + residual[i][j]
 * The sum, Z, the activation and the residual's addition are held in fp32 and
 * rounded once into C (and once into preact).  Inputs are those of gemm_bt;
 * out_dtype is GEMM_BT_F32, _BF16 or _F16 for every input type: an int8
 * product's exact int32 sum is converted to fp32 (rounded above 2^24) before
 * its scales.  The activations use the hardware's exponential and reciprocal
 * of arguments rounded to fp32.  Their relative error, in units of 2^-24, is
 * below 8 + 1.5 |z| for silu, 24 + 1.25 z^2 for gelu and 8 + 6 |a| for
 * gelu_tanh, a = 2 sqrt(2/pi) (z + 0.044715 z^3): small next to 16-bit
 * results' rounding everywhere, and in a tail a few times what the rounding of
 * z itself costs.  Results below 2^-126 |z| may be 0.  Their derivatives (in the
 * backward passes) are within 2^-19 (1 + |z|).
 *   epilogue   NULL, or every pointer in it NULL and the activation none: C is
 *              the plain product (in floating point for int8 inputs too)
 *   workspace  as for gemm_bt_ws (NULL: no split along K), of
 *              gemm_bt_epi_workspace_size bytes.  Products of 16-bit inputs are
 *              planned as gemm_bt_ws plans them; 8-bit ones of few tiles are cut
 *              along K too (64 x 64 tiles, pieces of at least 2048 elements).
 *              For M <= 16 either run the streaming kernel where N is more than
 *              16 per compute unit, and 16-bit ones without a workspace (the
 *              faster choice where the size is 0, unless B is in the caches)
 *              for any N; else tiles
 * K == 0 is the empty sum: C = act(bias) + residual, A and B are not read.
 * bias, residual and preact need the alignment of their elements only.
 * preact must not overlap C or an input.  Types that are none of the above,
 * an unknown activation: INVALID_VALUE.  Everything else is as for gemm_bt_ws.
 */
int gemm_bt_epi(const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K, int in_dtype,
                int out_dtype, const gemm_bt_epilogue_t* epilogue, void* workspace, size_t workspace_bytes,
                void* stream);

/* The workspace gemm_bt_epi needs for these sizes and types (as
   gemm_bt_workspace_size). */
int gemm_bt_epi_workspace_size(int64_t M, int64_t N, int64_t K, int in_dtype, int out_dtype, size_t* bytes);

/*
 * Row operators around the product.  Matrices are row-major with `d` (or `n`)
 * contiguous elements per row; an input's rows start `ld` elements apart (ld
 * >= d), outputs are dense.  x, residual and h share x_dtype; a weight is of
 * x_dtype or GEMM_BT_F32 (else UNSUPPORTED).  Pointers need the alignment of
 * their elements only; every size from 0 up is served (no rows: nothing is
 * written but a gradient's zeros; up to 2^26 columns and 2^31 rows, else
 * UNSUPPORTED).  Statistics are held in fp32 and every output is rounded
 * once.  Results are the same bits on every run on the same device.  Calls
 * are asynchronous on `stream`, allocate nothing and report argument errors
 * before anything is enqueued, as the products do.
 */

/*
 * Root-mean-square norm with the residual's addition:
 *   h = x + residual        (h = x where residual is NULL)
 *   rstd = 1 / sqrt(mean(h^2) + eps)
 *   y = h * rstd * weight
 * y_dtype GEMM_BT_F32, _F16 or _BF16, or 8 bits with one scale per row, for
 * an 8-bit product: with amax the row's largest |y| and Q = 448 (_FP8_E4M3)
 * or 127 (_INT8), scale = max(amax / Q, 2^-100) and y holds y / scale rounded
 * to nearest even.  A row with an infinity or a NaN among its y gets the
 * scale NaN (its codes then hold no value).
 *   y      rows x d of y_dtype
 *   h      rows x d of x_dtype, or NULL: receives h rounded.  It may be x or
 *          residual itself where that one's rows are dense; y may not
 *   scale  rows fp32 (8-bit y; else not used)
 *   rstd   rows fp32, or NULL: receives 1 / sqrt(...) for the backward pass
 * A row of no elements (d == 0) has mean 0 and amax 0: rstd = 1 / sqrt(eps),
 * scale = 2^-100.
 *   eps    >= 0 (else INVALID_VALUE)
 */
int gemm_bt_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight, void* y,
                     void* h, float* scale, float* rstd, int64_t rows, int64_t d, float eps, int x_dtype,
                     int w_dtype, int y_dtype, void* stream);

/* The rows of x in 8 bits (q_dtype GEMM_BT_FP8_E4M3 or GEMM_BT_INT8) and their
   scales, as gemm_bt_rms_norm leaves its y. */
int gemm_bt_quantize_rows(const void* x, int64_t ldx, void* q, float* scale, int64_t rows, int64_t d, int x_dtype,
                          int q_dtype, void* stream);

/*
 * The norm's backward pass.  With xhat = h * rstd, g = dy * weight and dy the
 * gradient of y (of the values before rounding, for 8-bit y):
 *   dx = rstd * (g - xhat * mean(g * xhat)) + dh,   dweight = sum over rows of dy * xhat
 * dx is the gradient of x and of residual alike.
 *   h, rstd    as gemm_bt_rms_norm left them (x itself where there was no residual)
 *   dh         the gradient that reaches h from elsewhere, or NULL
 *   dx         rows x d of x_dtype; may be dh itself where its rows are dense,
 *              not dy or h, which dweight's sums read (INVALID_VALUE)
 *   dweight    d elements of w_dtype
 *   workspace  at least gemm_bt_rms_norm_backward_workspace bytes (0 for few
 *              rows), 4-byte aligned, any contents
 */
int gemm_bt_rms_norm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ldh, const void* weight,
                              const float* rstd, const void* dh, int64_t ld_dh, void* dx, void* dweight,
                              int64_t rows, int64_t d, int x_dtype, int w_dtype, void* workspace,
                              size_t workspace_bytes, void* stream);
int gemm_bt_rms_norm_backward_workspace(int64_t rows, int64_t d, size_t* bytes);

/*
 * Layer norm with the residual's addition:
 *   h = x + residual        (h = x where residual is NULL)
 *   mean = mean(h),  rstd = 1 / sqrt(mean((h - mean)^2) + eps)
 *   y = (h - mean) * rstd * weight + bias
 * As gemm_bt_rms_norm in everything else: types, strides, 8-bit y with one
 * scale per row, what may be what.  The squares are those of h - mean (never
 * mean(h^2) - mean^2), and the mean's own rounding is taken out of h - mean.
 * Rows whose sums or squares leave fp32's range are summed once more, scaled.
 * A row with an infinity or a NaN has y, mean and rstd NaN, and so has one whose
 * h - mean leaves fp32's range (not in 8 bits: there it is held in 64 bits, and
 * the row has its values).
 *   bias   d elements of w_dtype, or NULL
 *   mean   rows fp32, or NULL: receives mean for the backward pass
 * A row of no elements has mean 0.
 */
int gemm_bt_layer_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                       const void* bias, void* y, void* h, float* scale, float* mean, float* rstd, int64_t rows,
                       int64_t d, float eps, int x_dtype, int w_dtype, int y_dtype, void* stream);

/*
 * Layer norm's backward pass.  With xhat = (h - mean) * rstd and g = dy * weight:
 *   dx = rstd * (g - mean(g) - xhat * mean(g * xhat)) + dh
 *   dweight = sum over rows of dy * xhat,   dbias = sum over rows of dy
 * As gemm_bt_rms_norm_backward in everything else.
 *   mean, rstd  as gemm_bt_layer_norm left them.  mean is rounded to fp32, which
 *               xhat does not make up for: it shows where a row's entries differ
 *               by little more than that
 *   dbias       d elements of w_dtype, or NULL: not wanted
 *   workspace   at least gemm_bt_layer_norm_backward_workspace bytes
 */
int gemm_bt_layer_norm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ldh, const void* weight,
                                const float* mean, const float* rstd, const void* dh, int64_t ld_dh, void* dx,
                                void* dweight, void* dbias, int64_t rows, int64_t d, int x_dtype, int w_dtype,
                                void* workspace, size_t workspace_bytes, void* stream);
int gemm_bt_layer_norm_backward_workspace(int64_t rows, int64_t d, size_t* bytes);

/*
 * The backward pass of gemm_bt_epi's activation and bias:
 *   dz = dy * act'(preact),   dbias = sum over rows of dz
 * (gemm_bt_linear_backward is this with the gradients of A and B).
 *   preact  rows x n of preact_dtype as gemm_bt_epi left it (not read for GEMM_BT_ACT_NONE)
 *   dz      rows x n of dtype, or NULL; may be dy itself
 *   dbias   n elements of bias_dtype, or NULL (then no workspace is needed)
 *   workspace  at least gemm_bt_act_backward_workspace bytes, 4-byte aligned, any contents
 */
int gemm_bt_act_backward(const void* dy, const void* preact, void* dz, void* dbias, int64_t rows, int64_t n,
                         int activation, int dtype, int preact_dtype, int bias_dtype, void* workspace,
                         size_t workspace_bytes, void* stream);
int gemm_bt_act_backward_workspace(int64_t rows, int64_t n, size_t* bytes);

/*
 * The whole backward pass of C = act(X W^T + bias) for 16-bit X (M x K) and W
 * (N x K), dy the gradient of C (M x N), all of dtype GEMM_BT_F16 or _BF16:
 *   dz = dy * act'(preact), rounded into dtype (dy itself for GEMM_BT_ACT_NONE)
 *   dx = dz W,   dw = dz^T X,   dbias = sum over rows of dz before its rounding
 * Sums are held in fp32 and rounded once.  X, W and dy are read as they lie in
 * memory: nothing is transposed or copied but rows that are not whole 16-byte
 * chunks (N or K not a multiple of 8), which are padded in the workspace.  A
 * product whose sum is long and whose result is small is cut along the sum
 * into fp32 slices that are added in order, so results are the same bits on
 * every run on the same device.
 *   preact     M x N of preact_dtype, as gemm_bt_epi left it (activation NONE: not read)
 *   dx, dw, dbias  M x K, N x K and N elements of dtype; NULL: not wanted
 *   workspace  at least gemm_bt_linear_backward_workspace bytes, 16-byte
 *              aligned, any contents
 * N and K up to 2^21 - 1, dx and dw up to 2^21 tiles of 128 x 128 each.  x, w and (for GEMM_BT_ACT_NONE with N % 8 == 0) dy
 * need 16-byte alignment where K % 8 == 0 (else UNSUPPORTED); the rest needs
 * the alignment of its elements.  dx, dw and dbias must not overlap an input or
 * each other.  A gradient whose sum has no terms is zeros.
 * The gradient of an epilogue's residual is dy itself.
 */
int gemm_bt_linear_backward(const void* dy, const void* x, const void* w, const void* preact, void* dx, void* dw,
                            void* dbias, int64_t M, int64_t N, int64_t K, int activation, int dtype,
                            int preact_dtype, void* workspace, size_t workspace_bytes, void* stream);
int gemm_bt_linear_backward_workspace(int64_t M, int64_t N, int64_t K, int activation, size_t* bytes);

/*
 * The gated product of a feed-forward block, both projections and what follows
 * them in one kernel.  B has 2 N rows: the gate's N, then the other factor's.
 *   Zg[i][j] = row_scale[i] * col_scale[j] * sum_k A[i][k] B[j][k] + bias[j]
 *   Zu[i][j] = row_scale[i] * col_scale[N + j] * sum_k A[i][k] B[N + j][k] + bias[N + j]
 *   C[i][j] = act(Zg[i][j]) * Zu[i][j]
 * As gemm_bt_epi in everything else: inputs of 16 or 8 bits, float results, Z and
 * everything after it in fp32, rounded once.  8-bit floats are multiplied by the matrix
 * units' own instructions for every type of result, as gemm_bt and gemm_bt_epi do: within
 * a group of 8 consecutive k each product is cut to a multiple of 2^-13 of the largest one.
 *   C         M x N of out_dtype
 *   epilogue  col_scale and bias have 2 N elements, preact M x 2 N (receives Zg
 *             and Zu, row by row); residual must be NULL (else INVALID_VALUE)
 *   workspace as for gemm_bt_epi, of gemm_bt_gated_workspace_size bytes
 * The plan is that of gemm_bt_epi with 2 N columns, whose limits apply to 2 N.
 */
int gemm_bt_gated(const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K, int in_dtype,
                  int out_dtype, const gemm_bt_epilogue_t* epilogue, void* workspace, size_t workspace_bytes,
                  void* stream);
int gemm_bt_gated_workspace_size(int64_t M, int64_t N, int64_t K, int in_dtype, int out_dtype, size_t* bytes);

/*
 * Its backward pass for 16-bit X (M x K) and W (2 N x K), dy the gradient of C
 * (M x N):
 *   dz = [dy * Zu * act'(Zg), dy * act(Zg)] (M x 2 N), rounded into dtype
 *   dx = dz W,   dw = dz^T X (2 N x K),   dbias = sums over rows of dz (2 N) before its rounding
 * As gemm_bt_linear_backward with 2 N columns in everything else; preact (M x 2 N)
 * is read for every activation, and dy needs the alignment of its elements only.
 *   workspace  at least gemm_bt_gated_backward_workspace bytes, 16-byte aligned, any contents
 */
int gemm_bt_gated_backward(const void* dy, const void* x, const void* w, const void* preact, void* dx, void* dw,
                           void* dbias, int64_t M, int64_t N, int64_t K, int activation, int dtype,
                           int preact_dtype, void* workspace, size_t workspace_bytes, void* stream);
int gemm_bt_gated_backward_workspace(int64_t M, int64_t N, int64_t K, int activation, size_t* bytes);

/*
 * A matrix in 8 bits with one scale per block of 128 along its rows.  V is x (rows
 * x d) or, with transpose = 1, x transposed (d x rows); a block is 1 x 128 entries of
 * V (block_rows 1) or 128 x 128 (block_rows 128), the last ones of a row or column
 * shorter.  With amax a block's largest |v|, scale = max(amax / 448, 2^-100) and q
 * holds v / scale rounded to nearest even (v 448 / amax, not v over the scale as it
 * is rounded to fp32: they differ where v lies half-way between two codes); a block
 * with an infinity or a NaN gets the scale NaN (its codes then hold no value).
 *   x      as for gemm_bt_quantize_rows
 *   q      q_dtype GEMM_BT_FP8_E4M3 (else UNSUPPORTED): V row-major, dense; with
 *          transpose the rows are rows rounded up to a multiple of 16 long, the
 *          rest zeros (for a product that sums over the rows of x)
 *   scale  fp32, block by block: scale[b * R + r] belongs to block b of row r of V (of
 *          rows 128 r .. 128 r + 127 for block_rows 128), R the number of those
 */
int gemm_bt_quantize_blocks(const void* x, int64_t ldx, void* q, float* scale, int64_t rows, int64_t d,
                            int block_rows, int transpose, int x_dtype, int q_dtype, void* stream);

/*
 * The product of two such matrices, with gemm_bt_epi's epilogue:
 *   S[i][j] = sum_b sa(i, b) sb(j, b) sum_{k in block b} A[i][k] B[j][k],  b = k / 128
 *   Z[i][j] = row_scale[i] * col_scale[j] * S[i][j] + bias[j],   C[i][j] = act(Z[i][j]) + residual[i][j]
 * A (M x K) has blocks of 1 x 128, B (N x K) of 1 x 128 (b_block_rows 1: sb(j, b) is that of
 * row j) or of 128 x 128 (128: that of row j / 128).  A scale lies at
 * row * row_stride + b * block_stride floats: strides (1, R) as gemm_bt_quantize_blocks
 * leaves them (the fastest), or others (0 .. 2^20 - 1 and 0 .. 2^26 - 1, else UNSUPPORTED).
 * A block's sum and everything after it is held in fp32; before the sum over blocks
 * either sa * sb (tiles, where B has blocks of 128 x 128) or a block's sum times sa (else)
 * is rounded to fp32, so neither must leave fp32's range.  For results of 16 bits the
 * matrix units' instructions for 8-bit floats multiply, which cut each product to a
 * multiple of 2^-13 of the largest of its group of 8 consecutive k; for GEMM_BT_F32
 * the codes are widened to 16 bits (exactly) and every sum is a sum of fp32 roundings, at
 * about half the rate.
 *   in_dtype   GEMM_BT_FP8_E4M3 (else UNSUPPORTED); K % 16 == 0, A and B 16-byte
 *              aligned (else UNSUPPORTED), as for 8-bit inputs of gemm_bt
 *   out_dtype, epilogue, K == 0 as for gemm_bt_epi
 *   workspace  as for gemm_bt_ws, of gemm_bt_block_workspace_size bytes (NULL: no split along K)
 * For M <= 16 and N more than 16 per compute unit the streaming kernel; else the
 * tiles with the shortest estimate: 256 x 128 (the plan's variant 0), 128 x 128 (1),
 * 64 x 64 in steps of 128 (2) or 256 (4) along K, and for B in blocks of 128 x 128 256 x
 * 256 (3); 64 x 64 ones cut along K where they leave half the compute units idle, and
 * rows past whole waves of large tiles in a second launch (gemm_bt_plan_block).
 */
int gemm_bt_block(const void* A, const void* B, void* C, int64_t M, int64_t N, int64_t K, const float* a_scale,
                  int64_t a_row_stride, int64_t a_block_stride, const float* b_scale, int64_t b_row_stride,
                  int64_t b_block_stride, int b_block_rows, int in_dtype, int out_dtype,
                  const gemm_bt_epilogue_t* epilogue, void* workspace, size_t workspace_bytes, void* stream);
int gemm_bt_block_workspace_size(int64_t M, int64_t N, int64_t K, int b_block_rows, int out_dtype, size_t* bytes);

/* Workspace gemm_bt_ws needs for these sizes and types (0 when it runs the
   plain grid), for the current device (256 compute units without one).  At
   most 16 KiB + 256 * 64 KiB (16.02 MiB) on an MI355X, whatever the
   sizes.  Returns gemm_bt's status for invalid arguments. */
int gemm_bt_workspace_size(int64_t M, int64_t N, int64_t K, int in_dtype, int out_dtype, size_t* bytes);

/* Human-readable text for a status code (static storage; never NULL). */
const char* gemm_bt_status_string(int status);

/* Library version, major * 10000 + minor * 100 + patch. */
int gemm_bt_version(void);

/*
 * Launch plan: which kernel and tile shape gemm_bt would use for a problem;
 * lets callers and tests see the tiling and the grid.  No kernel runs.  The
 * plan is made for the current device's compute-unit count when it is a
 * gfx950 (one cached device query), else for 256 (an MI355X).  `a_align`,
 * `b_align`, `c_align` are the byte alignments of the pointers that would be
 * passed (e.g. 256 for fresh allocations).
 */
typedef struct {
    int kernel;       /* 0 = none (empty), 1 = zero fill (K == 0), 2 = LDS-tiled MFMA with register-staged
                         loads (no longer planned: kind 4 takes every row alignment), 3 = skinny streaming
                         (M <= 16), 4 = LDS-tiled MFMA with direct global->LDS loads, 5 = LDS-tiled MFMA
                         with LDS transpose reads (an operand stored K-outer) */
    int variant;      /* tile-shape variant index within the kernel family */
    int bm, bn, bk;   /* workgroup tile (rows of C, columns of C, K step) */
    int threads;      /* threads per workgroup */
    int vec;          /* elements per global load: 16 (16 bytes of 8-bit data), 8 (16 bytes), 2 or 1 */
    int group_m;      /* tile-rows per group in the grouped tile order */
    int ksplit;       /* waves that split K inside a workgroup (skinny kernel) */
    int stages;       /* LDS pipeline depth: A+B stages (tiled kernels), or for the 256x256 tile the 5 slots of
                         its ring of single-operand tiles */
    int lds_bytes;    /* LDS per workgroup */
    int64_t tiles_m, tiles_n;
    int64_t grid;     /* workgroups per batch item (grid * batch are launched); for a split plan the
                         workgroups of the one launch (split_tiles * pieces per tile) */
    int64_t batch;    /* batch items (1 for gemm_bt) */
    int64_t split_tiles;     /* split plan: tiles whose K range is split over several workgroups (0: one
                                workgroup per tile) */
    int64_t workspace_bytes; /* workspace the plan needs (0 unless a launch of it splits tiles along K) */
    int64_t split_rows;      /* > 0: the product runs as two launches in stream order, rows [0, split_rows)
                                of C first, planned as the fields above describe (one wave of 256 x 256
                                tiles), then the remaining rows on their own plan; 0: one launch */
    int64_t split_items;     /* > 0: stacked items run as two launches in stream order, items
                                [0, split_items) first, planned as the fields above describe (one wave of
                                256 x 256 tiles), then the remaining items on their own plan; 0: one launch */
} gemm_bt_plan_t;

int gemm_bt_plan(int64_t M, int64_t N, int64_t K, int in_dtype, int out_dtype, int a_align,
                 int b_align, int c_align, gemm_bt_plan_t* plan);

/* The plan of gemm_bt_ws given a large enough workspace (the plan gemm_bt_ws
   runs when its workspace is not NULL). */
int gemm_bt_plan_ws(int64_t M, int64_t N, int64_t K, int in_dtype, int out_dtype, int a_align,
                    int b_align, int c_align, gemm_bt_plan_t* plan);

/* The plan of gemm_bt_epi given a workspace (not NULL, also where its size is 0)
   that is large enough. */
int gemm_bt_plan_epi(int64_t M, int64_t N, int64_t K, int in_dtype, int out_dtype, int a_align, int b_align,
                     int c_align, gemm_bt_plan_t* plan);

/* The plan of gemm_bt_block given a workspace that is large enough. */
int gemm_bt_plan_block(int64_t M, int64_t N, int64_t K, int b_block_rows, int out_dtype, int a_align, int b_align,
                       gemm_bt_plan_t* plan);

/* The plan of gemm_bt_layout (for kernel 5 the variant is 0: A K-outer, 1: B
   K-outer, 2: both, on 128 x 128 tiles; 3, 4, 5 the same on 256 x 256 tiles). */
int gemm_bt_plan_layout(int64_t M, int64_t N, int64_t K, int a_layout, int b_layout, int in_dtype, int out_dtype,
                        int a_align, int b_align, int c_align, gemm_bt_plan_t* plan);

/* The plan of gemm_bt_batched_layout. */
int gemm_bt_plan_batched_layout(int64_t batch, int64_t M, int64_t N, int64_t K, int a_layout, int b_layout,
                                int in_dtype, int out_dtype, int a_align, int b_align, int c_align,
                                gemm_bt_plan_t* plan);

/* The plan of gemm_bt_batched: the tile tier counts the workgroups of all
   items; the alignments are those of every item's pointers. */
int gemm_bt_plan_batched(int64_t batch, int64_t M, int64_t N, int64_t K, int in_dtype, int out_dtype,
                         int a_align, int b_align, int c_align, gemm_bt_plan_t* plan);

/*
 * Tile order used by the tiled kernel: workgroup `pid` (0 <= pid < tiles_m *
 * tiles_n) computes output tile (tm, tn).  Workgroups are first regrouped by
 * the XCD (accelerator die, 8 on MI355X, each with its own L2) that the
 * hardware dispatches them to, round-robin, so that each die receives a
 * contiguous run of tiles; that run is then walked in bands of `group_m`
 * tile-rows, column by column inside a band, so that tiles running at the
 * same time share A-row and B-row panels in L2 ("Writing Mosaic GPU kernels
 * with Pallas", section "Using the L2 cache": reorder the grid into bands of
 * mt rows so that concurrently scheduled blocks touch less data).  A batched
 * call stacks its items along the tile rows (tiles_m = batch * tile rows per
 * item), so each die receives whole items and their panels stay in its L2.
 * Host-callable copy of the device function; returns INVALID_VALUE for a pid
 * outside the grid.
 */
int gemm_bt_tile_coord(int64_t pid, int64_t tiles_m, int64_t tiles_n, int group_m, int64_t* tm,
                       int64_t* tn);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_BT_H */
