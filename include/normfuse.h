/*
 * normfuse: the fused normalization block on one GPU (sm_103a).
 *
 * Forward: bias + residual add, then LayerNorm or RMSNorm over the hidden
 * dimension, with an optional amax of |y| for FP8 scaling, in one pass over
 * HBM. Backward: the per-row dx reduction over the hidden dimension and the
 * dgamma/dbeta reductions over the rows in one persistent kernel, followed by
 * a small deterministic finalize.
 *
 * Conventions shared by every entry point:
 *  - Matrices are row-major and contiguous, [rows, hidden]. gamma, beta and
 *    bias are [hidden] in the I/O dtype. mean and rstd are fp32 [rows].
 *    dgamma and dbeta are fp32 [hidden]. amax is one fp32 scalar.
 *  - Every tensor pointer is a DEVICE pointer on the current device, owned by
 *    the caller; the library never allocates, frees or keeps one. Pointers
 *    must be aligned to their element size. When every matrix/vector pointer
 *    is 16-byte aligned and hidden * sizeof(dtype) is a multiple of 16, the
 *    128-bit vectorised kernels run; otherwise a scalar kernel handles the
 *    call with the same results.
 *  - Outputs must not overlap inputs or each other (ln_softmax_fwd alone
 *    also runs in place).
 *  - Work is enqueued on `stream` (0 = the legacy default stream) and the call
 *    returns without waiting for it. The library calls no allocating CUDA API,
 *    and none that synchronises except ln_device_error().
 *  - Failure: arguments are validated on the host first; a validation failure
 *    returns its status before anything is enqueued and leaves every output
 *    untouched. A CUDA error from an enqueue returns LN_ERR_CUDA; the CUDA
 *    error code is then available from ln_last_cuda_error() on the calling
 *    thread. No entry point aborts, throws or prints.
 *  - Limits: rows >= 0; 1 <= hidden <= LN_MAX_HIDDEN_VEC16 (bf16/fp16) or
 *    LN_MAX_HIDDEN_VEC32 (fp32) on the vectorised path, and
 *    1 <= hidden <= LN_MAX_HIDDEN_SCALAR on the scalar path. Element
 *    offsets are 64-bit: rows * hidden may exceed 2^31 (tensors past 4 GiB).
 *
 * Citations are to the four pages the method comes from: NVIDIA/cutlass
 * discussion 874 (GEMM -> residual add -> LayerNorm), iree-org/iree issue
 * 9139 (LayerNorm as mean, variance and normalize over one read of the input),
 * NVIDIA/Fuser issue 1660 (bias + residual -> LayerNorm -> FP8 amax, with the
 * amax split into a fused partial and a final reduction) and pytorch/pytorch
 * PR 165370 (mixed-order fusion of the norm-backward reductions).
 */
#ifndef NORMFUSE_H
#define NORMFUSE_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LN_MAX_HIDDEN_VEC16 16384
#define LN_MAX_HIDDEN_VEC32 8192
#define LN_MAX_HIDDEN_SCALAR 8192

/* Size of the static device scratch array behind ln_bwd_noalloc (16 MiB). */
#define LN_NOALLOC_SCRATCH_BYTES (16u << 20)

typedef enum { LN_F32 = 0, LN_BF16 = 1, LN_F16 = 2 } ln_dtype;
typedef enum { LN_LAYERNORM = 0, LN_RMSNORM = 1 } ln_mode;
typedef enum {
  LN_OK = 0,
  LN_ERR_NULL = 1,        /* a required pointer is NULL */
  LN_ERR_ALIGN = 2,       /* a pointer is not aligned to its element size */
  LN_ERR_SHAPE = 3,       /* rows < 0, hidden out of range */
  LN_ERR_UNSUPPORTED = 4, /* unknown dtype or mode */
  LN_ERR_CUDA = 5,        /* a CUDA call failed; see ln_last_cuda_error() */
  LN_ERR_WORKSPACE = 6,   /* backward workspace missing, misaligned or too small */
  LN_ERR_INVALID = 7,     /* eps negative or not finite; outputs overlap inputs */
  LN_ERR_SCRATCH_LIMIT = 8 /* ln_bwd_noalloc: the shape needs more scratch than
                              LN_NOALLOC_SCRATCH_BYTES */
} ln_status;

/*
 * ln_fwd: out_sum = (x + bias) + residual; y = norm(out_sum) * w + beta;
 * amax = max |y|.
 *
 * Defined by the forward snippet of NVIDIA/Fuser issue 1660 (bias and
 * residual add, w = gamma or 1 + gamma, layer_norm, amax of |y| written into
 * a preallocated scalar) and by iree-org/iree issue 9139 (mean, variance and
 * normalize over a single read of the input; bias and skip operands optional).
 * RMSNorm, named on pytorch/pytorch PR 165370, is y = s * rstd * w with
 * rstd = 1/sqrt(mean(s^2) + eps).
 *
 * Per row, in fp32 arithmetic:
 *   s      = (x + bias) + residual, stored to out_sum rounded to dtype;
 *   the statistics are taken from the stored (rounded) sum:
 *   LayerNorm: mean = sum(s)/H, var = sum((s - mean)^2)/H (biased),
 *              rstd = 1/sqrt(var + eps), y = (s - mean) * rstd * w + beta;
 *   RMSNorm:   rstd = 1/sqrt(sum(s^2)/H + eps), y = s * rstd * w;
 *   w = gamma, or 1 + gamma (formed in fp32) when zero_centered_gamma != 0;
 *   y is rounded to dtype; amax = max over all stored y of |y| (exact).
 *
 * x         [rows, hidden] dtype, required.
 * bias      [hidden] dtype, NULL = no bias.
 * residual  [rows, hidden] dtype, NULL = no residual.
 * gamma     [hidden] dtype, required.
 * beta      [hidden] dtype, NULL = 0; ignored for RMSNorm.
 * eps       >= 0 and finite.
 * out_sum   [rows, hidden] dtype, NULL = not stored (the backward needs it
 *           whenever bias or residual is given).
 * y         [rows, hidden] dtype, required.
 * mean      [rows] fp32, NULL = not stored; ignored for RMSNorm.
 * rstd      [rows] fp32, NULL = not stored.
 * amax      one fp32, NULL = not computed. When given it is overwritten
 *           (set to 0 on `stream`, then maxed into), not accumulated.
 */
ln_status ln_fwd(const void* x, const void* bias, const void* residual,
                 const void* gamma, const void* beta, float eps, ln_mode mode,
                 int zero_centered_gamma, void* out_sum, void* y, float* mean,
                 float* rstd, float* amax, cudaStream_t stream, int64_t rows,
                 int64_t hidden, ln_dtype dtype);

/*
 * ln_fwd_ex: ln_fwd plus an FP8 (E4M3) copy of y.
 *
 * NVIDIA/Fuser issue 1660 computes the amax of |y| to scale y for an FP8
 * cast; the pages stop at the amax. This entry point also writes that cast,
 * with a per-tensor scale the caller provides (delayed scaling: typically
 * 448 / an amax from an earlier step). Per element:
 *   y_fp8 = E4M3(round_fp32(y_stored * scale)), round to nearest even,
 *   finite values beyond +-448 saturate to +-448 (no infinities in E4M3);
 * y_stored is y rounded to dtype (what y holds), so y_fp8 is the FP8 cast of
 * the stored y. amax is that of y_stored, as in ln_fwd.
 *
 * y_fp8      [rows, hidden] bytes (E4M3 codes), NULL = not written.
 * fp8_scale  one fp32 on the device, required when y_fp8 is given.
 * y          may be NULL when y_fp8 is given (only the FP8 copy is written).
 * Every other argument and the errors are those of ln_fwd; y_fp8 counts as a
 * tensor pointer for the 16-byte alignment of the vectorised path.
 */
ln_status ln_fwd_ex(const void* x, const void* bias, const void* residual,
                    const void* gamma, const void* beta, float eps, ln_mode mode,
                    int zero_centered_gamma, void* out_sum, void* y, float* mean,
                    float* rstd, float* amax, void* y_fp8, const float* fp8_scale,
                    cudaStream_t stream, int64_t rows, int64_t hidden,
                    ln_dtype dtype);

/* Form of the per-tile partial statistics ln_fwd_from_partials reads. */
typedef enum {
  LN_PARTIALS_SUM_SQ = 0, /* psum = sum of the tile's values, psq = sum of their squares */
  LN_PARTIALS_SUM_M2 = 1  /* psum as above, psq = sum of squares about the tile's own mean */
} ln_partials;

/*
 * ln_fwd_from_partials: y = norm(x) * w + beta with the row statistics
 * combined from per-column-tile partial sums instead of a pass over the row.
 *
 * Defined by NVIDIA/cutlass discussion 874 (the reply pointing at example
 * 37, gemm_with_layernorm.h): the GEMM that produces the row (with the
 * residual added in its epilogue) also sums each row over the column tile
 * every threadblock owns, and the LayerNorm that follows combines those
 * partials into the row's mean and variance. This is the
 * consumer, one read of x and one write of y; mx_product below is a producer of
 * such partials (of quantised operands), any other GEMM may be.
 *
 * Column tiles are tile_cols wide from column 0; the last one holds the
 * hidden - (n_tiles - 1) * tile_cols columns left, n_tiles =
 * ceil(hidden / tile_cols). With S and Q the per-row sums over the tiles of
 * psum and of the second quantity, and n_t a tile's width, in fp32:
 *   LN_PARTIALS_SUM_SQ: LayerNorm mean = S / H, var = max(Q / H - mean^2, 0)
 *     (Q = sum psq); RMSNorm mean square = Q / H.
 *   LN_PARTIALS_SUM_M2: LayerNorm var = (sum_t psq_t +
 *     sum_t (psum_t - n_t mean)^2 / n_t) / H (the parallel-variance
 *     identity); RMSNorm mean square = sum_t (psq_t + psum_t^2 / n_t) / H.
 *   rstd = 1/sqrt(var or mean square + eps); y = (x - mean) * rstd * w + beta
 *   (RMSNorm: x * rstd * w), w = gamma or 1 + gamma; y rounded to dtype;
 *   amax = max |y| over the stored y, as in ln_fwd.
 * The sum-of-squares form loses precision when |mean| is large against the
 * row's spread (Q / H and mean^2 cancel); the M2 form does not.
 *
 * x          [rows, hidden] dtype, the stored row (what the producer wrote),
 *            required when rows > 0.
 * psum, psq  [rows, n_tiles] fp32, row-major, 4-byte aligned, required when
 *            rows > 0.
 * n_tiles    must equal ceil(hidden / tile_cols), else LN_ERR_SHAPE.
 * tile_cols  >= 1 (a value >= hidden means one tile).
 * kind       LN_PARTIALS_SUM_SQ or LN_PARTIALS_SUM_M2, else LN_ERR_UNSUPPORTED.
 * gamma, beta, eps, mode, zero_centered_gamma, y, mean, rstd, amax: as in
 *            ln_fwd (mean, rstd are the statistics used, rounded to fp32).
 * Shapes, alignment, limits, streams and errors: the header's conventions.
 */
ln_status ln_fwd_from_partials(const void* x, const float* psum, const float* psq,
                               int64_t n_tiles, int64_t tile_cols, ln_partials kind,
                               const void* gamma, const void* beta, float eps,
                               ln_mode mode, int zero_centered_gamma, void* y,
                               float* mean, float* rstd, float* amax,
                               cudaStream_t stream, int64_t rows, int64_t hidden,
                               ln_dtype dtype);

/*
 * ln_bwd: dx, dgamma, dbeta of the normalization given dy and the forward's
 * saved sum and statistics.
 *
 * Defined by pytorch/pytorch PR 165370: the dx reduction runs over the hidden
 * dimension, the dgamma/dbeta reductions over the rows, and both share dy,
 * x_sum and the statistics, so one persistent kernel loads each input once,
 * keeps per-CTA partial sums of the row reduction (the PR's partial
 * accumulation) and a finalize adds the partials. Per row, in fp32:
 *   xhat = (x_sum - mean) * rstd   (RMSNorm: x_sum * rstd);  g = dy * w;
 *   c1 = sum(g)/H (LayerNorm only); c2 = sum(g * xhat)/H;
 *   dx = rstd * (g - c1 - xhat * c2)   (RMSNorm: no c1), rounded to dtype;
 *   dgamma = sum over rows of dy * xhat; dbeta = sum over rows of dy.
 * dx is also the gradient of the residual and of x through the identity add.
 * dgamma and dbeta are bitwise reproducible from run to run on the same GPU
 * model: the row-to-CTA assignment depends only on the SM count and the
 * finalize adds the partials in a fixed order (compensated fp32 sums, exact
 * up to the rounding of the compensation term, rounded once at the end).
 *
 * dy, x_sum [rows, hidden] dtype, required (x_sum is the forward's out_sum,
 *           or x itself when the forward had neither bias nor residual).
 * gamma     [hidden] dtype, required; w = gamma or 1 + gamma as in ln_fwd.
 * mean      [rows] fp32, required for LayerNorm, ignored for RMSNorm.
 * rstd      [rows] fp32, required.
 * dx        [rows, hidden] dtype, required.
 * dgamma    [hidden] fp32, required, overwritten.
 * dbeta     [hidden] fp32, NULL = not computed; ignored for RMSNorm.
 * workspace device scratch of at least ln_bwd_workspace_bytes() bytes,
 *           16-byte aligned, owned by the caller; may be NULL only when
 *           rows == 0. Its contents need no initialisation and are not
 *           meaningful after the call. Calls that share one workspace must
 *           not run concurrently.
 */
ln_status ln_bwd(const void* dy, const void* x_sum, const void* gamma,
                 const float* mean, const float* rstd, void* dx, float* dgamma,
                 float* dbeta, cudaStream_t stream, int64_t rows,
                 int64_t hidden, ln_dtype dtype, ln_mode mode,
                 int zero_centered_gamma, void* workspace,
                 size_t workspace_bytes);

/*
 * ln_bwd_ex: ln_bwd plus the gradient of the forward's bias, and a choice
 * of precision for the parameter gradients.
 *
 * The forward adds `bias` to every row before the norm (NVIDIA/Fuser issue
 * 1660), so dbias = sum over rows of dx, the gradient of the norm's input;
 * the gradients of x and of residual are dx itself (identity add). dbias is
 * a third column reduction over the rows, accumulated in the same persistent
 * kernel from the fp32 dx (before its rounding to dtype) and added up by the
 * same fixed-order finalize (pytorch/pytorch PR 165370's partial
 * accumulation of the outer reductions).
 *
 * dbias     [hidden] grad_dtype, NULL = not computed.
 * grad_dtype  the type of dgamma, dbeta and dbias: LN_F32 (as in ln_bwd), or
 *           LN_BF16 / LN_F16 for the low-precision epilogue PR 165370 names
 *           (a down cast after the outer reduction): the fixed-order
 *           compensated total of each column is rounded once, to nearest
 *           even, to that type. dgamma/dbeta/dbias must then be aligned to its size.
 * With dbias NULL and grad_dtype LN_F32 this is ln_bwd. Every other
 * argument, the workspace rule and the errors are those of ln_bwd;
 * ln_bwd_workspace_bytes() covers both entry points.
 */
ln_status ln_bwd_ex(const void* dy, const void* x_sum, const void* gamma,
                    const float* mean, const float* rstd, void* dx,
                    void* dgamma, void* dbeta, void* dbias,
                    cudaStream_t stream, int64_t rows, int64_t hidden,
                    ln_dtype dtype, ln_mode mode, int zero_centered_gamma,
                    void* workspace, size_t workspace_bytes,
                    ln_dtype grad_dtype);

/*
 * Bytes of workspace ln_bwd / ln_bwd_ex need for this shape on the current
 * device (the maximum over the vectorised and the scalar kernel and over
 * the layouts with and without dbias, so it holds whatever the pointers'
 * alignment). Queries device attributes; returns LN_ERR_CUDA when no device
 * is usable.
 */
ln_status ln_bwd_workspace_bytes(int64_t rows, int64_t hidden, ln_dtype dtype,
                                 ln_mode mode, size_t* bytes);

/*
 * ln_bwd_noalloc: ln_bwd for callers that cannot allocate device memory.
 *
 * The pages have no counterpart to this entry point; it exists for callers
 * that must not call cudaMalloc or any allocator around a backward pass: a
 * framework that owns every device allocation through its own caching pool
 * (a raw cudaMalloc behind its back fragments the pool and escapes its
 * accounting), a runtime whose device memory budget is fixed up front, and a
 * hot path where an allocation is not allowed because cudaMalloc may
 * synchronise the device. It computes exactly what ln_bwd
 * computes, with the same kernels, arguments and results; the difference is
 * that the per-CTA dgamma/dbeta partials go to a static device array of
 * LN_NOALLOC_SCRATCH_BYTES inside the library instead of a caller workspace.
 *
 * - The array belongs to the library's device code: a context holds its
 *   bytes from the moment the library's module is loaded in it until the
 *   context is destroyed. Under lazy module loading (the CUDA default) that
 *   is the first call of this entry point in the context, so that first call
 *   commits the array; make it before any stream capture and before any
 *   phase with a fixed memory budget. Later calls allocate and free nothing.
 * - Set-up: every call looks up the array's device address in the current
 *   context (the caller's device current), a host-side query that enqueues
 *   nothing; an address is never reused across contexts, so a
 *   cudaDeviceReset or a context of the caller's own is handled.
 * - Limit: shapes whose partials need more than LN_NOALLOC_SCRATCH_BYTES
 *   return LN_ERR_SCRATCH_LIMIT before anything is enqueued
 *   (ln_bwd_workspace_bytes() gives a bound of the need: it also covers
 *   ln_bwd_ex's dbias columns, which this entry point does not compute).
 *   The backward keeps one to three partial rows per SM for 16-byte
 *   aligned rows (one for rows wider than 4096 16-bit elements), so on a
 *   152-SM GB300 aligned LayerNorm rows fit up to about 13,700 elements
 *   and RMSNorm rows up to the 16,384 maximum.
 * - Every call on a device shares the one array and nothing in it needs to
 *   start at zero (each call overwrites the partials it reads). Calls whose
 *   execution overlaps on the GPU (different streams, or different host
 *   threads) race on the array; serialise them, e.g. on one stream.
 * - Other arguments, errors and results: as ln_bwd.
 */
ln_status ln_bwd_noalloc(const void* dy, const void* x_sum, const void* gamma,
                         const float* mean, const float* rstd, void* dx,
                         float* dgamma, float* dbeta, cudaStream_t stream,
                         int64_t rows, int64_t hidden, ln_dtype dtype,
                         ln_mode mode, int zero_centered_gamma);

/*
 * ln_softmax_fwd: row softmax, y[r, :] = exp(x[r, :] - m_r) / s_r with
 * m_r = max_j x[r, j] and s_r = sum_j exp(x[r, j] - m_r).
 *
 * Defined by iree-org/iree issue 9139 (the softmax IR: a max reduction, the
 * exponential of the shifted row, a sum reduction and a division, fused into
 * one dispatch). The ln_ prefix is the library's; this call has nothing to do
 * with a normalization's parameters. Each row is read from HBM once and
 * written once; the max, exponentials, sum and reciprocal are fp32, and y is
 * rounded to dtype. A row that is all -inf, or holds a NaN or +inf, gives NaN
 * in every column, as the definition does; -inf entries of an otherwise
 * finite row give exactly 0 (masking).
 *
 * x, y  [rows, hidden] dtype, device, required when rows > 0. y == x (in
 *       place) is allowed; any other overlap returns LN_ERR_INVALID.
 * Shapes, alignment, limits, streams and errors are those of the header's
 * conventions (no statistics or parameters are involved).
 */
ln_status ln_softmax_fwd(const void* x, void* y, cudaStream_t stream, int64_t rows,
                         int64_t hidden, ln_dtype dtype);

/*
 * Group norm with an activation, channels last.
 *
 * The pages behind the entry points above stop at LayerNorm and RMSNorm; in
 * the diffusion networks they name (NVIDIA/cutlass discussion 874), the
 * residual blocks have a group norm and an activation where the transformer
 * blocks have a LayerNorm. Group norm: Wu and He, 2018.
 *
 * Activations are [samples, rows, channels], channels contiguous: rows are
 * the pixels (or points) of a sample. Their strides are given in elements:
 * *_sample from one sample to the next, *_row from one row to the next, so
 * that a tensor may be a slice of the channels of a wider one. Group g has
 * the channels [g, g + 1) * channels / groups, M = rows * channels / groups
 * values in a sample. gamma and beta are [channels] (param_sample = 0), or
 * one row of [channels] for each sample, param_sample elements apart.
 *
 * Everything else is as above: device pointers owned by the caller, one
 * dtype for x, gamma, beta, y, dy and dx, fp32 arithmetic, work enqueued on
 * `stream`, a status for an answer, nothing touched on a refusal. Rows are
 * read and written 16, 8, 4 or 2 bytes at a time, by what all the call's rows
 * are aligned to (base, strides, channels * sizeof(dtype)). The results depend
 * on the arguments, that alignment, the number of SMs and the largest
 * thread-block cluster that the device places only.
 */
#define GN_MAX_CHANNELS 65536

typedef enum { GN_ACT_NONE = 0, GN_ACT_SILU = 1, GN_ACT_GELU = 2 } gn_act;

/*
 * gn_fwd: y = act((x - mean) * rstd * w + beta), with mean and the biased
 * variance of each sample's groups, rstd = 1/sqrt(var + eps), w = gamma or
 * 1 + gamma; act: none, z / (1 + e^-z), or z * Phi(z) (the exact GELU).
 *
 * x          [samples, rows, channels], required. rows up to 2^40, samples
 *            below 2^31; LN_ERR_SHAPE too where samples times the column
 *            tiles (64 bytes of channels and more) or times the slices of
 *            the rows reach 2^31, which no y below 128 GiB does.
 * gamma      NULL = 1; beta NULL = 0.
 * eps        >= 0 and finite.
 * y          as x, required; overlaps no input and not itself.
 * mean, rstd [samples, groups] fp32, NULL = not stored; the backward reads
 *            them. rows = 0 stores zeros.
 * groups     divides channels, else LN_ERR_SHAPE.
 * workspace  gn_workspace_bytes(..., backward = 0), which may be 0 (NULL is
 *            fine then), 16-byte aligned, owned by the caller, not
 *            initialised; calls that may run at the same time need one each.
 */
ln_status gn_fwd(const void* x, int64_t x_sample, int64_t x_row, const void* gamma,
                 const void* beta, int64_t param_sample, float eps, gn_act act,
                 int zero_centered_gamma, void* y, int64_t y_sample, int64_t y_row,
                 float* mean, float* rstd, cudaStream_t stream, int64_t samples,
                 int64_t rows, int64_t channels, int64_t groups, ln_dtype dtype,
                 void* workspace, size_t workspace_bytes);

/*
 * gn_bwd: the gradients of gn_fwd from dy, its x and its statistics. With
 * z as in gn_fwd, recomputed, dz = dy * act'(z) and sums in fp32:
 *   A[n, c] = sum over rows of dz, B[n, c] = sum over rows of dz * xhat;
 *   c1 = sum over the group of w A / M, c2 = sum over the group of w B / M;
 *   dx = rstd * (w dz - c1 - xhat * c2), rounded to dtype;
 *   dgamma = sum over samples of B, dbeta = sum over samples of A, or B and A
 *   themselves where gamma and beta are per sample.
 * dgamma and dbeta are added up in a fixed order (compensated sums over the
 * slices of the rows and the samples), rounded once to grad_dtype.
 *
 * dy, x      as in gn_fwd, each with its strides.
 * mean, rstd what gn_fwd stored.
 * dx         required; overlaps no input and not itself.
 * dgamma, dbeta  [channels], or [samples, channels] (contiguous) when
 *            param_sample is not 0 (65535 samples at most then); grad_dtype;
 *            NULL = not computed.
 * workspace  gn_workspace_bytes(..., backward = 1), as above.
 */
ln_status gn_bwd(const void* dy, int64_t dy_sample, int64_t dy_row, const void* x,
                 int64_t x_sample, int64_t x_row, const void* gamma, const void* beta,
                 int64_t param_sample, gn_act act, int zero_centered_gamma,
                 const float* mean, const float* rstd, void* dx, int64_t dx_sample,
                 int64_t dx_row, void* dgamma, void* dbeta, cudaStream_t stream,
                 int64_t samples, int64_t rows, int64_t channels, int64_t groups,
                 ln_dtype dtype, ln_dtype grad_dtype, void* workspace,
                 size_t workspace_bytes);

/* Bytes of workspace gn_fwd (backward = 0) or gn_bwd (backward != 0) need
 * for this shape on the current device, whatever the alignment. */
ln_status gn_workspace_bytes(int64_t samples, int64_t rows, int64_t channels, int64_t groups,
                             ln_dtype dtype, int backward, size_t* bytes);

/*
 * Rotary positions (Su et al., 2021) of a transformer's queries and keys,
 * with the RMSNorm of each head in front where a gamma is given.
 *
 * A tensor is [batch, tokens, heads, head_dim], head_dim contiguous, with
 * strides in elements for batch, token and head: slices of a packed
 * projection, [batch, heads, tokens, head_dim] in memory and expanded inputs
 * are all given that way. The first `rot` elements of a head form rot / 2
 * pairs: (j, j + rot / 2) for ROPE_HALF, (2j, 2j + 1) for ROPE_INTERLEAVED;
 * the elements after them pass through. Per head, in fp32:
 *   u = x * rstd * w, rstd = 1/sqrt(sum x^2 / head_dim + eps), w = gamma or
 *   1 + gamma (without a gamma u = x);
 *   t = sum over the axes of position * frequency, of the pair;
 *   y0 = scale * (u0 cos t - u1 sin t), y1 = scale * (u1 cos t + u0 sin t);
 * y is rounded once, to dtype. Angles are exact modulo one turn (the
 * frequency as a 64-bit fraction of a turn times the integer position), so
 * positions of any size, negative ones too, lose nothing to fp32. A frequency
 * that is infinite or NaN makes its pair's results NaN, at position 0 too.
 *
 * An output may be its own input (same pointer and strides); apart from that
 * outputs overlap neither inputs nor each other nor themselves. Interleaved
 * slices (queries and keys of one buffer) do not count as overlapping.
 */
#define ROPE_MAX_HEADS 65536

typedef enum { ROPE_HALF = 0, ROPE_INTERLEAVED = 1 } rope_layout;

typedef struct {
  const void* pos;      /* int32 or int64 positions, device */
  int bits;             /* 32 or 64 */
  int64_t axes;         /* 1..4 position axes (an image's tokens have 2) */
  int64_t stride[3];    /* of axis, batch and token, in elements; 0 = shared */
  const double* freqs;  /* [axes, rot / 2] radians a position, device */
  int64_t rot;          /* even, 2..head_dim */
  rope_layout layout;
  float scale;          /* of cos and sin; 1, or a long-context factor */
} rope_positions;

typedef struct {
  const void* x;        /* input */
  void* y;              /* output */
  const void* gamma;    /* [head_dim], NULL = no norm */
  int64_t heads;
  int64_t x_stride[3];  /* of batch, token and head */
  int64_t y_stride[3];
} rope_heads;

typedef struct {
  const void* dy;       /* gradient of y */
  const void* x;        /* the forward's input; needed with gamma only */
  void* dx;
  const void* gamma;    /* [head_dim], NULL = no norm */
  void* dgamma;         /* [head_dim] grad_dtype, NULL = not computed */
  int64_t heads;
  int64_t dy_stride[3];
  int64_t x_stride[3];
  int64_t dx_stride[3];
} rope_heads_grad;

/*
 * rope_fwd: both tensors in one launch; k may be NULL, and either may have 0
 * heads. head_dim even, 2..512; any batch and number of tokens.
 */
ln_status rope_fwd(const rope_heads* q, const rope_heads* k, const rope_positions* positions,
                   float eps, int zero_centered_gamma, cudaStream_t stream, int64_t batch,
                   int64_t tokens, int64_t head_dim, ln_dtype dtype);

/*
 * rope_bwd: with g' the transposed rotation of dy, xhat = x * rstd and
 * g = g' * w: dgamma = sum over tokens and heads of g' * xhat,
 * dx = rstd * (g - xhat * sum(g * xhat) / head_dim); without a gamma dx = g'.
 * The statistics are taken anew from x. dgamma is added up in a fixed order
 * and rounded once to grad_dtype.
 *
 * workspace  rope_bwd_workspace_bytes() bytes, 16-byte aligned, when a dgamma
 *            is given (else NULL is fine); not initialised; calls that may
 *            run at the same time need one each.
 */
ln_status rope_bwd(const rope_heads_grad* q, const rope_heads_grad* k,
                   const rope_positions* positions, float eps, int zero_centered_gamma,
                   cudaStream_t stream, int64_t batch, int64_t tokens, int64_t head_dim,
                   ln_dtype dtype, ln_dtype grad_dtype, void* workspace,
                   size_t workspace_bytes);

ln_status rope_bwd_workspace_bytes(int64_t head_dim, size_t* bytes);

/*
 * rope_frequencies: the rot / 2 frequencies base^(-2j / rot), in radians a
 * position, into a HOST array, scaled for contexts `factor` times as long as
 * the `original` one a model was trained with, and the scale of cos and sin
 * that goes with them. No device is needed.
 *   ROPE_SCALING_NONE    as they are, scale 1 (factor and original ignored).
 *   ROPE_SCALING_LINEAR  divided by factor (positions interpolated), scale 1.
 *   ROPE_SCALING_NTK     base * factor^(rot / (rot - 2)) for base: the slowest
 *                        pair is divided by factor, the fastest stays. Scale 1.
 *                        rot = 2 has one pair, which stays.
 *   ROPE_SCALING_YARN    (Peng et al., 2023) pairs that make more than
 *                        turns_fast turns in the original context stay, those
 *                        that make fewer than turns_slow are divided by
 *                        factor, a linear ramp over the pairs between;
 *                        scale 0.1 ln(factor) + 1.
 * base > 1, factor >= 1, original >= 1, turns_fast >= turns_slow > 0 where the
 * scaling uses them, else LN_ERR_INVALID; rot even and >= 2, else LN_ERR_SHAPE.
 */
typedef enum {
  ROPE_SCALING_NONE = 0,
  ROPE_SCALING_LINEAR = 1,
  ROPE_SCALING_NTK = 2,
  ROPE_SCALING_YARN = 3
} rope_scaling;

ln_status rope_frequencies(int64_t rot, double base, rope_scaling scaling, double factor,
                           int64_t original, double turns_fast, double turns_slow,
                           double* freqs, float* scale);

/*
 * Matrices in 8 and 4 bits with scales, the norms that end in them and the
 * product that starts from them.
 *
 * ln_fwd_ex casts y with one scale that the caller has from an earlier step.
 * Here the scales are found in the same pass, for a row or a block of columns:
 *   MX_FP8_ROW   E4M3 codes, one fp32 scale a row
 *   MX_FP8_BLOCK E4M3 codes, one fp32 scale for 128 columns of a row
 *   MX_MXFP8     E4M3 codes, one E8M0 scale (2^(byte - 127)) for 32 columns
 *   MX_MXFP4     E2M1 codes, one E8M0 scale for 32 columns
 *   MX_NVFP4     E2M1 codes, one E4M3 scale for 16 columns, of the values times
 *                *mul
 * The formats of the last three are those of the OCP microscaling
 * specification (2023) and NVIDIA's NVFP4. With amax the largest |v| of a row or
 * block, all in fp32, round to nearest even:
 *   fp32 scale   a = max(amax, 2^-100), scale = a / 448, code = E4M3(v * (448 / a))
 *   E8M0         scale = the least 2^e, e >= -127, with amax <= M 2^e (M = 448 or
 *                6), code = E4M3 or E2M1(v / 2^e)
 *   E4M3         u = v * *mul, scale = E4M3(amax(u) / 6), at most 448,
 *                code = E2M1(u / scale), at most 6; 0 where the scale is 0
 * so a value is code * scale (MX_NVFP4: / *mul). A row or block that holds an
 * infinity or a NaN has a NaN for its scale and codes of 0. The blocks begin at
 * column 0; the last one of a row may be narrower. Here E8M0 scales round up: the
 * OCP document's own conversion takes the exponent of amax less that of M, and the
 * values of a block that are past M 2^e then become M 2^e. Either reads the other's
 * matrices. MX_NVFP4's *mul is the caller's to find, an amax of this step or of one
 * before. The product below takes the microscaled formats; the two with fp32 scales
 * are for products elsewhere that scale by rows or by blocks of 128.
 *
 * Layout. MX_FP8_ROW and MX_FP8_BLOCK: codes [rows, cols] bytes, scales [rows]
 * or [rows, ceil(cols / 128)] fp32. The microscaled formats: a row of codes is
 * padded with zero codes to 32 columns; E2M1 codes go two a byte, the first in
 * the low half. Their scales lie in tiles of 128 rows by 4 blocks, 512 bytes,
 * the tiles of 128 rows one after the other: block b of row r is at
 *   ((r / 128) * ceil(blocks / 4) + b / 4) * 512 + (r % 32) * 16 +
 *   (r % 128 / 32) * 4 + b % 4,
 * and bytes of rows or blocks that the matrix does not have are 0. That is the
 * layout that block-scaled matrix products of this GPU generation take.
 */
typedef enum {
  MX_FP8_ROW = 0,
  MX_FP8_BLOCK = 1,
  MX_MXFP8 = 2,
  MX_MXFP4 = 3,
  MX_NVFP4 = 4
} mx_format;

typedef struct {
  void* codes;       /* device; microscaled formats: 16-byte aligned */
  void* scales;      /* device; 4-byte, microscaled formats 16-byte aligned */
  const float* mul;  /* MX_NVFP4: one positive finite fp32 on the device (commonly
                        2688 / amax of the matrix), NULL = 1; else ignored */
  mx_format format;
  int64_t rows;      /* 0 .. 2^31 - 129 */
  int64_t cols;      /* 1 .. 2^31 - 129 */
} mx_matrix;

/* Bytes of a matrix's codes and of its scales. */
ln_status mx_matrix_bytes(mx_format format, int64_t rows, int64_t cols, size_t* codes,
                          size_t* scales);

/*
 * mx_norm_fwd: ln_fwd with its result quantised into `q` ([rows, hidden]): the
 * fp32 result, not one rounded to dtype first. out_sum, mean and rstd are what
 * ln_bwd takes, so the backward is that of the norm with the gradient of the
 * dequantised result passed straight through.
 *
 * y    [rows, hidden] dtype, NULL = not stored.
 * q    overlaps no other tensor of the call.
 * Other arguments, alignment, limits of hidden and errors are those of ln_fwd
 * (q's codes count as a tensor pointer for the vectorised path); rows stay
 * below 2^31 - 128.
 */
ln_status mx_norm_fwd(const void* x, const void* bias, const void* residual, const void* gamma,
                      const void* beta, float eps, ln_mode mode, int zero_centered_gamma,
                      void* out_sum, void* y, float* mean, float* rstd, const mx_matrix* q,
                      cudaStream_t stream, ln_dtype dtype);

/*
 * mx_quantize: x, or with `transpose` its transpose, into q. x is [q.rows,
 * q.cols] ([q.cols, q.rows] with transpose), columns contiguous, x_row >= 0
 * elements from one row to the next. A transposed operand is what a product's
 * gradients need: they contract over the rows.
 */
ln_status mx_quantize(const void* x, int64_t x_row, int transpose, const mx_matrix* q,
                      cudaStream_t stream, ln_dtype dtype);

/* mx_dequantize: the values of q, rounded to dtype, into y [rows, cols], y_row
 * >= cols elements from one row to the next. */
ln_status mx_dequantize(const mx_matrix* q, void* y, int64_t y_row, cudaStream_t stream,
                        ln_dtype dtype);

/*
 * mx_product: out[m, n] = alpha * sum over k of A[m, k] * B[n, k] + bias[n] +
 * residual[m, n], A and B the values of two matrices of one microscaled format
 * with the same number of columns (for a projection: activations by rows and
 * weights by output features). Products are exact, sums fp32 in the tensor
 * cores, the scales' included; the rest is fp32, rounded once to dtype.
 *
 * bias      [N] dtype, NULL = none.
 * residual  [M, N] dtype, residual_row >= N elements a row, NULL = none; may be out
 *           itself (same row stride), shares no element with it otherwise (columns
 *           of one buffer side by side are accepted where that can be seen from the
 *           strides).
 * out       [M, N] dtype, out_row >= N elements a row.
 * psum, psq [M, ceil(N / 128)] fp32 or NULL (both or none): sums of the stored
 *           rows over tiles of 128 columns and their squares about the tile's
 *           mean: what ln_fwd_from_partials takes as LN_PARTIALS_SUM_M2 with
 *           tile_cols = 128.
 * The result does not depend on how often or where the call runs on one GPU
 * model: sums that are split are joined in a fixed order.
 */
ln_status mx_product(const mx_matrix* a, const mx_matrix* b, float alpha, const void* bias,
                     const void* residual, int64_t residual_row, void* out, int64_t out_row,
                     float* psum, float* psq, cudaStream_t stream, ln_dtype dtype);

/* Static, human-readable name of a status code. */
const char* ln_status_string(ln_status status);

/* The cudaError_t behind the last LN_ERR_CUDA on the calling thread. */
int ln_last_cuda_error(void);

/*
 * Device-side failure report. The pipelined kernels (the ring kernels, the
 * product and the transposing quantiser) wait on shared-memory barriers for
 * their copies and tensor-core work; every such wait gives up after about a second,
 * sets a bit in a device error word and lets the kernel finish early (its
 * outputs are then not valid). This call waits for `stream`, ORs the error
 * words of all kernels into *flags (bit 0: a wait timed out) and clears them.
 * It synchronises `stream`; 0 in *flags means no kernel reported a failure.
 */
ln_status ln_device_error(cudaStream_t stream, unsigned* flags);

#ifdef __cplusplus
}
#endif

#endif /* NORMFUSE_H */
