/*
 * awq_b200.h -- C ABI of libawq_b200.so, the AWQ W4A16 group-quantized linear
 * layer for NVIDIA B200 (sm_100a).
 *
 * The operations restate the activation-aware weight quantization described
 * on the AWQ pages:
 *   - lansai AWQ explainer (ai.lansai.wang/107648), section "AWQ 的四步链路":
 *     Y = XW is rewritten with a positive per-input-channel scale s as
 *     Y = (X/s)(sW); calibration activations give per-channel magnitudes;
 *     the scaled weights are quantized by group and packed with their
 *     scale and zero point;
 *   - "Awq Quantization" (skillselion.com), "How AWQ Works" (objective
 *     ||Q(W*s)(s^-1*X) - W*X||), "Group Size Configuration" (groups of 128,
 *     4 bits), "Zero-Point Quantization" (asymmetric codes with an offset),
 *     "WQLinear Kernel Variants" (a GEMV kernel for single-token decode and
 *     a GEMM kernel for batches).
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE memory owned by the caller, on the
 *     current CUDA device; the library allocates nothing on these calls and
 *     keeps no pointer after it returns.
 *   - float16 data are passed as IEEE binary16 bit patterns (uint16_t).
 *   - Every tensor is dense row-major; device pointers must be 16-byte aligned.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every
 *     call is asynchronous on that stream.
 *   - Errors detectable on the host (null pointers, shapes, alignment,
 *     device architecture, workspace size) are returned before anything is
 *     launched.  Errors found on the device (non-finite inputs, a bounded wait
 *     that ran out) are written as an awq_status_t value into *dev_status if
 *     dev_status is not NULL; the first error wins, the library never clears
 *     it: the caller zeroes it and reads it after synchronizing the stream.
 *   - Outputs must not alias inputs.
 *   - The library keeps per-device state (device checks, kernel attributes,
 *     encoded tensor maps, the no-allocation scratch address): do not use it
 *     on a device after cudaDeviceReset in the same process.
 *
 * Data layout (K input channels, N output channels, G = K/128 groups)
 *   W       binary16 [K, N]     Y = X W
 *   s       binary16 [K]        per-input-channel scale
 *   Q       int32 [K/8, N]      bits [4j, 4j+4) of Q[k8, n] hold the 4-bit code
 *                               of row 8*k8 + j, column n (sequential nibbles)
 *   scales  binary16 [G, N]     per-group step of the 4-bit grid
 *   zeros   int32 [G, N/8]      bits [4j, 4j+4) of zeros[g, n8] hold the zero
 *                               point of column 8*n8 + j; absent (NULL) for
 *                               symmetric weights, whose zero point is 8
 *   X       binary16 [M, K]     activations;  Y binary16 [M, N]
 */
#ifndef AWQ_B200_H
#define AWQ_B200_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define AWQ_API __attribute__((visibility("default")))
#else
#define AWQ_API
#endif

#define AWQ_GROUP_SIZE 128      /* q_group_size ("Group Size Configuration") */
#define AWQ_W_BIT 4             /* w_bit: codes 0..15                          */
#define AWQ_MAX_CALIB_ROWS 8192 /* keeps the double sum of |x| exact           */
#define AWQ_MAX_K 262144
#define AWQ_MAX_N 1048576
#define AWQ_MAX_M 1048576
#define AWQ_ABI_VERSION 5  /* 2: symmetric weights; 3: 1/s folded upstream;
                               4: every matmul takes a zero-filled workspace;
                               scale search over alpha; weight clipping;
                               5: matmul workspaces for M >= 64 hold the
                               prefill kernel's partial tiles.  Entry points
                               added without a change to earlier ones (the
                               fused epilogue, the 4-bit cache) keep it: look
                               them up by name */

typedef enum {
    AWQ_OK = 0,
    AWQ_ERR_NULL = 1,           /* a required pointer is NULL                      */
    AWQ_ERR_SHAPE = 2,          /* K % 128, N % 8, M < 1, R < 1, or above a limit  */
    AWQ_ERR_ALIGN = 3,          /* a device pointer is not 16-byte aligned         */
    AWQ_ERR_NONFINITE = 4,      /* NaN/Inf in W, s, X_cal or the statistics        */
    AWQ_ERR_ARCH = 5,           /* the current device is not sm_100 (B200)         */
    AWQ_ERR_CUDA = 6,           /* a CUDA runtime/driver call or launch failed     */
    AWQ_ERR_DEVICE_TIMEOUT = 7, /* a bounded wait inside a kernel ran out          */
    AWQ_ERR_WORKSPACE = 8,      /* workspace NULL or smaller than required         */
    AWQ_ERR_RANGE = 9,          /* a length, slot, page or offset in device memory lies
                                   outside what the call was given                 */
    AWQ_ERR_CAPACITY = 10       /* the free pages do not suffice                   */
} awq_status_t;

/* Activations of awq_w4a16_gemm_epilogue. */
typedef enum {
    AWQ_ACT_NONE = 0,
    AWQ_ACT_RELU = 1,
    AWQ_ACT_SILU = 2,           /* t / (1 + e^-t)                                  */
    AWQ_ACT_GELU = 3,           /* t (1 + erf(t / sqrt 2)) / 2                     */
    AWQ_ACT_GELU_TANH = 4       /* t (1 + tanh(sqrt(2/pi) (t + 0.044715 t^3))) / 2 */
} awq_act_t;

typedef void *awq_stream_t; /* a cudaStream_t */

/* Human-readable name of a status code (static storage). */
AWQ_API const char *awq_status_string(awq_status_t status);

/* AWQ_ABI_VERSION of the loaded library. */
AWQ_API int awq_abi_version(void);

/*
 * Activation statistics -- lansai explainer, "AWQ 的四步链路", row "采集激活"
 * (collect the layer-input magnitude on calibration data).
 *   m[k] = (1/R) * sum_r |xcal[r, k]|
 * The sum is exact (double; every binary16 is a multiple of 2^-24), divided
 * once in double and rounded once to float, so the result does not depend on
 * the reduction order.
 *   xcal  binary16 [R, K], 1 <= R <= AWQ_MAX_CALIB_ROWS ("Calibration samples
 *         are empty" is AWQ_ERR_SHAPE), K % 8 == 0
 *   m     float [K] (output)
 * Device errors: AWQ_ERR_NONFINITE if xcal holds NaN/Inf (m is still written).
 */
AWQ_API awq_status_t awq_act_stats(const uint16_t *xcal, int64_t R, int64_t K, float *m,
                           int32_t *dev_status, awq_stream_t stream);

/*
 * Per-channel scale -- lansai explainer, "AWQ 的四步链路" (Y = (X/s)(sW));
 * "Awq Quantization", "How AWQ Works" (s lowers ||Q(W*s)(s^-1*X) - W*X||).
 * One point of the scale family: s = m^0.5, normalised by the geometric
 * centre of its extremes:
 *   t_k = sqrt(max(m_k, 1e-8)),  c = sqrt(max_j t_j * min_j t_j),
 *   s_k = binary16_RNE(t_k / c)          (double arithmetic, IEEE rounding)
 *   m  float [K] (K >= 1);  s  binary16 [K] (output)
 * Device errors: AWQ_ERR_NONFINITE if some m_k is NaN/Inf/negative (s is
 * then left unspecified).
 */
AWQ_API awq_status_t awq_compute_scales(const float *m, int64_t K, uint16_t *s, int32_t *dev_status,
                                awq_stream_t stream);

/*
 * Fold, quantize and pack -- lansai explainer, "AWQ 的四步链路" (enlarge the
 * salient channels' weights, sW, then quantize by group; row "真实量化/打包");
 * "Awq Quantization", "Group Size Configuration", "Zero-Point Quantization".
 * Per group g (rows 128g..128g+127) and column n, with w' = float(w) * float(s_k):
 *   r       = max(max w' - min w', 1e-5f)
 *   scale_h = binary16_RNE(r / 15)  (the smallest subnormal if that is 0)
 *   z       = clamp(rint(-min w' / scale_h), 0, 15)
 *   q       = clamp(rint(w' / scale_h) + z, 0, 15)   (rint: ties to even)
 * all in IEEE float arithmetic; the outputs are bit-exact functions of W, s.
 *   W binary16 [K, N], s binary16 [K] (> 0), K % 128 == 0, N % 8 == 0
 *   Q int32 [K/8, N], scales binary16 [K/128, N], zeros int32 [K/128, N/8] (outputs)
 * Device errors: AWQ_ERR_NONFINITE if W or s holds NaN/Inf or s <= 0
 * ("NaN detected in weights", "Awq Quantization", Troubleshooting Guide).
 */
AWQ_API awq_status_t awq_quantize_pack(const uint16_t *W, const uint16_t *s, int64_t K, int64_t N,
                               int32_t *Q, uint16_t *scales, int32_t *zeros,
                               int32_t *dev_status, awq_stream_t stream);

/*
 * Symmetric variant -- "Awq Quantization", "Zero-Point Quantization"
 * (zero_point False: no per-group offset, for symmetric weight distributions
 * and for kernels without zero points).  The page names only the flag; this
 * library reads it as a grid centred at zero whose largest level is 7 steps:
 *   a       = max(max |w'|, 1e-5f)
 *   scale_h = binary16_RNE(a / 7)  (the smallest subnormal if that is 0)
 *   q       = clamp(rint(w' / scale_h), -8, 7) + 8          (rint: ties to even)
 * i.e. the asymmetric codes with z = 8.  No zeros tensor is written; pass
 * zeros = NULL to the matmul entry points for these weights.
 *   W, s, K, N, Q, scales as for awq_quantize_pack.
 * Device errors: as for awq_quantize_pack.
 */
AWQ_API awq_status_t awq_quantize_pack_symmetric(const uint16_t *W, const uint16_t *s, int64_t K,
                                         int64_t N, int32_t *Q, uint16_t *scales,
                                         int32_t *dev_status, awq_stream_t stream);

/*
 * Fold, quantize and pack with weight clipping -- "Awq Quantization",
 * calibration parameters: apply_clip ("Apply weight clipping"); the page names
 * only the flag.  This library reads it, per group g (rows 128g..128g+127)
 * and column n with w' = float(w) * float(s_k), as:
 *   candidates  c_i = 1 - i/20, i = 0 .. n_cand-1 (1 <= n_cand <= 11, down to
 *               c = 1/2; c_0 = 1 is no clipping)
 *   clipped     lo = c * min w', hi = c * max w' (float); step and zero point
 *               from [lo, hi] as in awq_quantize_pack (r = max(hi - lo, 1e-5f),
 *               scale_h = binary16_RNE(r / 15), z = clamp(rint(-lo / scale_h),
 *               0, 15)); every weight of the group coded on that grid,
 *               q = clamp(rint(w' / scale_h) + z, 0, 15)
 *   loss        sum over the R calibration rows of
 *               (sum_{k in g} (xcal[r,k] / s_k) ((q - z) scale_h - w'))^2
 *               (float arithmetic)
 *   choice      the first candidate (largest c) with the minimum loss.
 * With n_cand = 1 the outputs equal awq_quantize_pack's bit for bit.  The
 * step, zero point and codes of a chosen candidate are bit-exact functions of
 * W, s and that candidate; the choice itself rests on float losses, so it can
 * differ from an exact (double) evaluation only between candidates whose
 * losses agree to float rounding.
 *   W binary16 [K, N], s binary16 [K] (> 0), xcal binary16 [R, K]
 *   (1 <= R <= AWQ_MAX_CALIB_ROWS), K % 128 == 0, N % 8 == 0
 *   Q, scales, zeros as for awq_quantize_pack (outputs); ratio_index int32
 *   [K/128, N] receives the chosen i (may be NULL)
 * Device errors: AWQ_ERR_NONFINITE for NaN/Inf in W, s or xcal, or s <= 0.
 */
AWQ_API awq_status_t awq_quantize_pack_clip(const uint16_t *W, const uint16_t *s, const uint16_t *xcal,
                                            int64_t R, int64_t K, int64_t N, int32_t n_cand, int32_t *Q,
                                            uint16_t *scales, int32_t *zeros, int32_t *ratio_index,
                                            int32_t *dev_status, awq_stream_t stream);

/*
 * Fused-dequantization matmul -- lansai explainer, "AWQ 的四步链路"
 * (Y = (X/s)(sW)); "Awq Quantization", "WQLinear Kernel Variants" (GEMV for
 * batch size 1, GEMM for batches).
 *   Y[m, n] = sum_k (X[m, k] / s_k) * (q[k, n] - z[g(k), n]) * scale_h[g(k), n]
 * with the nibble unpack and (q - z) * scale dequantisation done inside the
 * kernel (no dequantised weight matrix is ever written to memory), X / s
 * rounded to binary16 for the tensor cores, float accumulation, Y rounded to
 * binary16.  Results agree with the exact definition within
 * max|dY| <= 1e-2 * max|Y| and ||dY||_F <= 5e-3 * ||Y||_F.
 *
 * awq_w4a16_gemv is the M = 1 (single-token decode) entry point:
 *   X binary16 [1, K], Y binary16 [1, N].
 * awq_w4a16_gemm takes any 1 <= M <= AWQ_MAX_M and picks its tile path
 * internally: the decode GEMV for M <= 2, register-fed tensor cores for
 * 3 <= M < 24, tcgen05/TMEM for M >= 24 (small batch from 24, prefill from 64).
 *   K % 128 == 0, N % 8 == 0, Q/scales/zeros as produced by awq_quantize_pack;
 *   zeros = NULL for weights from awq_quantize_pack_symmetric (zero point 8).
 *   s = NULL when X already holds X/s (1/s folded into the operator that
 *   produced X, e.g. by awq_fold_inverse_scale): X is then used as it is, and
 *   with X = awq_fold_inverse_scale(X, s) the result equals, bit for bit,
 *   the call with the original X and s.
 * Workspace: caller-owned device memory of at least *_workspace_size() bytes,
 * never NULL.  It must be zero-filled (e.g. cudaMemsetAsync) before its first
 * use: its first 32 KB are a counter block that a call expects at zero and
 * leaves at zero when it completes without a device error.  The rest holds
 * X / s and, for M >= 64, the partial sums of output tiles whose k range is
 * split between CTAs (at most 20 MB); it is overwritten.  The size depends on
 * M, K and N, not on the device.  Calls on one stream may share a
 * workspace, as long as no two host threads make them at once: a call enqueues
 * up to two kernels that pass X / s through it, and the other call's must not
 * come between.  Calls that can run at the same time need separate ones.  After a
 * device error (AWQ_ERR_DEVICE_TIMEOUT) zero the workspace again.
 * Device errors: AWQ_ERR_DEVICE_TIMEOUT if an internal pipeline wait ran out
 * (Y is then unspecified).  For M >= 64 with few output tiles the call may run
 * a grid whose CTAs wait (up to 1 s) for partial sums from later CTAs of the
 * same grid; the grid is sized so that all of its CTAs fit on the GPU at once,
 * so a kernel on another stream that keeps SMs occupied for longer than that
 * can make such a call report AWQ_ERR_DEVICE_TIMEOUT instead of finishing.
 * Stream ordering: these kernels use programmatic dependent launch, so a call
 * may start while the previous kernel on the stream is still finishing.  X and
 * the workspace are touched only after that kernel has completed.  Q, scales
 * and zeros are treated as layer state and may be read before it completes:
 * they must not be written by a kernel that triggers programmatic dependent
 * launch early.  Ordinary kernels, copies and awq_quantize_pack complete before
 * any dependent starts, so writing the weights with them is safe.
 */
/*
 * Fold 1/s upstream -- lansai explainer, "AWQ 的四步链路": Y = XW = (X/s)(sW),
 * with the X/s side carried by the operator that produces X (a normalisation
 * weight: rows = 1; or activations divided once for several projections).
 *   out[r, k] = binary16_RNE(float(a[r, k]) / float(s_k))   (IEEE division)
 * the same operations the matmul applies to X when it is given s.
 *   a    binary16 [rows, K], 1 <= rows <= AWQ_MAX_M, K % 8 == 0
 *   s    binary16 [K] (> 0);  out binary16 [rows, K] (output, not aliasing a)
 * Device errors: AWQ_ERR_NONFINITE if some s_k is NaN/Inf or <= 0 (out is
 * still written).
 */
AWQ_API awq_status_t awq_fold_inverse_scale(const uint16_t *a, int64_t rows, int64_t K,
                                    const uint16_t *s, uint16_t *out, int32_t *dev_status,
                                    awq_stream_t stream);

AWQ_API size_t awq_w4a16_gemv_workspace_size(int64_t K, int64_t N);
AWQ_API awq_status_t awq_w4a16_gemv(const uint16_t *X, const uint16_t *s, const int32_t *Q,
                            const uint16_t *scales, const int32_t *zeros, int64_t K, int64_t N,
                            uint16_t *Y, void *workspace, size_t workspace_bytes,
                            int32_t *dev_status, awq_stream_t stream);

AWQ_API size_t awq_w4a16_gemm_workspace_size(int64_t M, int64_t K, int64_t N);
AWQ_API awq_status_t awq_w4a16_gemm(const uint16_t *X, const uint16_t *s, const int32_t *Q,
                            const uint16_t *scales, const int32_t *zeros, int64_t M, int64_t K,
                            int64_t N, uint16_t *Y, void *workspace, size_t workspace_bytes,
                            int32_t *dev_status, awq_stream_t stream);

/*
 * Scales of one grid point of the scale search (below): alpha = j/8,
 * 0 <= j <= 8, by the same fixed chain of IEEE double operations,
 *   s = binary16_RNE(t / sqrt(max t * min t)),  t = m^(j/8)
 * (j = 4 gives awq_compute_scales bit for bit, j = 0 gives s = 1).
 *   m float [K] (K >= 1); s binary16 [K] (output)
 * Device errors: AWQ_ERR_NONFINITE if some m_k is NaN/Inf/negative.
 */
AWQ_API awq_status_t awq_scales_alpha(const float *m, int64_t K, int32_t j, uint16_t *s,
                                      int32_t *dev_status, awq_stream_t stream);

/*
 * Scale search over alpha -- "Awq Quantization", "How AWQ Works" (s is chosen
 * to make L(s) = ||Q(W*s)(s^-1*X) - W*X|| small); lansai explainer, "AWQ 的四步
 * 链路", row "搜索缩放" (try channel scalings, keep the one with the smallest
 * reconstruction error).  The pages give neither the family nor the grid;
 * this library reads them as:
 *   family  s(alpha) = m^alpha normalised as in awq_compute_scales (whose scale
 *           is the alpha = 1/2 point), m = awq_act_stats(xcal)
 *   grid    alpha = j/8, j = 0..8, m^alpha by one fixed chain of IEEE double
 *           operations: u = max(m, 1e-8), r1 = sqrt(u), r2 = sqrt(r1),
 *           r3 = sqrt(r2); t = u for j = 8, else the product of r1, r2, r3
 *           selected by the bits 4, 2, 1 of j, in that order;
 *           s = binary16_RNE(t / sqrt(max t * min t))
 *   loss    losses[j] = sum over the R calibration rows and N outputs of
 *           (Yq - Y)^2 (double), Yq = awq_w4a16_gemm(xcal, s(j), awq_quantize_pack(W, s(j)))
 *           and Y = xcal W (tensor cores, float accumulation)
 *   choice  *j_best = the smallest j with the minimum loss; s_best = s(j_best),
 *           bit for bit the scale of that grid point.
 *   xcal  binary16 [R, K], 1 <= R <= AWQ_MAX_CALIB_ROWS; W binary16 [K, N],
 *         K % 128 == 0, N % 8 == 0
 *   losses double [9], s_best binary16 [K], j_best int32 [1] (device outputs)
 *   workspace  at least awq_scale_search_workspace_size(R, K, N) bytes,
 *         zero-filled before its first use (it embeds a matmul workspace)
 * Device errors: AWQ_ERR_NONFINITE for NaN/Inf in xcal or W (the outputs are
 * then unspecified); AWQ_ERR_DEVICE_TIMEOUT as for the matmul.
 */
AWQ_API size_t awq_scale_search_workspace_size(int64_t R, int64_t K, int64_t N);
AWQ_API awq_status_t awq_scale_search(const uint16_t *xcal, int64_t R, int64_t K, const uint16_t *W,
                                      int64_t N, double *losses, uint16_t *s_best, int32_t *j_best,
                                      void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                      awq_stream_t stream);

/*
 * awq_w4a16_gemm_noalloc -- awq_w4a16_gemm for callers that cannot hand the
 * library a workspace.  No counterpart in the AWQ paper or pages: this is an
 * integration entry point of this library only.
 *
 * Who needs it: code that is not allowed to allocate device memory at the point
 * where it runs the layer -- for example an inference-engine plugin whose
 * execute callback may only use memory the engine planned beforehand, a
 * real-time or fixed-budget deployment that allocates everything at start-up,
 * or a plain C caller that has no device allocator of its own.  Instead of a
 * caller-provided workspace, X / s is staged in a fixed scratch array that is
 * part of the library's device image: AWQ_NOALLOC_SCRATCH_BYTES on every GPU
 * that loads the library, held until the process exits.  The call itself
 * allocates nothing (no cudaMalloc, no allocating library routine).
 *
 * Arguments, layouts, tolerance and errors are those of awq_w4a16_gemm, minus
 * the workspace.  Limit: awq_w4a16_gemm_workspace_size(M, K, N) must not exceed
 * AWQ_NOALLOC_SCRATCH_BYTES (32 KB of counters + 2 * M * K bytes of X / s +
 * for M >= 64 up to 20 MB of partial tiles; M * K <= 2 Mi - 16 Ki elements
 * always fits); larger problems return AWQ_ERR_WORKSPACE before anything runs.
 * Set-up: the first call on each device (with that device current) looks up
 * the scratch array's device address; make that first call before any stream
 * capture begins.
 * Sharing: every call on a device uses the same scratch array, which keeps the
 * last call's contents.  Its counter block starts at zero (the array is
 * zero-initialised when the library is loaded) and every call that completes
 * without a device error leaves it at zero; the rest is written before it is
 * read.  Calls whose executions overlap on the GPU (different streams without
 * ordering between them) race on the scratch array and give undefined
 * results; order them on one stream or with events.  Host threads may make
 * calls on one stream at the same time: each call's kernels are enqueued together.
 */
#define AWQ_NOALLOC_SCRATCH_BYTES ((size_t)24 << 20)
AWQ_API awq_status_t awq_w4a16_gemm_noalloc(const uint16_t *X, const uint16_t *s, const int32_t *Q,
                                            const uint16_t *scales, const int32_t *zeros,
                                            int64_t M, int64_t K, int64_t N, uint16_t *Y,
                                            int32_t *dev_status, awq_stream_t stream);

/*
 * awq_w4a16_gemm with what follows the product fused into it, before the
 * single rounding to binary16 ("Awq Quantization", "Layer Fusion": gate and up
 * as one projection):
 *   t[m, n] = sum_k (X[m, k] / s_k) dequant(Q)[k, n] + bias[n]      (float)
 *   a       = act(t)                          Y [M, N], or, gated != 0,
 *   a[m, j] = act(t[m, 2j]) * t[m, 2j + 1]    Y [M, N/2]: the columns of gate
 *             and up interleaved when the weights were quantized; N % 16 == 0
 *   Y       = binary16_RNE(a + residual)
 *   bias      binary16 [N] or NULL
 *   act       an awq_act_t
 *   residual  binary16, the shape of Y, or NULL; residual == Y adds in place
 *             (any other overlap is not allowed)
 * X, s, Q, scales, zeros, M, K, N, the workspace, the tile paths and the device
 * errors are those of awq_w4a16_gemm, and with no bias, activation, gate and
 * residual so is every bit of Y.  As there, from 24 tokens on the dequantized
 * weights are rounded to binary16 before they are multiplied; a gate times its
 * column holds that error twice (3.4e-4 of the output's norm, where the output's
 * own rounding is 2.1e-4).  bias is layer state like scales; residual is
 * read only after the previous kernel on the stream has completed.
 */
AWQ_API awq_status_t awq_w4a16_gemm_epilogue(const uint16_t *X, const uint16_t *s, const int32_t *Q,
                                             const uint16_t *scales, const int32_t *zeros, int64_t M,
                                             int64_t K, int64_t N, const uint16_t *bias, int32_t act,
                                             int32_t gated, const uint16_t *residual, uint16_t *Y,
                                             void *workspace, size_t workspace_bytes,
                                             int32_t *dev_status, awq_stream_t stream);

/* ------------------------------------------------------------------------
 * Paged 4-bit key/value cache.
 *
 * The weights' 4-bit grid applied to the other tensor that fills a serving
 * GPU: the keys and values of every token, one group per token and head.
 * Head dimension D = 64 or 128; page_size = 16, 32, 64, 128 or 256 tokens.
 *
 *   cache        uint8 [num_pages, kv_heads, page_size / 16] blocks; a block is
 *                16 tokens of one head, 16 D + 128 bytes: key codes (16 rows of
 *                D / 2 bytes, sequential nibbles as in Q), value codes, then 16
 *                words for the keys and 16 for the values: step (binary16) in
 *                bits 0..15, zero point in bits 16..31
 *   block_table  int32 [B, max_pages]: the pages of each request, in order
 *   lens         int32 [B]: cached tokens of each request
 *   free_pages   int32 [num_pages], free_count int32 [1]: a stack of free pages
 *   slot         page * page_size + position in the page (int64); negative: none
 * Lengths and tables live in device memory and are read there, so a captured
 * graph follows them.  What they hold is checked on the device: an entry out of
 * range is reported as AWQ_ERR_RANGE and skipped, never followed.
 * ------------------------------------------------------------------------ */
#define AWQ_KV4_BLOCK 16
#define AWQ_KV4_MAX_REQUESTS 4096
#define AWQ_KV4_MAX_HEADS 1024      /* query heads; key/value heads likewise */
#define AWQ_KV4_MAX_PAIRS ((int64_t)1 << 52) /* query rows x positions of one request and
                                       key/value head: close to an hour of GPU time */

/* Bytes of one page for one head; 0 for an unsupported page_size or D. */
AWQ_API size_t awq_kv4_page_bytes(int64_t page_size, int64_t D);

/*
 * Block table, slot map and positions of a step, from request lengths.
 * Request b has lens[b] tokens in ceil(lens[b] / page_size) pages and gets
 * new_lens[b] >= 0 more; the pages it lacks are popped from the stack, in the
 * order of requests, then of positions, and entered in its table row.
 *   slots      int64 [T] (output): of every new token, requests one after the
 *              other; -1 in the rows behind the last one (T >= their number)
 *   positions  int32 [T] (output) or NULL: position in the request; -1 there
 *   cu         int32 [B + 1] (output): first row of each request, and their end
 *   lens_out, free_count_out  (outputs): lengths and stack after the step; may be
 *              lens and free_count themselves
 *   1 <= B <= AWQ_KV4_MAX_REQUESTS, 1 <= T < 2^31, max_pages * page_size < 2^31
 * Device errors: AWQ_ERR_RANGE (a negative length, more tokens than T, more
 * pages than max_pages, free_count outside 0..num_pages), AWQ_ERR_CAPACITY (too few
 * free pages).  Then nothing is reserved: slots and positions are -1, cu is 0,
 * lengths, table and stack are unchanged.  AWQ_ERR_RANGE also for a page outside
 * the cache, in the table where new tokens go or on the stack: those tokens get slot
 * -1, a table entry from the stack becomes -1, and the rest of the step stands.
 */
AWQ_API awq_status_t awq_kv4_reserve(const int32_t *new_lens, const int32_t *lens, int64_t B,
                                     int64_t page_size, int32_t *block_table, int64_t max_pages,
                                     const int32_t *free_pages, const int32_t *free_count,
                                     int64_t num_pages, int64_t T, int64_t *slots, int32_t *positions,
                                     int32_t *cu, int32_t *lens_out, int32_t *free_count_out,
                                     int32_t *dev_status, awq_stream_t stream);

/*
 * Ends requests: the pages of every request b with done[b] != 0 are pushed onto
 * the stack, in the order of requests, then of positions; its length becomes 0
 * and the table entries of those pages -1.
 *   done int32 [B]; lens, block_table, free_pages, free_count updated in place
 * Entries of -1 are passed over: pages before a sliding window that the caller has
 * already pushed (to free_pages[free_count], entry -1, free_count + 1).
 * Device errors: AWQ_ERR_RANGE (a length or page out of range, more pages than
 * num_pages in the stack); then nothing is changed.  Every page that an ended
 * request still holds has to be in its row, and in no other request's: a page
 * that two rows share would be pushed twice, which is not detected.
 */
AWQ_API awq_status_t awq_kv4_release(const int32_t *done, int32_t *lens, int64_t B, int64_t page_size,
                                     int32_t *block_table, int64_t max_pages, int32_t *free_pages,
                                     int32_t *free_count, int64_t num_pages, int32_t *dev_status,
                                     awq_stream_t stream);

/*
 * Quantizes the keys and values of T tokens into their slots.  Per token and head:
 *   lo = min(0, min x), hi = max(0, max x)
 *   step = binary16_RNE(max(hi - lo, 1e-5f) / 15)
 *   z = clamp(rint(-lo / step), 0, 15)
 *   q = clamp(rint(x * (1 / step)) + z, 0, 15)            (rint: ties to even)
 * in IEEE float; the result is bit-exact.  The value it stands for is (q - z) step.
 *   k, v   binary16, token t at k + t * k_stride (elements), heads of D one after
 *          the other; strides >= kv_heads * D, multiples of 8: slices of a fused
 *          projection's rows are taken as they are
 *   slots  int64 [T]; a negative one stores nothing.  A slot named twice holds
 *          one token's codes or a mix of both
 * Device errors: AWQ_ERR_RANGE (a slot outside the cache; that token is not
 * stored), AWQ_ERR_NONFINITE (NaN or Inf; that token's row is unspecified).
 */
AWQ_API awq_status_t awq_kv4_append(const uint16_t *k, int64_t k_stride, const uint16_t *v,
                                    int64_t v_stride, const int64_t *slots, int64_t T, int64_t kv_heads,
                                    int64_t D, uint8_t *cache, int64_t num_pages, int64_t page_size,
                                    int32_t *dev_status, awq_stream_t stream);

/*
 * The stored keys and values of T slots: k, v binary16 [T, kv_heads, D]
 * (outputs), (q - z) step rounded once; zeros for a negative slot.
 * Device errors: AWQ_ERR_RANGE (a slot outside the cache; zeros).
 */
AWQ_API awq_status_t awq_kv4_load(const int64_t *slots, int64_t T, int64_t kv_heads, int64_t D,
                                  const uint8_t *cache, int64_t num_pages, int64_t page_size,
                                  uint16_t *k, uint16_t *v, int32_t *dev_status, awq_stream_t stream);

/*
 * Attention over the cache.  Request b owns the query rows cu[b] .. cu[b+1] - 1;
 * its i-th query stands at position p = lens[b] - n_b + i (n_b its number of
 * queries: the request's last tokens, already stored) and sees the cached
 * positions j <= p, with window > 0 only those with j > p - window:
 *   out = sum_j softmax_j(scale * q . k_j) v_j
 * in float, over the values the codes stand for, rounded once to binary16; a
 * query that sees nothing gives zeros.  Query head h reads key/value head
 * h / (q_heads / kv_heads).  Pages that lie wholly before the window of a
 * request's first query are not looked at: their table entries may be -1.
 * Requests of one call may differ in n_b: those with many query rows and those
 * with few go to two kernels, one after the other.
 *   q       binary16, row t at q + t * q_stride (elements, a multiple of 8,
 *           >= q_heads * D)
 *   cu      int32 [B + 1], ascending, or NULL: one query per request (T >= B)
 *   max_new the most queries of one request (a bound known on the host)
 *   out     binary16 [T, q_heads, D] (output); rows of no request are not written
 *   workspace  at least awq_kv4_attention_workspace_size(D) bytes, no initial
 *           contents required, overwritten; calls that can run at the same time
 *           need separate ones, and so do calls of two host threads, on one
 *           stream too (a call enqueues up to four kernels that share it)
 *   q_heads % kv_heads == 0, both <= AWQ_KV4_MAX_HEADS; 1 <= B <=
 *   AWQ_KV4_MAX_REQUESTS; 1 <= T, max_new < 2^31; tokens = max_pages * page_size < 2^31;
 *   with rows = max_new * q_heads / kv_heads (requests of more than 48 rows go to the
 *   kernel for many rows, so that more count as 48 in the first):
 *   B * kv_heads * (rows <= 8 ? 1 : ceil(min(rows, 48) / 16)) * (ceil(tokens / 64) + 8) < 2^32,
 *   rows * tokens <= AWQ_KV4_MAX_PAIRS
 * The result depends on the number of SMs and on the bounds max_new, max_pages
 * and T (which choose the kernel and the order of sums), never on timing: the
 * same call gives the same bits.
 * Device errors: AWQ_ERR_RANGE (a length above max_pages * page_size or negative:
 * clamped; a page outside the cache: its tokens are not seen; offsets outside
 * 0..T or a request with more than max_new queries: its rows are not written),
 * AWQ_ERR_DEVICE_TIMEOUT.
 */
AWQ_API size_t awq_kv4_attention_workspace_size(int64_t D);
AWQ_API awq_status_t awq_kv4_attention(const uint16_t *q, int64_t q_stride, int64_t T, int64_t q_heads,
                                       const uint8_t *cache, int64_t num_pages, int64_t page_size,
                                       int64_t kv_heads, int64_t D, const int32_t *block_table,
                                       int64_t max_pages, const int32_t *lens, const int32_t *cu, int64_t B,
                                       int64_t max_new, float scale, int64_t window, uint16_t *out,
                                       void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                       awq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* AWQ_B200_H */
