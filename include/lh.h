/*
 * lh.h -- C ABI of the MI355X (gfx950) local-Hessian NVFP4 weight-scale calibration library.
 *
 * The library computes, on one GPU, the two parts of local-Hessian-weighted NVFP4 weight-scale
 * calibration:
 *   1. per 16-wide input-channel block n, the local Hessian H_n = X[:,n]^T X[:,n] / B, the
 *      activation-aware cross matrix P_n = X_q^T (X_q - X) / B and the importance vector
 *      Imp_i = ||X[:,i]||^2;
 *   2. for every 16-element weight block, the exhaustive search over the 126 positive finite
 *      E4M3 block scales, scoring the E2M1 fake-quantization error e = quant(w) - w by
 *      e^T H_n e + 2 e^T (P_n w) (or sum_i Imp_i e_i^2) and keeping the argmin.
 *
 * Conventions shared by every entry point
 *   - Tensor pointers are DEVICE pointers, row-major and densely packed, owned by the caller.
 *     X, Xq and W must be 16-byte aligned (PyTorch allocations are); fp4 2-byte aligned.
 *     Inputs are never modified.  Outputs are fully overwritten (H, P and imp are read first
 *     only when beta != 0).
 *   - X is [rows, cin] (tokens x input channels, as a linear layer sees its input); W is
 *     [n_groups, cout, cin]; blocks run along cin in 16s (block n = channels 16n..16n+15).
 *   - Groups are MoE experts: rows [off[g], off[g+1]) of X belong to group g.  group_offsets is a
 *     device int64 array of n_groups+1 entries; pass NULL with n_groups == 1 for a dense layer
 *     (all rows).  Offsets must be non-decreasing with off[0] = 0 and off[n_groups] = rows; this is
 *     a caller contract (checking it would need a device read) and is not verified.
 *   - Calls are asynchronous on `stream` (a hipStream_t passed as void*; NULL = the null stream of
 *     the pointers' device).  The library never synchronizes the host, launches on the device that
 *     owns the pointers and restores the caller's current device.
 *   - Scratch memory, when an entry point needs it (accumulation partial sums and arrival
 *     counters), is a library-owned buffer per device, grown on demand in stream order from a
 *     device memory pool and kept between calls, so steady-state calls allocate nothing; calls
 *     on different streams are ordered through an event, so two calls never use it at once.
 *   - Return: LH_OK, or an error code with a message available from lh_last_error().  Argument
 *     checks run before any launch.  Faults inside kernels surface at the caller's next
 *     synchronization, as usual in HIP.  NaN or Inf in any input gives undefined results where an
 *     entry point does not say otherwise.
 *
 * Numerics
 *   - Accumulation reads bf16 or fp32 values exactly, multiplies them exactly (bf16) or in fp32
 *     (fp32 inputs), and sums in fp32 in a fixed order: results are bit-reproducible run to run.
 *   - The sweep returns the scale code and FP4 codes of the exact argmin of the float64 objective
 *     over all 126 candidates: a float32 pass scores each candidate that a proven lower bound does
 *     not rule out, with a rigorous error bound, and any block whose winner is not certain is
 *     re-scored in float64 with exact quantization.
 *
 * The entry points of a decode step (lh_rms_norm_quant, lh_matvec, lh_cache_write, lh_cache_read,
 * lh_paged_attention) run what the calibration leaves behind: 8-bit rows for quantized products,
 * products with the calibrated NVFP4 weights, and a key-value cache in the same formats.  Those around it
 * (lh_cache_extend, lh_rotary, lh_route, lh_moe, lh_adapter) grow the cache's sequences, turn queries and keys by
 * their positions, choose experts and run them, and add low-rank adapters to a product.  All of them keep
 * no state, allocate nothing and may be captured into a HIP graph.
 *
 * Citations are to the pages this library follows: "Add activation-aware local Hessian scale
 * calibration" (PR #1976), "add local hessian calibration" (PR #788), "Add WMSE weight scale
 * search calibration" (PR #2283) and "Add composable scale calibration to GPTQ" (PR #2004).
 */
#ifndef LH_H_
#define LH_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LH_VERSION 8

typedef enum {
  LH_OK = 0,
  LH_ERR_INVALID_ARGUMENT = 1, /* null pointer, bad size, host or foreign-device pointer */
  LH_ERR_UNSUPPORTED = 2,      /* unknown dtype or no gfx950 device */
  LH_ERR_HIP = 3               /* a HIP runtime call or launch failed */
} lh_status;

/* E4M3 is the type of lh_matvec's 8-bit rows alone; the other entry points take F32 and BF16.
 * The two sentinels widen the enum's value range to every 32-bit int: another value coming from a
 * caller is then a well-defined lh_dtype in C and C++, and every entry point rejects what it does
 * not take with LH_ERR_UNSUPPORTED.  They are not dtypes. */
typedef enum {
  LH_DTYPE_F32 = 0,
  LH_DTYPE_BF16 = 1,
  LH_DTYPE_E4M3 = 2,
  LH_DTYPE_RANGE_MIN_ = -2147483647 - 1,
  LH_DTYPE_RANGE_MAX_ = 2147483647
} lh_dtype;

/*
 * Per-block local Hessian and importance (PR #788, Overview / Changes: per-block Hessians
 * collected by forward hooks; PR #2283, How: the diagonal path accumulates x.square().sum(-1)).
 *
 *   H[g][n]   = beta * H[g][n]   + (1/T_g) * sum_{t in g} x_t[n] x_t[n]^T     (if H != NULL)
 *   imp[g][i] = beta * imp[g][i] + sum_{t in g} X[t,i]^2                      (if imp != NULL)
 *
 * X        [rows, cin], dtype x_dtype.
 * H        [n_groups, cin/16, 16, 16] fp32 or NULL.      imp  [n_groups, cin] fp32 or NULL.
 * At least one of H, imp must be non-NULL.  T_g = off[g+1]-off[g]; T_g == 0 makes the sum term 0.
 * beta lets a caller stream token batches (beta = 1 with sums, or a running mean).
 * Errors: INVALID_ARGUMENT for rows < 0, cin <= 0 or cin % 16, n_groups < 1, NULL X with rows > 0,
 * both outputs NULL, offsets NULL with n_groups > 1, non-device or mixed-device pointers.
 */
lh_status lh_accumulate(const void* X, lh_dtype x_dtype, int64_t rows, int64_t cin,
                        const int64_t* group_offsets, int64_t n_groups, float beta,
                        float* H, float* imp, void* stream);

/*
 * lh_accumulate for callers that cannot allocate device memory: code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation.  Same arguments, computation, results
 * (bit for bit) and errors as lh_accumulate, but the partial sums and arrival counters live in a
 * fixed array of 64 MiB per device that is part of the library's code object (each device the
 * library runs on holds it until the process ends), instead of the library's memory pool: the
 * call allocates nothing and records no event.  Every call on a device shares that device's
 * array, so calls that overlap on one device (other streams, graph replays in flight at once)
 * race and give wrong results; order them.  The arrival counters are cleared by a kernel at the
 * start of each call.  A problem that needs more scratch than the array holds (dense layers need
 * little; grouped rows need up to 2 * rows / R pieces x cin/64 slices x 4 KiB, R about
 * rows * cin / 262144 rows, between 64 and 1024) fails with INVALID_ARGUMENT before any launch.
 */
lh_status lh_accumulate_noalloc(const void* X, lh_dtype x_dtype, int64_t rows, int64_t cin,
                                const int64_t* group_offsets, int64_t n_groups, float beta,
                                float* H, float* imp, void* stream);

/*
 * Activation-aware Hessian and cross matrix (PR #1976, What does this PR do?):
 *   H[g][n] = beta*H[g][n] + X_q^T X_q / T_g,   P[g][n] = beta*P[g][n] + X_q^T (X_q - X) / T_g
 * per 16-channel block, over the rows of group g.  X and Xq are [rows, cin] of the same dtype.
 * P is formed from the difference D = X_q - X rounded once to fp32 (exact when X_q and X are
 * within a factor 2^15 of each other, as a fake-quant of X is; otherwise within 2^-24 of D) and
 * split exactly into bf16 pieces, never as the difference of two products.  H and P are both
 * required.  Errors as lh_accumulate.
 */
lh_status lh_accumulate_act_aware(const void* X, const void* Xq, lh_dtype dtype, int64_t rows,
                                  int64_t cin, const int64_t* group_offsets, int64_t n_groups,
                                  float beta, float* H, float* P, void* stream);

/*
 * The same H and P with X_q made from X inside the kernel, so the activations are read once
 * (PR #1976, What does this PR do?: X_q is the activation as the layer's NVFP4 input quantizer
 * emits it; the quantizer below is the NVFP4 recipe of PR #2004, What does this PR do?
 * (448-normalized), applied to activations per token):
 *   gX = fp32(x_amax[g] / (6*448)) per group;
 *   per row and 16-channel block: v = the E4M3 value (0 or one of the 126 positive finite values)
 *     nearest to max|x| / (6 gX), ties to the even code (so it saturates at 448 and a block whose
 *     max rounds to 0 becomes 0), s = fp32(v gX);
 *   x_q = sign(x) * E2M1(|x| / s) * s for each element (nearest of {0,0.5,1,1.5,2,3,4,6}, ties
 *     to the even grid index, saturating at 6; every rounding decision is the exact one), the
 *     product taken in fp32 and rounded to nearest-even bf16 when dtype is bf16.
 * x_amax [n_groups] fp32 device: the input quantizer's amax per group (>= 0 and finite; 0 gives
 * X_q = 0).  Other arguments, outputs and errors as lh_accumulate_act_aware, plus
 * INVALID_ARGUMENT for a NULL x_amax.
 */
lh_status lh_accumulate_act_aware_fq(const void* X, lh_dtype dtype, int64_t rows, int64_t cin,
                                     const int64_t* group_offsets, int64_t n_groups,
                                     const float* x_amax, float beta, float* H, float* P,
                                     void* stream);

/*
 * The activation fake-quant alone: writes X_q, the NVFP4 fake-quant of X that
 * lh_accumulate_act_aware_fq applies inside its kernel (same definition, same bits), for callers
 * that need the quantized activations themselves or feed lh_accumulate_act_aware (PR #1976, What
 * does this PR do?: X_q is what the layer's input quantizer emits).
 * X, Xq [rows, cin] of dtype (Xq is written, fully; it must not overlap X).  x_amax [n_groups]
 * fp32 device as in lh_accumulate_act_aware_fq; groups as everywhere (row r uses the amax of the
 * group that holds it).  Errors: INVALID_ARGUMENT for the shape checks of lh_accumulate, NULL
 * x_amax, NULL X or Xq with rows > 0, Xq == X, misaligned, non-device or mixed-device pointers.
 */
lh_status lh_activation_fake_quant(const void* X, lh_dtype dtype, int64_t rows, int64_t cin,
                                   const int64_t* group_offsets, int64_t n_groups, const float* x_amax,
                                   void* Xq, void* stream);

/*
 * Options of the weight-scale search, taken by the *_ex entry points (the others use the
 * defaults: 448-normalized scaling and all 126 candidates).
 *   scale_norm     the E4M3 value the global amax maps to: g = fp32(global_amax / (6 * scale_norm)).
 *                  448 is NVFP4's scaling, 256 that of its "4/6" variant ("Add composable scale
 *                  calibration to GPTQ", What does this PR do?: 448-normalized scaling, 4/6 uses
 *                  256).  It must be one of the 126 positive finite E4M3 values.
 *   n_multipliers  0: the FP8 scale sweep over all 126 candidates.  1..128: the amax-multiplier
 *                  search ("add local hessian calibration", Changes: configurable step size and
 *                  multipliers for the amax search): a block of amax a = max_i |w_i| takes only the
 *                  candidates whose code is the positive finite E4M3 value nearest to the exact
 *                  a * m / (6 g) for one of the multipliers m (ties to the even code, saturating
 *                  at 448 and at 2^-9), and keeps the lowest-loss one of those (lowest code on
 *                  ties, which is the first in an ascending grid).
 *   multipliers    HOST array of n_multipliers positive finite values, any order (a grid
 *                  start + j * step is the usual choice), read during the call.
 */
typedef struct {
  float scale_norm;
  int32_t n_multipliers;
  const float* multipliers;
} lh_sweep_options;

/*
 * Exhaustive FP8 block-scale sweep with the local-Hessian objective (PR #788, review: block loss
 * cnb,nbd,cnd->cn; PR #1976, review: dw = quant(w) - w, coupling term 2 dw^T (P W0) with
 * P.W0 = nbd,cnd->cnb, best_loss = inf so negative losses are handled; PR #2283, How: the 126
 * candidate scales; PR #2004: NVFP4 scaling is 448-normalized).
 *
 * For every block (g, c, n) with weights w = W[g][c][16n..16n+15]:
 *   g_g  = fp32(global_amax[g] / (6*448))
 *   s_k  = fp32(v_k * g_g), v_k the E4M3 value of byte k, k = 0x01..0x7E (126 candidates)
 *   q_k  = E2M1 fake-quant of w with scale s_k: each |w_i|/s_k (exact quotient) is rounded to the
 *          nearest of {0,0.5,1,1.5,2,3,4,6}, ties to the even grid index, saturating at 6
 *   e_k  = q_k - w,  L_k = e_k^T H_n e_k + 2 e_k^T (P_n w)      (P == NULL: no cross term)
 *   k*   = argmin_k L_k, lowest code on ties.
 * A block whose H_n has zero trace (no activation energy) is scored with H = I and no cross term.
 *
 * W           [n_groups, cout, cin] dtype w_dtype.
 * global_amax [n_groups] fp32 device, >= 0 and finite (normally max |W_g|, see lh_absmax).
 * H, P        [n_groups, cin/16, 16, 16] fp32 (P may be NULL).
 * scale_code  [n_groups, cout, cin/16] uint8: the E4M3 byte k* (0x01..0x7E).
 * fp4         [n_groups, cout, cin/2] uint8 or NULL: nibble = (w < 0) << 3 | grid index,
 *             element 2j in the low nibble of byte j.
 * best_loss   [n_groups, cout, cin/16] fp32 or NULL: L_{k*} (may be negative with P).
 * Errors: INVALID_ARGUMENT for n_groups outside [1, 65535], cout outside [0, 2097120], cin <= 0
 * or cin % 16, NULL required pointers, non-device or mixed-device pointers.
 */
lh_status lh_scale_sweep(const void* W, lh_dtype w_dtype, int64_t n_groups, int64_t cout,
                         int64_t cin, const float* global_amax, const float* H, const float* P,
                         uint8_t* scale_code, uint8_t* fp4, float* best_loss, void* stream);

/*
 * lh_scale_sweep with options (see lh_sweep_options; NULL = the defaults, identical to
 * lh_scale_sweep).  Errors as lh_scale_sweep, plus INVALID_ARGUMENT for a scale_norm that is not
 * a positive finite E4M3 value, n_multipliers outside [0, 128], a NULL multipliers array with
 * n_multipliers > 0, or a multiplier that is not positive and finite.
 */
lh_status lh_scale_sweep_ex(const void* W, lh_dtype w_dtype, int64_t n_groups, int64_t cout,
                            int64_t cin, const float* global_amax, const float* H, const float* P,
                            const lh_sweep_options* options, uint8_t* scale_code, uint8_t* fp4,
                            float* best_loss, void* stream);

/*
 * Accumulation and sweep of grouped rows (MoE experts) in one launch, the Hessians kept on chip:
 * per expert, the per-block Hessian of its routed rows and the weight-scale search of its weight
 * matrix against it, without writing H to memory ("[2/3] Speed up layerwise GPTQ on MoE models",
 * embedded #2840 text: one Hessian per expert and projection, over exactly the tokens routed to
 * it; its size per MoE layer is what makes such calibration memory-bound).
 *   H[g][n] = (1/T_g) sum_{t in g} x_t[n] x_t[n]^T   (as lh_accumulate, beta = 0)
 *   then the search of lh_scale_sweep_ex on W[g] with H[g], P = NULL and `options`.
 * For n_groups >= 2 each H is summed in the order lh_accumulate's grouped path uses, so codes,
 * nibbles and losses are bit-identical to lh_accumulate followed by lh_scale_sweep_ex; with one
 * group lh_accumulate takes its dense path, whose order differs (results agree within its
 * rounding).  A group without rows gets H = 0, i.e. the plain weight-MSE search.
 * X [rows, cin] and W [n_groups, cout, cin] of dtype; group_offsets as everywhere (NULL with one
 * group); global_amax [n_groups]; outputs as lh_scale_sweep.
 * Errors: those of lh_accumulate and lh_scale_sweep_ex, plus INVALID_ARGUMENT for cout > 8192.
 */
lh_status lh_accumulate_sweep(const void* X, const void* W, lh_dtype dtype, int64_t rows, int64_t cin,
                              const int64_t* group_offsets, int64_t n_groups, int64_t cout,
                              const float* global_amax, const lh_sweep_options* options,
                              uint8_t* scale_code, uint8_t* fp4, float* best_loss, void* stream);

/*
 * Same sweep scored by the importance-weighted error L_k = sum_i imp[g][16n+i] * e_{k,i}^2
 * (PR #2283, What / How: H replaced by diag(Imp), einsum cnb,nb->cn, no diag_embed and no
 * matmul on the hot path).  A block whose importance sums to zero uses Imp = 1.
 * imp [n_groups, cin] fp32.  Other arguments and errors as lh_scale_sweep.
 */
lh_status lh_scale_sweep_diag(const void* W, lh_dtype w_dtype, int64_t n_groups, int64_t cout,
                              int64_t cin, const float* global_amax, const float* imp,
                              uint8_t* scale_code, uint8_t* fp4, float* best_loss, void* stream);

/*
 * Same sweep scored by the plain squared error L_k = sum_i e_{k,i}^2 (H = I, no activations): the
 * weight-only "mse" calibration that "Add WMSE weight scale search calibration" runs as its control
 * arm (verification: mse control; Ablation table: mse rows).  Equal to lh_scale_sweep_diag with
 * every importance 1 and to lh_scale_sweep with H_n = I, P = NULL.  Arguments and errors as
 * lh_scale_sweep_diag without imp.
 */
lh_status lh_scale_sweep_mse(const void* W, lh_dtype w_dtype, int64_t n_groups, int64_t cout,
                             int64_t cin, const float* global_amax, uint8_t* scale_code, uint8_t* fp4,
                             float* best_loss, void* stream);

/*
 * lh_scale_sweep_diag with options (see lh_sweep_options); imp may be NULL for the plain-MSE
 * objective of lh_scale_sweep_mse.  Errors as lh_scale_sweep_ex.
 */
lh_status lh_scale_sweep_diag_ex(const void* W, lh_dtype w_dtype, int64_t n_groups, int64_t cout,
                                 int64_t cin, const float* global_amax, const float* imp,
                                 const lh_sweep_options* options, uint8_t* scale_code, uint8_t* fp4,
                                 float* best_loss, void* stream);

/*
 * Fake-quantized weights and per-block amax from a sweep's result: the calibrated quantizer state
 * ("Add WMSE weight scale search calibration": the shared-path check fingerprints the quantizers'
 * amax and scales and the final fake-quantized weights):
 *   s_k  = fp32(v_k * fp32(global_amax[g] / (6*448)))  for the block's code k (the sweep's scale)
 *   Wq[g][c][16n+j] = sign * E2M1 value of nibble j * s_k, rounded to fp32 and, for a bf16
 *                     out_dtype, to nearest-even bf16 (a negative value that quantized to 0
 *                     gives -0)
 *   block_amax[g][c][n] = fp32(6 * s_k)
 * scale_code [n_groups, cout, cin/16] u8 and fp4 [n_groups, cout, cin/2] u8 as lh_scale_sweep
 * writes them (codes 0x01..0x7E); global_amax [n_groups] fp32; Wq [n_groups, cout, cin] in
 * out_dtype or NULL (16-byte aligned); block_amax [n_groups, cout, cin/16] fp32 or NULL.
 * Errors: INVALID_ARGUMENT for shapes as lh_scale_sweep, NULL scale_code or global_amax, both
 * outputs NULL, NULL fp4 with Wq, misaligned pointers, non-device or mixed-device pointers.
 */
lh_status lh_dequantize(const uint8_t* scale_code, const uint8_t* fp4, lh_dtype out_dtype,
                        int64_t n_groups, int64_t cout, int64_t cin, const float* global_amax,
                        void* Wq, float* block_amax, void* stream);

/*
 * lh_dequantize for codes a sweep chose under scale_norm (see lh_sweep_options):
 * s_k = fp32(v_k * fp32(global_amax[g] / (6 * scale_norm))).  Errors as lh_dequantize, plus
 * INVALID_ARGUMENT for a scale_norm that is not a positive finite E4M3 value.
 */
lh_status lh_dequantize_ex(const uint8_t* scale_code, const uint8_t* fp4, lh_dtype out_dtype,
                           int64_t n_groups, int64_t cout, int64_t cin, const float* global_amax,
                           float scale_norm, void* Wq, float* block_amax, void* stream);

/*
 * Per-group absolute maximum amax_out[g] = max |W_g| over elems_per_group elements: the max
 * calibration that fixes the weight's global amax before the search (PR #788, Sequence diagram:
 * initial max_calibrate).  W is [n_groups, elems_per_group]; an empty group gives 0.
 * Errors: INVALID_ARGUMENT for n_groups < 1, elems_per_group < 0, NULL pointers, non-device or
 * mixed-device pointers.
 */
lh_status lh_absmax(const void* W, lh_dtype w_dtype, int64_t n_groups, int64_t elems_per_group,
                    float* amax_out, void* stream);

/*
 * Root-mean-square norm of a residual stream, with the residual's addition and 8-bit output: the
 * input of a quantized product.
 *   h[t,i] = X[t,i] + R[t,i] rounded to dtype          (h = X when R is NULL)
 *   y[t,i] = h[t,i] / sqrt(mean_i h[t,i]^2 + eps) * gamma[i]                        (in fp32)
 *   per row (group = 0) or per 128 channels of a row (group = 128, the last run may be shorter):
 *     scale = max|y| * fp32(1/448),  q = the E4M3 value nearest to y / scale, the exact quotient of the
 *     two fp32 numbers, ties to the even code (0 where scale = 0)
 * X, R [rows, cin] of dtype; gamma [cin] of dtype; eps >= 0 and finite.  summed [rows, cin] of dtype
 * receives h; it is required with R, must be NULL without, and may be X or R itself.
 * q [rows, cin] E4M3 bytes; q_scale [rows] or [rows, ceil(cin/128)] fp32.  All 16-byte aligned
 * but q_scale.  Sums are fp32; a row of zeros (with eps = 0, too) gives q = 0.
 * A NaN in a row of h makes all scales of the row NaN, an infinity the scale of its run (the other
 * channels become 0); one in gamma makes its run's scale NaN or infinite.  q is 0 where the scale is
 * not finite.  The sum of squares keeps fp32's range: a row over it (elements near 2^60) gives zeros, and
 * with eps = 0 one under it (near 2^-60) loses bits and then gives zeros.
 * Errors: INVALID_ARGUMENT for rows < 0 or more than a launch takes (2^26-4 rows of up to 1024 bf16 or 512
 * fp32 channels, 2^24-1 of up to 16384 or 8192, 2^22-1 longer ones), cin <= 0 or cin % 16 or cin > 2^24, a group
 * other than 0 and 128, a bad eps, R without summed or the reverse, NULL required pointers,
 * misaligned, non-device or mixed-device pointers.
 */
lh_status lh_rms_norm_quant(const void* X, const void* R, lh_dtype dtype, int64_t rows, int64_t cin,
                            const void* gamma, float eps, int64_t group, void* summed, uint8_t* q,
                            float* q_scale, void* stream);

/*
 * Products of a few rows with NVFP4 weights as lh_scale_sweep writes them, dense or per expert (a
 * decode step's tokens, drafted tokens, small batches):
 *   Y[t,c] = sum_k Wq[g][c][k] x[t,k] for the rows t of group g,
 *   Wq[g][c][k] = E2M1(nibble) * v_code * g_g,  g_g = fp32(global_amax[g] / (6 * scale_norm)),
 * that is lh_dequantize_ex's weights before their rounding.  Products are exact (an fp32 element under
 * 2^-110 enters to within 2^-133) and sums fp32, in a fixed order; g_g multiplies the sum, which is rounded once to Y's type.
 * Infinities and NaN in a row of X give what the row's sums of products are, and change no other row.
 * scale_code [n_groups, cout, cin/16], fp4 [n_groups, cout, cin/2] (8-byte aligned), global_amax
 * [n_groups], scale_norm as in lh_sweep_options.
 * X [rows, cin], 16-byte aligned: F32, BF16, or E4M3 bytes with x_scale fp32, one per row (x_group = 0,
 * [rows]) or one per 128 channels (x_group = 128, [rows, ceil(cin/128)]), as lh_rms_norm_quant
 * writes them; x_scale is NULL and x_group 0 for the other types.
 * Y [rows, cout]: F32 for F32 rows, BF16 otherwise.
 * Groups as everywhere; a group without rows is skipped.  Any number of rows works; the weights are
 * read again for every 64 rows (32 of fp32), with several groups for every 16 rows of a group (4 of fp32, and
 * where 4 * rows <= n_groups).
 * Errors: INVALID_ARGUMENT for the shapes of lh_accumulate and lh_scale_sweep, cin > 2^24, a launch of
 * 2^32 or more work-items, scale_norm that is not a positive finite E4M3 value, x_scale or x_group
 * that do not fit the type, NULL required pointers, misaligned, non-device or mixed-device pointers.
 */
lh_status lh_matvec(const void* X, lh_dtype x_dtype, const float* x_scale, int64_t x_group, int64_t rows,
                    int64_t cin, const int64_t* group_offsets, int64_t n_groups, int64_t cout,
                    const uint8_t* scale_code, const uint8_t* fp4, const float* global_amax,
                    float scale_norm, void* Y, void* stream);

/*
 * A paged key-value cache in one of two formats, owned by the caller.  Pages hold page_size tokens
 * of every key-value head, head by head; a token's slot is page * page_size + its place in the page.
 *   LH_CACHE_E4M3   k, v [n_pages, n_heads, page_size, head_dim] bytes; k_scale, v_scale NULL.
 *                   value = fp32(E4M3 * s), s = fp32(amax[head] * fp32(1/448))
 *   LH_CACHE_FP4    k, v [n_pages, n_heads, page_size, head_dim/2], element 2j in the low nibble of
 *                   byte j; k_scale, v_scale [n_pages, n_heads, page_size, head_dim/16] E4M3 bytes.
 *                   value = fp32(E2M1 * s), s = fp32(v * g), g = fp32(amax[head] * fp32(1/2688)):
 *                   the NVFP4 rule of lh_activation_fake_quant along head_dim, the head as the
 *                   group, with g a product by the rounded reciprocal (GPU tensor libraries
 *                   evaluate amax / 2688 that way; codes made there by this rule are the same)
 * k_amax, v_amax [n_heads] fp32 device: the calibrated largest magnitude per head (>= 0, finite;
 * see lh_absmax); larger elements and infinities saturate.  A NaN is held as a NaN code (E4M3) or as the
 * NaN scale of its 16 elements (NVFP4) and reads back as NaN.  Codes are 16-byte, scales 4-byte aligned.
 */
typedef enum {
  LH_CACHE_E4M3 = 0,
  LH_CACHE_FP4 = 1,
  LH_CACHE_RANGE_MIN_ = -2147483647 - 1, /* not formats; see lh_dtype */
  LH_CACHE_RANGE_MAX_ = 2147483647
} lh_cache_format;

typedef struct {
  lh_cache_format format;
  int64_t n_pages, page_size, n_heads, head_dim;
  uint8_t *k, *v, *k_scale, *v_scale;
  const float *k_amax, *v_amax;
} lh_cache;

/*
 * Quantizes new tokens' keys and values and writes them to their slots.  Every rounding is that of
 * the exact quotient, ties to the even code.
 * cache: HOST struct, read during the call.  K, V: element (t, head, i) at t * stride + head *
 * head_dim + i, strides in elements (at least n_heads * head_dim), so they may be parts of a wider
 * projection's rows; 16-byte aligned, strides multiples of 16 bytes.
 * slots [tokens] int64 device; a slot outside [0, n_pages * page_size) is skipped.  A slot named
 * twice in one call is left with unspecified contents (its blocks' codes and scales are written apart, so
 * they may be of either token, and a block may mix them); all other slots are as asked.
 * Errors: UNSUPPORTED for an unknown dtype or format; INVALID_ARGUMENT for n_pages, page_size,
 * n_heads or head_dim < 1, head_dim % 16, head_dim > 65536, n_heads * head_dim over 2^27,
 * page_size over 2^31-1, over 2^40 slots, a launch of 2^32 or more work-items (one for 16 elements),
 * tokens < 0, bad strides, NULL required pointers or block scales that do not fit the format, misaligned, non-device or mixed-device pointers.
 */
lh_status lh_cache_write(const lh_cache* cache, const void* K, int64_t k_stride, const void* V,
                         int64_t v_stride, lh_dtype dtype, int64_t tokens, const int64_t* slots,
                         void* stream);

/*
 * Reads slots back: K, V [tokens, n_heads, head_dim] of dtype (fp32 value, rounded to nearest-even
 * bf16 for BF16), dense, 16-byte aligned.  A slot outside the cache reads as zeros.  Errors as
 * lh_cache_write.
 */
lh_status lh_cache_read(const lh_cache* cache, const int64_t* slots, int64_t tokens, lh_dtype dtype,
                        void* K, void* V, void* stream);

/*
 * Attention of one new token per sequence over the cache (its own key and value already written):
 *   O[b,h] = sum_t p_t V[t, h/share],  p = softmax_t(scale * Q[b,h] . K[t, h/share]),
 *   t < lengths[b], share = n_q_heads / n_heads; token t of sequence b is in page
 *   block_table[b][t / page_size] at place t % page_size.
 * Q: element (b, h, i) at b * q_stride + h * head_dim + i; O [batch, n_q_heads, head_dim] dense, both
 * of dtype, 16-byte aligned, q_stride a multiple of 16 bytes.  block_table [batch, max_pages] and
 * lengths [batch] int32 device.  A length is taken as between 0 and max_pages * page_size; a
 * sequence of length 0 gives zeros.  Entries of the table past a sequence's last page are not
 * read; a page outside the cache is read as page 0.  head_dim is 64, 128 or 256.
 * K and V enter exactly; q is held to 2^-39 of its head's largest element (bf16: exactly from 2^-31 of it
 * on; fp32: to 2^-22 of each element too), p to fp16 (fp32: two fp16 pieces), and maxima, sums and outputs
 * are fp32.  A NaN or an infinity in a head's q gives that head NaN, a NaN key or value of the sequence's
 * tokens the outputs that depend on it.
 * Two calls with the same arguments give the same bits; where a sequence is cut depends on all
 * lengths of the batch, so beside other sequences its last bits may differ.
 * workspace: device memory of at least lh_paged_attention_workspace bytes (16-byte aligned; NULL if
 * that is 0) that no other call uses until this one has run.
 * Errors: UNSUPPORTED for an unknown dtype or format, or another head_dim; INVALID_ARGUMENT as
 * lh_cache_write, n_q_heads not a positive multiple of n_heads, batch < 0, max_pages < 0,
 * max_pages * page_size over 2^31-4096, a launch of 2^32 or more work-items (256 for a sequence's 16 query
 * heads of a key-value head), a scale that is not finite, a short workspace.
 */
lh_status lh_paged_attention(const lh_cache* cache, const void* Q, int64_t q_stride, lh_dtype dtype,
                             int64_t batch, int64_t n_q_heads, const int32_t* block_table,
                             int64_t max_pages, const int32_t* lengths, float scale, void* O,
                             void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Bytes of workspace that lh_paged_attention needs for these sizes (a host computation; 0 for
 * arguments that it refuses).
 */
int64_t lh_paged_attention_workspace(const lh_cache* cache, int64_t batch, int64_t n_q_heads,
                                     int64_t max_pages);

/*
 * Growth of a paged cache's sequences by one step's tokens: block tables, lengths and free pages on the
 * device, and for each row of new tokens its slot (for lh_cache_write), position (for lh_rotary) and sequence.
 * With request b of length l = lengths[b] (taken as between 0 and max_pages * page_size), n = new_tokens[b]
 * (NULL: 1 for every request), up(x) = x / page_size rounded up, and the stack free_pages[0 .. c), c =
 * free_count[0] (taken as between 0 and capacity), its top at c - 1:
 *   n < 0  takes back the last min(-n, l) tokens: the request's length becomes l' = max(l + n, 0), and the pages
 *          up(l') .. up(l) - 1 of its table go on the stack, in the order of requests and pages (those past
 *          `capacity` are lost).  All of them are on the stack before any page is taken, the top then at a - 1.
 *   n > 0  asks for n tokens, rows offsets[b] .. offsets[b] + n - 1, and needs up(l + n) - up(l) pages.  It is
 *          granted if l + n <= max_pages * page_size, its rows end by max_tokens, and either it needs no page or the
 *          needs of all requests up to it that meet those two conditions come to at most a: first come, first
 *          served.  It then takes its pages from the top, the first for its lowest tokens, and its length
 *          becomes l + n.  Otherwise its length and pages stay as they are.
 * block_table [batch, max_pages] int32: entries of new pages are written, all others stay as they are.
 * free_pages [capacity] int32: c .. c + the pages given back are written; new_count[0] is what is then held.
 * slots [max_tokens] int64, positions and sequence [max_tokens] int32: for each row the token's slot and position (both
 * -1 where the request was not granted) and its request; behind the last row of the batch all three are -1.
 * offsets [batch + 1] int32: the first row of each request, whether granted or not, at most max_tokens.
 * new_lengths may be lengths and new_count free_count, for an update in place; with others in their place, two
 * calls with the same arguments do the same.  No other arguments may overlap.
 * Page numbers are handed on as they are.  workspace: device memory of at least lh_cache_extend_workspace bytes (16-byte
 * aligned; NULL if that is 0) that no other call uses until this one has run.
 * Errors: INVALID_ARGUMENT for batch outside [0, 2^28-1], page_size < 1, max_pages < 0, max_pages * page_size over
 * 2^31-4096, max_tokens or capacity outside [0, 2^31-1], NULL required pointers, a short workspace, misaligned,
 * non-device or mixed-device pointers.
 */
lh_status lh_cache_extend(int32_t* block_table, int64_t batch, int64_t max_pages, int64_t page_size,
                          const int32_t* lengths, const int32_t* new_tokens, int32_t* free_pages,
                          int64_t capacity, const int32_t* free_count, int64_t max_tokens, int64_t* slots,
                          int32_t* positions, int32_t* sequence, int32_t* offsets, int32_t* new_lengths,
                          int32_t* new_count, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that lh_cache_extend needs for these sizes (a host computation; 0 for ones outside the ranges above). */
int64_t lh_cache_extend_workspace(int64_t batch, int64_t max_tokens);

/*
 * Angles per position of rotary positions, f_j = theta^(-2j / rot_dim) for j < rot_dim / 2, scaled for contexts
 * longer than the one they were trained for; computed in 64 bits on the host and rounded once to fp32:
 *   PLAIN   f_j
 *   LINEAR  f_j / factor (positions interpolated)
 *   BASE    f_j with theta * factor^(rot_dim / (rot_dim - 2)) for theta
 *   PARTS   f_j (k + (1 - k) / factor), k = (t - low_turns) / (high_turns - low_turns) clamped to [0, 1], t =
 *           original_context * f_j / (2 pi) the turns over the trained context: fast angles stay, slow ones are interpolated
 * frequencies [rot_dim / 2] and scale: HOST memory; *scale is what lh_rotary's scale is meant to be, 0.1 ln(factor) + 1 for
 * PARTS and 1 otherwise.
 * Errors: UNSUPPORTED for an unknown scaling; INVALID_ARGUMENT for theta not positive and finite, rot_dim odd or
 * outside [2, 65536] (below 4 with BASE), factor < 1 or not finite (but with PLAIN), original_context < 1 or not 0 <=
 * low_turns < high_turns < infinity with PARTS, NULL pointers.
 */
typedef enum {
  LH_ROTARY_PLAIN = 0,
  LH_ROTARY_LINEAR = 1,
  LH_ROTARY_BASE = 2,
  LH_ROTARY_PARTS = 3,
  LH_ROTARY_RANGE_MIN_ = -2147483647 - 1, /* not scalings; see lh_dtype */
  LH_ROTARY_RANGE_MAX_ = 2147483647
} lh_rotary_scaling;

lh_status lh_rotary_frequencies(double theta, int64_t rot_dim, lh_rotary_scaling scaling, double factor,
                                int64_t original_context, double low_turns, double high_turns,
                                float* frequencies, float* scale);

/*
 * Rotary positions: the pairs of the first rot_dim elements of every head of Q and K, turned by their token's angles
 *   (a, b) -> scale * (a cos w - b sin w, a sin w + b cos w),   w = positions[t] * frequencies[j]
 * for pair j < rot_dim / 2: elements (j, j + rot_dim / 2), or (2j, 2j + 1) if interleaved.  With `inverse`, -w for w, which is
 * the transpose: it takes a gradient back through the rotation.  Other elements are copied.  A token of negative position
 * is copied as it is, scale or not (a row without a token, see lh_cache_extend).
 * Q: element (t, h, i) at t * q_stride + h * head_dim + i, t < tokens; K and the outputs in the same way, so each may be part of
 * wider rows.  Q_out may be Q and K_out K (with equal strides), for a turn in place; otherwise they overlap no input.
 * All of dtype, 16-byte aligned, strides multiples of 16 bytes.  n_k_heads may be 0 (K and K_out NULL).
 * positions [tokens] int32, frequencies [rot_dim / 2] fp32 (see lh_rotary_frequencies; magnitudes up to 2^16), both device.
 * The angle is the exact product, reduced in 64-bit arithmetic (positions up to 2^31-1 lose nothing); sine and cosine
 * are fp32 to within 2^-23, products and sums fp32, rounded once to dtype.
 * Errors: UNSUPPORTED for an unknown dtype; INVALID_ARGUMENT for tokens outside [0, 2^31-1], head_dim < 1, over 65536 or
 * not a multiple of 16, rot_dim odd or outside [2, head_dim], n_q_heads < 1, n_k_heads < 0, heads * head_dim over
 * 2^27, a scale that is not finite, bad strides, a launch of 2^32 or more work-items (at most one for 2 elements), NULL
 * required pointers, misaligned, non-device or mixed-device pointers.
 */
lh_status lh_rotary(const void* Q, int64_t q_stride, int64_t n_q_heads, const void* K, int64_t k_stride,
                    int64_t n_k_heads, lh_dtype dtype, int64_t tokens, int64_t head_dim, int64_t rot_dim,
                    const int32_t* positions, const float* frequencies, int32_t interleaved,
                    int32_t inverse, float scale, void* Q_out, int64_t q_out_stride, void* K_out,
                    int64_t k_out_stride, void* stream);

/*
 * The choice of experts for each token: ids[t] are the topk largest of logits[t], in descending order, equal ones by
 * ascending index, and weights[t] their softmax weights times `scale`:
 *   p_e = exp(logits[t,e] - m) / sum over all experts, or over the chosen ones if renormalize;  m the largest logit
 * A logit of -infinity or NaN is never chosen and has weight 0; where fewer than topk are left, ids are -1 and weights 0
 * (lh_moe skips those).  Where m is +infinity, the logits equal to it count as 1 and all others as 0.
 * logits [tokens, n_experts] of dtype; ids [tokens, topk] int32, weights [tokens, topk] fp32.  Sums are fp32.
 * Errors: UNSUPPORTED for an unknown dtype; INVALID_ARGUMENT for tokens outside [0, 2^31-1], n_experts outside [1, 4096], topk
 * outside [1, 64] or over n_experts, a scale that is not finite, a launch of 2^32 or more work-items (64 a token), NULL required
 * pointers, non-device or mixed-device pointers.
 */
lh_status lh_route(const void* logits, lh_dtype dtype, int64_t tokens, int64_t n_experts, int64_t topk,
                   int32_t renormalize, float scale, int32_t* ids, float* weights, void* stream);

/*
 * A mixture-of-experts layer on NVFP4 expert weights as lh_scale_sweep writes them, for a few tokens:
 *   Y[t] = sum_j weights[t,j] * D_e (silu(G_e x_t) * U_e x_t),   e = ids[t,j],   silu(g) = g / (1 + exp(-g))
 * G_e and U_e are the first and the last `inner` rows of expert e's gate_up matrix, D_e its down matrix; a choice outside
 * [0, n_experts) adds nothing, a token without choices gives zeros, one chosen twice has the sum of its weights.
 * gate_up_code [n_experts, 2 * inner, hidden/16], gate_up_fp4 [n_experts, 2 * inner, hidden/2], down_code [n_experts, hidden,
 * inner/16], down_fp4 [n_experts, hidden, inner/2] (both fp4 8-byte aligned), amax [n_experts] each, scale_norm as in
 * lh_sweep_options.  ids and weights [tokens, topk] int32 and fp32, as lh_route gives them.
 * X [tokens, hidden], x_scale and x_group as in lh_matvec; Y [tokens, hidden] F32 for F32 rows, BF16 otherwise.
 * Weights enter exactly, and so do E4M3 rows and their scales.  Of each 128 elements of other rows with the largest magnitude m, BF16
 * ones enter exactly from 2^-31 m on and to within 2^-39 m below, F32 ones to within 2^-23 of themselves and 2^-39 m.  What comes between the two
 * products is held to 2^-11 of itself (F32 rows: 2^-23) and 2^-39 of the largest of its 128; where exp(-g) is over 2^224 (g under -155) its silu
 * counts as 0.  Sums are fp32, in a fixed order, of products that the matrix's global scale amax / (6 * scale_norm) multiplies afterwards; the
 * routing weights multiply the rows of the second product, and Y is rounded once.  Infinities and NaN in a row give what the formula
 * gives in that row's Y and change no other row.
 * Any number of tokens works; the weights of an expert are read again for every 64 tokens, and among those for every 32 rows of it (16
 * with up to 16 tokens; up to 64 of rows that are not F32, where tokens > 16, tokens * topk > 4 * n_experts, and hidden and inner >= 128).
 * workspace: device memory of at least lh_moe_workspace bytes (16-byte aligned) that no other call uses until this one has run.
 * Errors: UNSUPPORTED for an unknown dtype; INVALID_ARGUMENT for tokens outside [0, 4194240], hidden or inner < 1, over 2^24
 * or not multiples of 16, hidden * inner over 2^32, n_experts outside [1, 4096], topk outside [1, 64], scale_norm that is not a
 * positive finite E4M3 value, x_scale or x_group that do not fit the type, a launch of 2^32 or more work-items, NULL required
 * pointers, a short workspace, misaligned, non-device or mixed-device pointers.
 */
lh_status lh_moe(const void* X, lh_dtype x_dtype, const float* x_scale, int64_t x_group, int64_t tokens,
                 int64_t hidden, int64_t inner, int64_t n_experts, int64_t topk, const int32_t* ids,
                 const float* weights, const uint8_t* gate_up_code, const uint8_t* gate_up_fp4,
                 const float* gate_up_amax, const uint8_t* down_code, const uint8_t* down_fp4,
                 const float* down_amax, float scale_norm, void* Y, void* workspace, int64_t workspace_bytes,
                 void* stream);

/* Bytes of workspace that lh_moe needs for these sizes (a host computation; 0 for types and sizes outside the ranges above). */
int64_t lh_moe_workspace(lh_dtype x_dtype, int64_t tokens, int64_t hidden, int64_t inner, int64_t n_experts,
                         int64_t topk);

/*
 * Low-rank adapters of many requests at once, beside a projection that they share (lh_matvec's, of the same rows):
 *   Y[t] = base[t] + scaling[a] * B_a (A_a x_t),   a = index[t];   Y[t] = base[t] where a is outside [0, n_adapters)
 * A [n_adapters, rank, cin] and B [n_adapters, cout, rank] of w_dtype (F32 or BF16); ranks [n_adapters] int32 or NULL: adapter a has
 * ranks[a] (taken as between 0 and rank) rows of A and columns of B, and what is stored past those does not count, whatever it is;
 * NULL: all have `rank`.  scaling [n_adapters] fp32 or NULL (1).  index [rows] int32.
 * X [rows, cin], x_scale and x_group as in lh_matvec; base and Y [rows, cout], F32 for F32 rows, BF16 otherwise; Y may be base.
 * Products of BF16 weights are exact (fp32 elements as in lh_matvec), those of F32 weights fp32 (E4M3 elements are then multiplied by
 * their scale first); A_a x_t is held to 2^-16 of itself with BF16 weights and Y, otherwise to 2^-24; sums are fp32, in a
 * fixed order, and Y is rounded once.  Infinities and NaN in a row change no other row.  (Infinite weights may give NaN where the formula gives
 * an infinity: they meet rows and A_a x_t in pieces, some of them 0.)
 * The weights of an adapter are read again for every 64 rows, and among those A for every 16 rows of it, and B for every 32 where rank
 * is over 64 and every 16 where it is over 128.
 * workspace: device memory of at least lh_adapter_workspace bytes (16-byte aligned) that no other call uses until this one has run.
 * Errors: UNSUPPORTED for an unknown dtype; INVALID_ARGUMENT for rows outside [0, 4194240], cin <= 0, over 2^24 or not a multiple of
 * 16, cout outside [0, 2^24], n_adapters outside [1, 4096], rank outside [8, 256] or not a multiple of 8, x_scale or x_group that do
 * not fit the type, a launch of 2^32 or more work-items, NULL required pointers, a short workspace, pointers not 16-byte
 * aligned (X, A, B, base, Y), non-device or mixed-device pointers.
 */
lh_status lh_adapter(const void* X, lh_dtype x_dtype, const float* x_scale, int64_t x_group, int64_t rows,
                     int64_t cin, int64_t cout, int64_t n_adapters, int64_t rank, const void* A, const void* B,
                     lh_dtype w_dtype, const int32_t* index, const float* scaling, const int32_t* ranks,
                     const void* base, void* Y, void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace that lh_adapter needs for these sizes (a host computation; 0 for ones outside the ranges above). */
int64_t lh_adapter_workspace(int64_t rows, int64_t cin, int64_t n_adapters, int64_t rank);

/* Message of the last error on the calling thread ("" if none); valid until its next call. */
const char* lh_last_error(void);

/* LH_VERSION of the built library. */
int lh_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LH_H_ */
