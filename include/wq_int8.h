/*
 * wq_int8.h -- C ABI of libwq: 8-bit serving products (W8A8).  INT8 weights
 * (the per-channel artifact of wq_quantize_w8) times INT8 activations with one
 * scale per token, for one weight matrix and for one matrix per expert, and
 * the quantizer that makes the activations.
 *
 * Sources: "LLM Quantization: GPTQ, AWQ, SmoothQuant, FP8, KV Cache (7/10)",
 * SmoothQuant section (W8A8: weights and activations in INT8, the activation's
 * large channels divided out and folded into the weights) and Granularity
 * (per-channel weights, per-token activations); "Quantization Algorithms"
 * study notes 1.8 (symmetric INT8 uses [-127, 127]).
 *
 * The conventions of wq.h hold here: device pointers owned by the caller,
 * dense row-major matrices, asynchronous calls on `stream`, argument errors
 * returned before anything is launched, conditions found on the device in the
 * status word, no device memory allocated, no other library called.  Every
 * entry point belongs to the current device; none needs a workspace, so calls
 * on several streams and replays of captured graphs share nothing but the
 * buffers that the caller gives them.
 */
#ifndef WQ_INT8_H_
#define WQ_INT8_H_

#include "wq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest d_in of these products: 128 * 128 * d_in stays below 2^31, so that
 * an INT32 sum never wraps whatever the codes are. */
#define WQ_INT8_MAX_D_IN 131040

/* Largest number of experts of wq_linear_w8a8_grouped. */
#define WQ_INT8_MAX_EXPERTS 1024

/* Status word bit: wq_quantize_tokens met a row index outside [0, T), or
 * wq_linear_w8a8_grouped offsets that decrease or leave [0, R].
 * wq_get_device_error reports it in *flags and, when no other bit is set, as
 * WQ_ERR_INVALID_ARG. */
#define WQ_DEVFLAG_INDEX 0x8u

/*
 * wq_quantize_tokens -- symmetric INT8 codes of bf16 activations, one scale
 * per token.
 *
 *   x'_k  = bf16_rn(fl32(x_k / smooth_k)) when smooth is given (the values of
 *           wq_awq_scale_activations), else x_k;
 *   s     = fl32(max |x'_k| / 127) over the row's finite values, 1 if that is 0;
 *   q_k   = clamp(rint(fl32(x'_k / s)), -127, 127), ties to even; NaN -> 0,
 *           +-Inf -> +-127 (both raise WQ_DEVFLAG_NONFINITE).
 *
 *   X_bf16       [T][d_in] bf16, input.  16-byte aligned.
 *   T            rows of X, 0 .. 2^31 - 1.
 *   d_in         a multiple of 32, 32 .. WQ_INT8_MAX_D_IN.
 *   rows         device int32 [R] or NULL.  Output row r quantizes X row
 *                rows[r] (a token sent to several experts is quantized into
 *                each expert's rows).  NULL: R must equal T (or be 0), row r is X row r.
 *                An index outside [0, T) gives a row of zero codes with scale
 *                1 and raises WQ_DEVFLAG_INDEX.
 *   R            output rows, 0 .. 2^31 - 1; 0 enqueues nothing (the arrays
 *                may then be NULL).
 *   smooth_bf16  device bf16 [d_in] or NULL.  2-byte aligned.
 *   Xq           [R][d_in] int8 output, two's complement.  16-byte aligned.
 *   x_scales     [R] fp32 output.  4-byte aligned.
 * The outputs may not overlap the inputs.
 * Errors: WQ_ERR_INVALID_ARG for null or misaligned pointers and sizes outside
 * the rules above; WQ_ERR_CUDA if a launch fails.
 */
wq_status wq_quantize_tokens(const void* X_bf16, int64_t T, int64_t d_in, const int32_t* rows, int64_t R,
                             const void* smooth_bf16, int8_t* Xq, float* x_scales, void* stream);

/*
 * wq_linear_w8a8 -- Y[m][n] = s_m w_n sum_k Xq[m][k] q[n][k]: INT8 x INT8 on
 * tensor cores with exact INT32 sums.  The result is
 *   fl32(fl32(fl32(sum) * w_n) * s_m),
 * rounded once more to bf16 for y_dtype WQ_OUT_BF16.  (The weight's scale
 * first: |sum| w_n is below 2^47, so only the true result can overflow.)
 * Deterministic: integer sums do not depend on their order.
 *
 *   Xq           [M][d_in] int8, input (wq_quantize_tokens).  16-byte aligned.
 *   x_scales     [M] fp32, input.  4-byte aligned.
 *   M            tokens, 0 .. 2^31 - 1; 0 enqueues nothing (Xq, x_scales and Y
 *                may then be NULL).
 *   qweight      uint32 [d_out][d_in/4], the codes of wq_quantize_w8.  16-byte
 *                aligned.
 *   scales_fp16  fp16 [d_out]: wq_quantize_w8 with group_size = d_in (one
 *                scale per output channel).  2-byte aligned.
 *   d_out        1 .. 2^31 - 1.
 *   d_in         a multiple of 32, 32 .. WQ_INT8_MAX_D_IN.
 *   Y            [M][d_out] output, y_dtype as wq_linear_w4a16.  16-byte aligned.
 *                May not overlap the inputs.
 * All arrays are read, and Y written, after the work ahead on the stream has
 * ended, also where the kernels ahead let their successors start early
 * (programmatic dependent launch).
 * Errors: WQ_ERR_INVALID_ARG as above; WQ_ERR_UNSUPPORTED for a product of
 * more than 2^30 output tiles; WQ_ERR_CUDA if a launch fails.
 * Device flags: WQ_DEVFLAG_TIMEOUT if a pipeline wait inside the kernel gave
 * up (the output is then incomplete).
 */
wq_status wq_linear_w8a8(const int8_t* Xq, const float* x_scales, int64_t M, const uint32_t* qweight,
                         const void* scales_fp16, int64_t d_out, int64_t d_in, void* Y, int32_t y_dtype,
                         void* stream);

/*
 * wq_linear_w8a8_grouped -- the same product with one weight matrix per
 * expert over tokens sorted by expert: rows offsets[e] .. offsets[e+1] - 1 of
 * Xq are multiplied by expert e's matrix.  Experts may have no rows.  Rows
 * before offsets[0] and from offsets[E] on take no part; Y is not written there.
 *
 *   Xq, x_scales  [R][d_in] int8 and [R] fp32, as wq_linear_w8a8.
 *   R             rows of Xq and Y, 0 .. 2^31 - 1; 0 enqueues nothing.
 *   offsets       device int32 [E + 1], non-decreasing, within [0, R]; read by
 *                 the kernel (the host never waits for the router).  Offsets
 *                 outside these rules raise WQ_DEVFLAG_INDEX; each is then
 *                 taken as the largest of it and those before it, clamped to
 *                 [0, R] (memory-safe, no row belongs to two experts).
 *   E             experts, 1 .. WQ_INT8_MAX_EXPERTS.
 *   qweight       uint32 [E][d_out][d_in/4]; scales_fp16 fp16 [E][d_out]:
 *                 wq_quantize_w8 of the experts' matrices stacked by rows.
 *                 E * d_out <= 2^31 - 1.
 *   d_out, d_in, Y, y_dtype, errors, flags: as wq_linear_w8a8; WQ_ERR_UNSUPPORTED
 *                 also for E > WQ_INT8_MAX_EXPERTS.
 */
wq_status wq_linear_w8a8_grouped(const int8_t* Xq, const float* x_scales, int64_t R, const int32_t* offsets, int64_t E,
                                 const uint32_t* qweight, const void* scales_fp16, int64_t d_out, int64_t d_in,
                                 void* Y, int32_t y_dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* WQ_INT8_H_ */
