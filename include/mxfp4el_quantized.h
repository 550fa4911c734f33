/*
 * mxfp4el_quantized.h -- C ABI of the operators around the MXFP4 routed
 * experts on quantised tokens, in the same library as mxfp4_expert_linear.h,
 * with the same status codes, dtypes and rules (device pointers owned by the
 * caller, work enqueued on `stream`, arguments checked before anything is
 * enqueued, no output overlapping an input).
 *
 *   mxfp4_route_experts            experts and mixture weights from logits
 *   mxfp4_quantize                 rows of values to MXFP4
 *   mxfp4_dequantize               the values that MXFP4 rows stand for
 *   mxfp4_linear                   product of MXFP4 tokens and MXFP4 weights
 *   mxfp4_expert_linear_quantized  the routed expert linear on MXFP4 tokens
 *
 * MXFP4. A row of I values (I a multiple of 32) is I/32 groups of 16 bytes
 * (two E2M1 codes each, the lower value in the low nibble) and one scale byte
 * per group, the layout of the experts' weights: packed (rows, I/32, 16),
 * scales (rows, I/32). A code of magnitude 0, 0.5, 1, 1.5, 2, 3, 4 or 6 under
 * the scale byte s stands for that times 2^(s-127). The operators of this
 * header take s = 255 as NaN, as the OCP format has it (the calls of
 * mxfp4_expert_linear.h take it as 2^128); no finite row quantises to it.
 */
#ifndef MXFP4EL_QUANTIZED_H
#define MXFP4EL_QUANTIZED_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Experts and mixture weights of T tokens. logits (T, E) of `dtype`
 * (MXFP4EL_DTYPE_F32 or _BF16), rows row_stride elements apart; bias (E)
 * float32 or NULL; selected_experts (T, K) int32 and mixture_weights (T, K)
 * float32 are written.
 *
 *   score  = softmax(logits) over the E experts, or sigmoid(logit)
 *   choice = score + bias
 *
 * With groups > 1 the experts are `groups` runs of E / groups, a group's
 * score is the sum of its group_best (1 or 2) highest choices (of fewer where
 * it has fewer), and only the top_groups groups of highest score take part.
 * Of those experts the K of highest choice are selected, highest first; equal
 * choices and equal groups go to the lower index. Without a bias experts
 * rank by logit (the same order, without the scores' rounding). The
 * weights are the selected experts' scores, divided by their sum plus 1e-20
 * where `normalize` is not 0, times `scaling`.
 *
 * Ranks are those of scores and choices in float64, also where float32 does
 * not tell two apart; weights are computed in float32 (2^-18 relative at most,
 * about 2^-24 as a rule). An expert whose logit or choice is NaN is never selected,
 * nor is a group whose score is NaN (infinities of both signs); one whose logit is
 * NaN has no share in the softmax. A softmax row whose
 * largest logit is infinite shares its weight among the experts that have
 * it. Slots that are left over get id -1 and weight 0, which the expert
 * linear skips.
 *
 * 0 < E <= 1024, 0 <= K <= 32, groups a divisor of E up to 32, K at most
 * top_groups * (E / groups); group_best 1 or 2; scaling finite. Up to some 16
 * picks most tokens are decided in float32 with an error bound; with more, tokens
 * over more experts than picks go to float64, some 30 times as slow.
 *
 * mxfp4_router_topk (mxfp4_expert_linear.h) is the router that
 * mxfp4_expert_linear_routed and the SwiGLU expert run in front: sigmoid, no groups,
 * float32 logits, ranked by float32 choices. On the same formula the two may pick
 * differently where float32 does not tell choices apart; take this one where the
 * choice is made in a call of its own.
 */
#define MXFP4EL_SCORE_SOFTMAX 0
#define MXFP4EL_SCORE_SIGMOID 1
int mxfp4_route_experts(const void* logits, int dtype, int64_t row_stride, const float* bias,
                        int64_t T, int64_t E, int64_t K, int score, int64_t groups,
                        int64_t top_groups, int64_t group_best, int normalize, float scaling,
                        int32_t* selected_experts, float* mixture_weights, void* stream);

/*
 * Rows of values to MXFP4: x (rows, I) of `dtype`, rows row_stride elements
 * apart (any alignment of whole elements); packed (rows, I/32, 16) and scales
 * (rows, I/32) are written, packed on a 16-byte boundary.
 *
 * A group of largest magnitude a gets s = clamp(floor(log2 a) - 2 + 127, 0,
 * 252), 0 where a = 0, and each value x 2^(127-s) rounded to the nearest of
 * the code's magnitudes, ties to the even code, beyond 6 to 6; the sign is
 * kept, a zero's too. A group that holds an infinity or a NaN gets s = 255
 * and zero codes.
 */
int mxfp4_quantize(const void* x, int dtype, int64_t row_stride, int64_t rows, int64_t I,
                   uint8_t* packed, uint8_t* scales, void* stream);

/*
 * The values of MXFP4 rows, out (rows, I) of `dtype`: exact, except that
 * codes under s >= 253 may pass the largest finite number and become
 * infinite, and s = 255 gives NaN. packed and out on 16-byte boundaries.
 */
int mxfp4_dequantize(const uint8_t* packed, const uint8_t* scales, int64_t rows, int64_t I,
                     void* out, int dtype, void* stream);

/*
 * out[t, o] = sum_i x[t, i] w[o, i] of MXFP4 tokens (T, I) and MXFP4 weights
 * (O, I). Products are exact and add up in float32 on the tensor cores; the
 * result is rounded once to `out_dtype`. The order of every sum is fixed, so
 * the same call on the same inputs gives the same bits. x_packed and
 * packed_weights lie on 16-byte boundaries, scale bytes anywhere.
 *
 * workspace: mxfp4_linear_workspace_size() bytes on a 256-byte boundary (0
 * bytes for most sizes: NULL then), not needing any contents, used by this
 * call alone until it is done.
 */
size_t mxfp4_linear_workspace_size(int64_t T, int64_t I, int64_t O);
int mxfp4_linear(const uint8_t* x_packed, const uint8_t* x_scales, const uint8_t* packed_weights,
                 const uint8_t* scale_bytes, void* out, int64_t T, int64_t I, int64_t O,
                 int out_dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * mxfp4_expert_linear on MXFP4 tokens:
 *
 *   out[t] = shared_output[t] + sum_k mixture_weights[t,k] W_{selected_experts[t,k]} x_t
 *
 * x_packed (T, I/32, 16) and x_scales (T, I/32) are the tokens; the weights,
 * the routing and the shared output are as there, except for scale bytes of
 * 255 (NaN). `dtype` is that of shared_output and out. Each pair's result is
 * a float32 sum, as in mxfp4_linear; they are added to the shared output in
 * slot order in float32 and rounded once. An expert id out of range
 * contributes nothing and is counted for mxfp4el_device_errors(). At most
 * 4096 experts may have tokens: min(E, T * K) <= 4096.
 *
 * workspace: mxfp4_expert_linear_quantized_workspace_size() bytes on a
 * 256-byte boundary, as in mxfp4_linear.
 */
size_t mxfp4_expert_linear_quantized_workspace_size(int64_t T, int64_t E, int64_t I, int64_t O,
                                                    int64_t K);
int mxfp4_expert_linear_quantized(const uint8_t* x_packed, const uint8_t* x_scales,
                                  const uint8_t* packed_weights, const uint8_t* scale_bytes,
                                  const void* selected_experts, const float* mixture_weights,
                                  const void* shared_output, void* out, int64_t T, int64_t E,
                                  int64_t I, int64_t O, int64_t K, int dtype, int index_dtype,
                                  void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif
