/*
 * kt_block.h: C ABI of the operators around the routed experts of kt_rawint4.h
 * on MI355X (gfx950): routing of tokens to experts with its gradient, dense
 * products with bias, activation and residual in their epilogue with their
 * gradients, and activation checkpoints in 8 bits with the backward passes
 * that read them.
 *
 * They are in the same library and follow the conventions stated in
 * kt_rawint4.h: device pointers, dense row-major tensors, bf16 as uint16 bit
 * patterns, caller-owned workspaces (256-byte aligned), work enqueued on
 * `stream` of the current device and nothing else, no allocation of device
 * memory, no synchronisation, nothing that a stream capture refuses, the same
 * return codes, and kt_rawint4_last_error for the message.  Outputs overlap no
 * other argument unless an entry point allows it.  Results depend on
 * the inputs alone, bit for bit: no kernel accumulates floating-point numbers
 * with atomics.  A workspace holds nothing between calls; calls that may run
 * at the same time, replays of captured graphs among them, need workspaces of
 * their own.
 */
#ifndef KT_BLOCK_H
#define KT_BLOCK_H

#include "kt_rawint4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element types */
#define KT_TYPE_BF16 0
#define KT_TYPE_F32 1

/* ------------------------------------------------------------------ routing (at most 2^23 tokens a call) */

#define KT_SCORE_SOFTMAX 0
#define KT_SCORE_SIGMOID 1
#define KT_ROUTER_MAX_GROUPS 64

/*
 * How tokens choose experts.  E = num_experts (1 .. KT_RAWINT4_MAX_EXPERTS),
 * k = top_k (1 .. E); experts form num_groups groups of E / num_groups
 * neighbours (num_groups divides E and is at most KT_ROUTER_MAX_GROUPS), of
 * which a token keeps top_groups; k <= top_groups * E / num_groups.  group_top is 1 or
 * 2 and at most E / num_groups.  scale is finite.
 */
typedef struct kt_router {
  int32_t num_experts;
  int32_t top_k;
  int32_t num_groups;
  int32_t top_groups;
  int32_t group_top;
  int32_t score;       /* KT_SCORE_* */
  int32_t renormalize; /* 0 or 1 */
  float scale;
  int32_t logits_type; /* KT_TYPE_* of the logits and of their gradient */
} kt_router;

/*
 * For every token, from its logits l [tokens, E] and the bias b [E] (fp32, or
 * NULL for none; it takes part in the choice alone, for balance):
 *   s = softmax(l) or sigmoid(l) (1 / (1 + exp(-l))),   c = s + b,
 *   a group's score is the sum of its group_top largest c; the top_groups
 *   groups of the largest scores stay (num_groups > 1),
 *   expert_ids [tokens, k] int64: the k experts of those groups with the
 *   largest c, in descending order,
 *   route_weights [tokens, k] fp32: scale * s / (renormalize ? sum of the k s
 *   + 1e-20 : 1).
 * Choices are made on c to 64 bits (without a bias on the logits, which order
 * as s does); equal values go to the lower index.  The outputs are what
 * kt_rawint4_moe_fwd takes as expert_ids and route_weights.
 *   - An expert whose logit or bias is -inf is never chosen; where fewer than
 *     k are left, the other slots hold id -1 (which the experts drop) and
 *     weight 0.  Its logit counts in the softmax as a probability of 0.
 *   - token_mask [tokens] uint8, or NULL: a token whose byte is 0 (padding)
 *     gets ids -1 and weights 0; its logits may hold anything.
 *   - A token with a NaN logit (with softmax a logit of +inf too), and every token if a bias
 *     is NaN or +inf, gets ids 0 .. k-1 and weights NaN.
 *   - load [E] int32, or NULL: load = (accumulate ? load : 0) + how many slots
 *     chose each expert.
 *   - Weights, like the gradient below, are computed in fp32 whatever the choice
 *     takes: a score below 2^-149 is 0, and the terms of a softmax's sum are within
 *     2^-23 (2 + 1.5 |l - max|) of their size.
 * tokens == 0 is valid (load is still cleared where accumulate is 0).
 * logits must be 16-byte aligned, expert_ids 8-byte, the rest by their type.
 */
int kt_router_fwd(const kt_router* router, int32_t tokens, const void* logits, const float* bias,
                  const uint8_t* token_mask, int64_t* expert_ids, float* route_weights, int32_t* load,
                  int32_t accumulate, void* stream);

/*
 * Gradient of route_weights with respect to the logits, at given expert_ids
 * (the choice itself has none): grad_route [tokens, k] fp32 is dL/droute_weights as
 * kt_rawint4_moe_bwd gives it, grad_logits [tokens, E] has the logits' type.
 *   S = sum of the chosen s + 1e-20,  d = sum g s / S,
 *   ds = scale * (renormalize ? (g - d) / S : g) at the chosen experts, else 0
 *   dl = s * (ds - sum ds s)  (softmax)   or   ds * s * (1 - s)  (sigmoid)
 * Slots whose id lies outside [0, E) take no part; a token without any other
 * slot gets zeros.  A token with another slot and a NaN logit (softmax: or a
 * +inf one) gets NaN.  An id that a token holds twice counts twice.
 * grad_logits must not overlap the logits.
 */
int kt_router_bwd(const kt_router* router, int32_t tokens, const void* logits, const int64_t* expert_ids,
                  const float* grad_route, void* grad_logits, void* stream);

/*
 * The balance rule for the bias: bias[e] += rate where load[e] is below the
 * mean load, -= rate where it is above, unchanged where it is equal (decided
 * in whole numbers: load[e] * E against the sum).  num_experts as above; rate
 * finite; every load >= 0.
 */
int kt_router_update_bias(float* bias, const int32_t* load, int32_t num_experts, float rate, void* stream);

/* ---------------------------------------------- activation checkpoints in 8 bits */

#define KT_CKPT8_INT8 0
#define KT_CKPT8_E4M3 1
#define KT_CKPT8_GROUP 32

/*
 * Rows x [rows, cols] of bf16 as codes [rows, cols] (one byte each) and scales
 * [rows, ceil(cols / 32)] (one byte for 32 columns of a row, the last group of
 * a row may be shorter): the value is code * 2^(scale - 127).
 *   KT_CKPT8_INT8: two's complement -127 .. 127; the group's exponent is the
 *   smallest at which its largest magnitude rounds to at most 127.
 *   KT_CKPT8_E4M3: the 8-bit floating-point number of the OCP formats (bias 7,
 *   largest 448); the exponent is the smallest at which the largest magnitude
 *   is at most 448.
 * Exponents below -127 become -127 (scale byte 0, also of a group of zeros).
 * Codes are rounded to nearest even; a value that would become larger than bf16
 * holds takes the next code below (the exponent is at most 121, INT8, or 120,
 * E4M3, whose codes are then at most 240).  Every value that a checkpoint of bf16 rows
 * stands for is itself a bf16 value, so unpacking rounds nothing.  A group that
 * holds an infinity or a NaN gets scale byte 255 and codes 0; it unpacks to NaNs.
 * Error of a value: at most amax / 127 (INT8), or max(2^-4 |x|, 2^-17 amax)
 * (E4M3), amax the group's largest magnitude (and up to 2^-128 where the
 * exponent is at its lowest).
 * x must be 16-byte aligned, codes and scales 4-byte; at most
 * 2^32 groups a call.
 */
int kt_ckpt8_pack(const uint16_t* x, int64_t rows, int64_t cols, int32_t format, uint8_t* codes, uint8_t* scales,
                  void* stream);
int kt_ckpt8_unpack(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, int32_t format,
                    uint16_t* x, void* stream);

/*
 * kt_rawint4_moe_bwd_recompute for a caller that kept the experts' inputs as
 * a checkpoint (codes [qlen, H], scales [qlen, H / 32]) instead of bf16 rows:
 * the inputs are unpacked into the workspace and the rest is that call, with
 * the same results, bit for bit, as on unpacked inputs.  The gradients are
 * those at the unpacked inputs.  The workspace
 * (kt_moe_bwd_ckpt8_workspace_bytes) holds those rows behind the recompute's; its
 * size is for that qlen, as the recompute's is (a smaller one may need more).
 */
size_t kt_moe_bwd_ckpt8_workspace_bytes(const kt_rawint4_moe_layer* layer, int32_t qlen);
int kt_moe_bwd_ckpt8(const kt_rawint4_moe_layer* layer, int32_t qlen, int32_t format, const uint8_t* codes,
                     const uint8_t* scales, const int64_t* expert_ids, const float* route_weights,
                     const uint16_t* grad_output, uint16_t* grad_input, float* grad_route, float* d_gate_a,
                     float* d_gate_b, float* d_up_a, float* d_up_b, float* d_down_a, float* d_down_b,
                     int32_t accumulate, float grad_scale, void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------- dense products (at most 2^20 tokens a call) */

#define KT_ACT_NONE 0
#define KT_ACT_RELU 1
#define KT_ACT_SILU 2
#define KT_ACT_GELU 3      /* z Phi(z) */
#define KT_ACT_GELU_TANH 4 /* z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2 */

/*
 * A dense layer: weight [N, K] bf16, bias [N] fp32 or NULL.  K = in_features
 * is a multiple of 8 (rows of 16 bytes) in [8, 65536], N = out_features any
 * number in [1, 65536].
 */
typedef struct kt_linear {
  int32_t in_features;
  int32_t out_features;
  int32_t activation; /* KT_ACT_* */
  const uint16_t* weight;
  const float* bias;
} kt_linear;

/*
 * z = x W^T + b,  output = act(z) + residual.
 * inputs [tokens, K] bf16; residual [tokens, N] bf16 or NULL (it may be the
 * output itself where that is bf16); output [tokens, N] of output_type; preact
 * [tokens, N] bf16 or NULL receives z, which the backward of an activation
 * reads.  Sums are fp32, each output is rounded once.  Within a call, equal rows
 * of inputs (and residual) give equal rows of outputs, wherever they stand.  All tensors 16-byte
 * aligned.  The router's logits are a call of this with a weight of [E, H]
 * and KT_TYPE_F32.  tokens == 0 is a valid no-op.  A workspace of the size for
 * some number of tokens serves every smaller number too.  The size may be 0; the
 * workspace may then be NULL.
 */
size_t kt_linear_workspace_bytes(const kt_linear* linear, int32_t tokens);
int kt_linear_fwd(const kt_linear* linear, int32_t tokens, const uint16_t* inputs, const uint16_t* residual,
                  void* output, int32_t output_type, uint16_t* preact, void* workspace, size_t workspace_bytes,
                  void* stream);

/* Inputs kept as a checkpoint (see above). */
typedef struct kt_ckpt8 {
  int32_t format; /* KT_CKPT8_* */
  const uint8_t* codes;
  const uint8_t* scales;
} kt_ckpt8;

/*
 * Gradients of kt_linear_fwd:
 *   dz = grad_output * act'(preact)             (relu' is 0 at 0)
 *   grad_input [tokens, K] bf16 = dz W + grad_residual
 *   d_weight [N, K] fp32 = (accumulate ? d_weight : 0) + grad_scale * dz^T x
 *   d_bias [N] fp32 = (accumulate ? d_bias : 0) + grad_scale * sum of dz
 * (the window rule of kt_rawint4_moe_bwd; the residual's gradient is
 * grad_output).  The inputs x are given as bf16 rows or as a checkpoint, the
 * other pointer NULL.  preact is the one that the forward wrote; NULL, and
 * not read, for KT_ACT_NONE.  grad_output is of grad_output_type.
 * grad_residual [tokens, K] bf16 or NULL is added to grad_input and may be
 * grad_input itself, such as the experts' grad_input when this is the router's
 * product.  grad_input, d_weight and d_bias may each be NULL: not
 * computed.  d_bias needs no bias in the layer.
 * d_weight and d_bias come from dz to fp32's precision, grad_input from dz to
 * 2^-16 of it, far below its own rounding to bf16: a dz that bf16 may not hold
 * (of an fp32 gradient, or behind an activation) takes part as a sum of bf16 numbers of
 * its sign.  Its product with an infinite input or weight is infinite for
 * |dz| above 2^-100 and may be NaN below.
 * tokens == 0: only the window rule runs.  A workspace of the size for some
 * number of tokens serves every smaller number too.  It is larger for calls with a
 * checkpoint (from_checkpoint nonzero); such a one serves both.
 */
size_t kt_linear_bwd_workspace_bytes(const kt_linear* linear, int32_t tokens, int32_t from_checkpoint);
int kt_linear_bwd(const kt_linear* linear, int32_t tokens, const uint16_t* inputs, const kt_ckpt8* checkpoint,
                  const uint16_t* preact, const void* grad_output, int32_t grad_output_type,
                  const uint16_t* grad_residual, uint16_t* grad_input, float* d_weight, float* d_bias,
                  int32_t accumulate, float grad_scale, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KT_BLOCK_H */
