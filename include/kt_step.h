/*
 * kt_step.h: C ABI of what completes a training and a decoding step around the
 * routed experts of kt_rawint4.h on MI355X (gfx950): norms before and after a
 * block, fused with its gate, its scale and the residual stream, with their
 * gradients; an AdamW step over many tensors at once; and the routed experts
 * for a few tokens.
 *
 * They are in the same library and follow the conventions of kt_block.h:
 * device pointers, dense row-major tensors, bf16 as uint16 bit patterns,
 * caller-owned workspaces (256-byte aligned), work enqueued on `stream` of the
 * current device and nothing else, no allocation of device memory, no
 * synchronisation, nothing that a stream capture refuses, the same return codes,
 * and kt_rawint4_last_error for the message.  Outputs overlap no other
 * argument unless an entry point allows it.  Results depend on the inputs
 * alone, bit for bit.  A workspace holds nothing between calls; calls that
 * may run at the same time, replays of captured graphs among them, need
 * workspaces of their own.
 */
#ifndef KT_STEP_H
#define KT_STEP_H

#include "kt_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ norms (at most 2^23 tokens a call) */

#define KT_NORM_RMS 0   /* N(v) = v / sqrt(mean(v^2) + eps) */
#define KT_NORM_LAYER 1 /* N(v) = (v - mean(v)) / sqrt(mean((v - mean(v))^2) + eps) */
#define KT_NORM_MAX_HIDDEN 16384

/*
 * The norms on both sides of a block.  H = hidden is any number in
 * [1, KT_NORM_MAX_HIDDEN]; eps >= 0 and scale are finite.  The vectors are fp32 [H],
 * each may be NULL: a weight of ones, a bias of zeros, a gate of ones.
 * branch_weight and branch_bias belong to the norm behind the block, which is
 * there where branch_norm is 1.
 */
typedef struct kt_norm {
  int32_t hidden;
  int32_t kind;        /* KT_NORM_* of both norms */
  int32_t stream_type; /* KT_TYPE_* of the residual stream and its gradient */
  int32_t branch_norm; /* 0 or 1 */
  float eps;
  float scale; /* of the block's output */
  const float* weight;
  const float* bias;
  const float* branch_weight;
  const float* branch_bias;
  const float* gate;
} kt_norm;

/*
 * From the residual stream x [tokens, H] (stream_type) and a block's output
 * b [tokens, H] (bf16, or NULL for none):
 *   n = branch_norm ? N(b) * branch_weight + branch_bias : b
 *   h = x + scale * gate * token_gate * n       (h = x without b)
 *   y = N(h) * weight + bias
 * token_gate [tokens] fp32 or NULL.  h [tokens, H] (stream_type) may be x itself; y [tokens, H]
 * bf16.  Either may be NULL (not wanted), h has to be without b.  y is
 * computed from h before h's rounding.  Sums are fp32; each output is rounded
 * once.  Values that N takes are up to 2^56 in magnitude, and with eps = 0 not all of a row's
 * below 2^-50: squares of others leave fp32, and N may be 0, infinite or NaN.  The vectors, and all tensors, 16-byte aligned, token_gate 4-byte.  tokens == 0
 * is a valid no-op.
 */
int kt_norm_fwd(const kt_norm* norm, int32_t tokens, const void* x, const uint16_t* branch, const float* token_gate,
                void* h, uint16_t* y, void* stream);

/*
 * Gradients of kt_norm_fwd at the h that it wrote (x itself without b), from
 * grad_h (stream_type: what reaches h along the residual stream) and grad_y
 * (bf16), of which one may be NULL:
 *   grad_x [tokens, H] (stream_type) = grad_h + the part of h in grad_y; it
 *   may be grad_h itself;
 *   grad_branch [tokens, H] bf16, grad_token_gate [tokens] fp32;
 *   d_weight, d_bias (of y), d_branch_weight, d_branch_bias, d_gate: fp32 [H],
 *   each (accumulate ? itself : 0) + grad_scale * the sum over the tokens (the window
 *   rule of kt_rawint4_moe_bwd).
 * Every output may be NULL; those of a part that the call does not have (no
 * branch, no branch_norm, no grad_y, no token_gate) have to be.  d_bias,
 * d_branch_bias and d_gate need no such vector in the struct.  Sums over the tokens have a
 * fixed order.  tokens == 0: only the window rule runs.  A workspace of the size for some number of tokens
 * serves every smaller number too.
 */
size_t kt_norm_bwd_workspace_bytes(const kt_norm* norm, int32_t tokens);
int kt_norm_bwd(const kt_norm* norm, int32_t tokens, const void* h, const uint16_t* branch, const float* token_gate,
                const void* grad_h, const uint16_t* grad_y, void* grad_x, uint16_t* grad_branch,
                float* grad_token_gate, float* d_weight, float* d_bias, float* d_branch_weight, float* d_branch_bias,
                float* d_gate, int32_t accumulate, float grad_scale, void* workspace, size_t workspace_bytes,
                void* stream);

/* ------------------------------------------------------------------ AdamW over many tensors */

#define KT_ADAMW_STATES_F32 0
#define KT_ADAMW_STATES_E4M3 1
#define KT_ADAMW_BLOCK 256 /* values of an 8-bit state that share a scale */
#define KT_ADAMW_MAX_TENSORS 65536

/* The step's numbers; beta1, beta2 in [0, 1), the others finite, eps >= 0, max_norm >= 0 (0: no clipping). */
typedef struct kt_adamw {
  double lr;
  double beta1;
  double beta2;
  double eps;
  double weight_decay;
  double max_norm;
  double grad_scale;
  int32_t state_format; /* KT_ADAMW_STATES_* */
} kt_adamw;

/*
 * One tensor of `count` values (at most 2^36), 16-byte aligned: param (param_type), grad
 * (grad_type), the moments m and v.  master: fp32 [count] or NULL; the update
 * is made to it and param, which has to be bf16, receives it rounded.  KT_ADAMW_STATES_F32: m and v
 * are fp32 [count], the scales NULL.  KT_ADAMW_STATES_E4M3: m holds codes of m and
 * v of sqrt(v), one byte each, [count], and m_scale, v_scale fp32
 * [ceil(count / 256)] what a code of 1 stands for in each block of 256
 * values: the block's largest magnitude / 448.  The code of a positive
 * sqrt(v) is never 0.  A block whose largest magnitude is below 2^-100 holds zeros.
 * A moment that is not finite (the square of a gradient from 2^64 on is not) stays in its block, whose other
 * moments may not be finite from then on; grad_norm finds gradients that are not finite before anything changes.
 */
typedef struct kt_adamw_tensor {
  int64_t count;
  int32_t param_type; /* KT_TYPE_* */
  int32_t grad_type;  /* KT_TYPE_* */
  int32_t decay;      /* 0: no weight decay for this tensor */
  void* param;
  float* master;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
} kt_adamw_tensor;

/*
 * step[0] (int64 on the device, the number of steps made before) grows by
 * one to t, and for every tensor, with g = grad_scale * c * grad:
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * in fp32; p is the master where there is one.  c = 1, or with max_norm > 0
 * min(1, max_norm / (norm + 1e-6)) by the global norm = |grad_scale * grad|_2 over all tensors (64-bit sums).
 * grad_norm [1] fp32 on the device, or NULL: receives that norm; needed with
 * max_norm > 0.  With it, a norm that is not finite makes the call change
 * nothing but grad_norm.  lr [1] fp32 on the device, or NULL: replaces
 * hyper->lr (a schedule that replays of a captured graph follow).
 * `tensors` is read on the host during the call.  A tensor stands in the
 * list once.
 */
size_t kt_adamw_workspace_bytes(int32_t num_tensors);
int kt_adamw_step(const kt_adamw* hyper, const kt_adamw_tensor* tensors, int32_t num_tensors, int64_t* step,
                  float* grad_norm, const float* lr, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ the experts for a few tokens */

#define KT_MOE_DECODE_MAX_TOKENS 64
#define KT_MOE_DECODE_MAX_SLOTS 1024 /* tokens * top_k */
#define KT_MOE_DECODE_MAX_HIDDEN 16384

/*
 * kt_rawint4_moe_infer for up to KT_MOE_DECODE_MAX_TOKENS tokens (and a hidden
 * of up to KT_MOE_DECODE_MAX_HIDDEN): the same arguments and formula, in two
 * or three kernels (two more with LoRA), without sorting, converted scales or staged rows.
 * Gate and up go through the packed rows of each chosen expert once for two of its token-slots, down once for each.
 * Which of the two is faster goes by the slots that an expert in use has on average: as measured, this
 * one up to about 2 where many experts are in use (of 64 to 384) and about 6 where 8 are; above that
 * kt_rawint4_moe_infer, by up to 6 times (64 tokens that share 8 experts).  bf16
 * scales have no numeric domain; inputs are up to 2^120 in magnitude (of larger
 * ones sums may leave fp32's range and become infinite or NaN).  Products and
 * sums are fp32; h is kept in between to 2^-22 of the largest of 16 neighbours
 * and better.  An input that is NaN makes its token's output NaN, and with
 * RAWINT4 so does an infinite one; with MXFP4 that goes by the formula (infinite
 * or NaN sums; infinite ones are clamped as others are).  A token without a
 * valid id gets zeros whatever its input.  tokens == 0 is a valid no-op.  A workspace of the size for some
 * number of tokens serves every smaller number too.
 */
size_t kt_moe_decode_workspace_bytes(const kt_rawint4_moe_layer* layer, int32_t tokens);
int kt_moe_decode(const kt_rawint4_moe_layer* layer, int32_t tokens, const uint16_t* inputs, const int64_t* expert_ids,
                  const float* route_weights, uint16_t* output, void* workspace, size_t workspace_bytes,
                  void* stream);

#ifdef __cplusplus
}
#endif

#endif /* KT_STEP_H */
