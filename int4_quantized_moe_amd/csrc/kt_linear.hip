// Dense products with bias, activation and residual in their epilogue, and
// their gradients.
#include <math.h>

#include "kt_common.hpp"
#include "kt_internal.hpp"

namespace kt {

// ---------------------------------------------------------------- activations

constexpr float kSqrt2OverPi = 0.7978845608028654f, kInvSqrt2 = 0.7071067811865476f, kInvSqrt2Pi = 0.3989422804014327f;

// GELU's tanh form through 0.5 (1 + tanh u) = sigmoid(2u); |z| is held to 16
// inside the polynomial, beyond which the sigmoid is 0 or 1 in fp32, so that
// nothing overflows there.
__device__ __forceinline__ float gelu_tanh_arg(float z) {
  const float c = fminf(fmaxf(z, -16.f), 16.f);
  return 2.f * kSqrt2OverPi * (c + 0.044715f * c * c * c);
}
__device__ __forceinline__ float sigmoid_lin(float u) { return 1.f / (1.f + expf(-u)); }

__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case KT_ACT_RELU: return z < 0.f ? 0.f : z;  // NaN stays
    case KT_ACT_SILU: return z * sigmoid_lin(z);
    case KT_ACT_GELU: return 0.5f * z * (1.f + erff(z * kInvSqrt2));
    case KT_ACT_GELU_TANH: return z * sigmoid_lin(z != z ? z : gelu_tanh_arg(z));
    default: return z;
  }
}

__device__ __forceinline__ float act_slope(int act, float z) {
  switch (act) {
    case KT_ACT_RELU: return z > 0.f ? 1.f : z != z ? z : 0.f;
    case KT_ACT_SILU: {
      const float p = sigmoid_lin(z);
      return p * (1.f + fminf(fmaxf(z, -128.f), 128.f) * (1.f - p)) + (z != z ? z : 0.f);
    }
    case KT_ACT_GELU: {
      const float c = fminf(fmaxf(z, -16.f), 16.f);
      return 0.5f * (1.f + erff(z * kInvSqrt2)) + c * expf(-0.5f * c * c) * kInvSqrt2Pi;
    }
    case KT_ACT_GELU_TANH: {
      if (z != z) return z;
      const float c = fminf(fmaxf(z, -16.f), 16.f);
      const float p = sigmoid_lin(gelu_tanh_arg(z));
      return p + c * p * (1.f - p) * (2.f * kSqrt2OverPi) * (1.f + 3.f * 0.044715f * c * c);
    }
    default: return 1.f;
  }
}

// ---------------------------------------------------------------- product

// C[m, n] = sum_k A(m, k) B(n, k) with A(m, k) = a[m * am + k * ak] and likewise
// B, then the epilogue of one of the three products.
enum LinearKind { kLinFwd, kLinDx, kLinDw };

struct LinearGemm {
  const uint16_t *a, *b;
  int64_t am, ak, bn, bk;
  int64_t M, N, K;
  int planes;       // A is the sum of so many bf16 planes ...
  int64_t a_plane;  // ... so many elements apart
  // forward: bias, act, residual, out (type), preact; dx: residual, out; dw: out (fp32), accumulate, scale
  const float* bias;
  const uint16_t* residual;
  void* out;
  int out_f32;
  uint16_t* preact;
  int act;
  int accumulate;
  float scale;
};

template <int KIND>
__device__ __forceinline__ void finish(const LinearGemm& g, int64_t m, int64_t n, float v) {
  const int64_t i = m * g.N + n;
  if (KIND == kLinDw) {
    float* o = static_cast<float*>(g.out) + i;
    *o = (g.accumulate ? *o : 0.f) + g.scale * v;
    return;
  }
  if (KIND == kLinFwd) {
    if (g.bias) v += g.bias[n];
    if (g.preact) g.preact[i] = float_to_bf16(v);
    v = act_value(g.act, v);
  }
  if (g.residual) v += bf16_to_float(g.residual[i]);
  if (KIND == kLinFwd && g.out_f32)
    static_cast<float*>(g.out)[i] = v;
  else
    static_cast<uint16_t*>(g.out)[i] = float_to_bf16(v);
}

// 64 x 64 outputs per block of four waves (32 x 32 each), 32 values of the
// contraction per step, staged through LDS one element at a time.
template <int KIND>
__global__ __launch_bounds__(256) void k_linear(LinearGemm g) {
  __shared__ __align__(16) uint16_t sa[64][40], sb[64][40];
  const int64_t nt = (g.N + 63) / 64;
  const int64_t m0 = (int64_t)blockIdx.x / nt * 64, n0 = (int64_t)blockIdx.x % nt * 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  floatx4 acc[2][2] = {};
  for (int p = 0; p < g.planes; ++p)
    for (int64_t k0 = 0; k0 < g.K; k0 += 32) {
      for (int i = threadIdx.x; i < 64 * 32; i += 256) {
        // consecutive threads along the operand's contiguous direction
        const int ra = g.ak == 1 ? i >> 5 : i & 63, ka = g.ak == 1 ? i & 31 : i >> 6;
        const int rb = g.bk == 1 ? i >> 5 : i & 63, kb = g.bk == 1 ? i & 31 : i >> 6;
        sa[ra][ka] = m0 + ra < g.M && k0 + ka < g.K ? g.a[p * g.a_plane + (m0 + ra) * g.am + (k0 + ka) * g.ak] : 0;
        sb[rb][kb] = n0 + rb < g.N && k0 + kb < g.K ? g.b[(n0 + rb) * g.bn + (k0 + kb) * g.bk] : 0;
      }
      __syncthreads();
      u32x4 fa[2], fb[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        fa[q] = *reinterpret_cast<const u32x4*>(&sa[wm + 16 * q + (lane & 15)][8 * (lane >> 4)]);
        fb[q] = *reinterpret_cast<const u32x4*>(&sb[wn + 16 * q + (lane & 15)][8 * (lane >> 4)]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma_bf16(fa[i], fb[j], acc[i][j]);
      __syncthreads();
    }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t m = m0 + wm + 16 * i + 4 * (lane >> 4) + r, n = n0 + wn + 16 * j + (lane & 15);
        if (m < g.M && n < g.N) finish<KIND>(g, m, n, acc[i][j][r]);
      }
}

// ---------------------------------------------------------------- dz and its column sums

// dz = grad_output * act'(preact) as one or two bf16 planes (hi and, where a
// product needs more than bf16 holds, lo = bf16(dz - hi)).
struct DzArgs {
  const void* dy;
  int dy_f32;
  const uint16_t* z;
  int act;
  int64_t T, N;
  uint16_t *hi, *lo;
  float* part;  // [row blocks][N] column sums
};

__device__ __forceinline__ float dz_at(const DzArgs& a, int64_t i) {
  const float dy =
      a.dy_f32 ? static_cast<const float*>(a.dy)[i] : bf16_to_float(static_cast<const uint16_t*>(a.dy)[i]);
  if (a.act == KT_ACT_NONE) return dy;
  const float z = bf16_to_float(a.z[i]);
  if (a.act == KT_ACT_RELU) return z > 0.f ? dy : z != z ? z : 0.f;
  return dy * act_slope(a.act, z);
}

// hi + lo with a relative error of at most 2^-17; the sum stays finite where v is, and infinite
// where v is infinite.
__device__ __forceinline__ void split_planes(float v, uint16_t& hi, uint16_t& lo) {
  split_bf16(v, hi, lo);
  if ((hi & 0x7fff) == 0x7f80) {
    if (fabsf(v) < INFINITY) {
      hi -= 1;  // the largest finite number of bf16
      lo = float_to_bf16(v - bf16_to_float(hi));
    } else {
      lo = 0;
    }
  }
}

constexpr int kDzRows = 64;

// 64 columns x kDzRows rows per block.
__global__ __launch_bounds__(256) void k_linear_dz(DzArgs a) {
  __shared__ float red[4][64];
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int64_t n = (int64_t)blockIdx.x * 64 + c;
  float sum = 0.f;
  if (n < a.N)
    for (int r = q; r < kDzRows; r += 4) {
      const int64_t t = (int64_t)blockIdx.y * kDzRows + r;
      if (t >= a.T) break;
      const int64_t i = t * a.N + n;
      const float v = dz_at(a, i);
      sum += v;
      uint16_t hi, lo;
      split_planes(v, hi, lo);
      if (a.hi) a.hi[i] = hi;
      if (a.lo) a.lo[i] = lo;
    }
  red[q][c] = sum;
  __syncthreads();
  if (a.part && q == 0 && n < a.N)
    a.part[(int64_t)blockIdx.y * a.N + n] = (red[0][c] + red[1][c]) + (red[2][c] + red[3][c]);
}

__global__ __launch_bounds__(256) void k_linear_db(const float* __restrict__ part, int64_t nb, int64_t N,
                                                   float* __restrict__ db, int accumulate, float scale) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (n >= N) return;
  float s = 0.f;
  for (int64_t b = 0; b < nb; ++b) s += part[b * N + n];
  db[n] = (accumulate ? db[n] : 0.f) + scale * s;
}

// ---------------------------------------------------------------- host

static int check_linear(const kt_linear* L, int32_t tokens) {
  if (!L) return set_error(KT_RAWINT4_EINVAL, "linear is NULL");
  if (L->in_features < 8 || L->in_features > 65536 || L->in_features % 8)
    return set_error(KT_RAWINT4_EINVAL, "in_features must be a multiple of 8 in [8, 65536]");
  if (L->out_features < 1 || L->out_features > 65536)
    return set_error(KT_RAWINT4_EINVAL, "out_features must be in [1, 65536]");
  if (L->activation < KT_ACT_NONE || L->activation > KT_ACT_GELU_TANH)
    return set_error(KT_RAWINT4_EINVAL, "activation must be one of KT_ACT_*");
  if (tokens < 0 || tokens > (1 << 20)) return set_error(KT_RAWINT4_EINVAL, "tokens must be in [0, 2^20]");
  if (!L->weight) return set_error(KT_RAWINT4_EINVAL, "weight is NULL");
  if (!is_aligned(L->weight, 16) || !is_aligned(L->bias, 16))
    return set_error(KT_RAWINT4_EINVAL, "weight and bias must be 16-byte aligned");
  return KT_RAWINT4_OK;
}

struct LinearBwdPlan {
  size_t hi, lo, part, x, total;
  int64_t nb;
};

static LinearBwdPlan plan_linear_bwd(const kt_linear* L, int64_t T, bool ckpt) {
  LinearBwdPlan p{};
  const size_t plane = round256(2 * (size_t)T * (size_t)L->out_features);
  p.nb = (T + kDzRows - 1) / kDzRows;
  p.hi = 0;
  p.lo = p.hi + plane;
  p.part = p.lo + plane;
  p.x = p.part + round256(4 * (size_t)p.nb * (size_t)L->out_features);
  p.total = p.x + (ckpt ? round256(2 * (size_t)T * (size_t)L->in_features) : 0);
  return p;
}

template <int KIND>
static void launch_linear(const LinearGemm& g, hipStream_t st) {
  const int64_t blocks = (g.M + 63) / 64 * ((g.N + 63) / 64);
  k_linear<KIND><<<(unsigned)blocks, 256, 0, st>>>(g);
  note_launch();
}

}  // namespace kt

using namespace kt;

extern "C" {

size_t kt_linear_workspace_bytes(const kt_linear* linear, int32_t tokens) {
  if (check_linear(linear, tokens)) return 0;
  (void)set_error(KT_RAWINT4_OK, "");  // 0 is a valid size: no message stays
  return 0;
}

int kt_linear_fwd(const kt_linear* linear, int32_t tokens, const uint16_t* inputs, const uint16_t* residual,
                  void* output, int32_t output_type, uint16_t* preact, void* workspace, size_t workspace_bytes,
                  void* stream) {
  int rc = check_linear(linear, tokens);
  if (rc) return rc;
  if (output_type != KT_TYPE_BF16 && output_type != KT_TYPE_F32)
    return set_error(KT_RAWINT4_EINVAL, "output_type must be KT_TYPE_BF16 or KT_TYPE_F32");
  if (tokens > 0 && (!inputs || !output)) return set_error(KT_RAWINT4_EINVAL, "inputs and output must be non-NULL");
  if (!is_aligned(inputs, 16) || !is_aligned(residual, 16) || !is_aligned(output, 16) || !is_aligned(preact, 16))
    return set_error(KT_RAWINT4_EINVAL, "inputs, residual, output and preact must be 16-byte aligned");
  const int64_t K = linear->in_features, N = linear->out_features;
  (void)workspace;
  (void)workspace_bytes;
  begin_launches();
  if (tokens > 0) {
    LinearGemm g{};
    g.a = inputs;
    g.am = K;
    g.ak = 1;
    g.b = linear->weight;
    g.bn = K;
    g.bk = 1;
    g.M = tokens;
    g.N = N;
    g.K = K;
    g.planes = 1;
    g.bias = linear->bias;
    g.residual = residual;
    g.out = output;
    g.out_f32 = output_type == KT_TYPE_F32;
    g.preact = preact;
    g.act = linear->activation;
    launch_linear<kLinFwd>(g, static_cast<hipStream_t>(stream));
  }
  return finish_launches();
}

size_t kt_linear_bwd_workspace_bytes(const kt_linear* linear, int32_t tokens, int32_t from_checkpoint) {
  if (check_linear(linear, tokens)) return 0;
  (void)set_error(KT_RAWINT4_OK, "");
  return plan_linear_bwd(linear, tokens, from_checkpoint != 0).total;
}

int kt_linear_bwd(const kt_linear* linear, int32_t tokens, const uint16_t* inputs, const kt_ckpt8* checkpoint,
                  const uint16_t* preact, const void* grad_output, int32_t grad_output_type,
                  const uint16_t* grad_residual, uint16_t* grad_input, float* d_weight, float* d_bias,
                  int32_t accumulate, float grad_scale, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_linear(linear, tokens);
  if (rc) return rc;
  if (grad_output_type != KT_TYPE_BF16 && grad_output_type != KT_TYPE_F32)
    return set_error(KT_RAWINT4_EINVAL, "grad_output_type must be KT_TYPE_BF16 or KT_TYPE_F32");
  if (!isfinite(grad_scale)) return set_error(KT_RAWINT4_EINVAL, "grad_scale must be finite");
  if (checkpoint && inputs) return set_error(KT_RAWINT4_EINVAL, "give inputs or a checkpoint, not both");
  if (checkpoint && checkpoint->format != KT_CKPT8_INT8 && checkpoint->format != KT_CKPT8_E4M3)
    return set_error(KT_RAWINT4_EINVAL, "format must be KT_CKPT8_INT8 or KT_CKPT8_E4M3");
  const bool act = linear->activation != KT_ACT_NONE;
  const int64_t T = tokens, K = linear->in_features, N = linear->out_features;
  if (T > 0) {
    if (!grad_output) return set_error(KT_RAWINT4_EINVAL, "grad_output must be non-NULL");
    if (d_weight && !inputs && !(checkpoint && checkpoint->codes && checkpoint->scales))
      return set_error(KT_RAWINT4_EINVAL, "d_weight needs the inputs, as rows or as a checkpoint");
    if (act && !preact) return set_error(KT_RAWINT4_EINVAL, "an activation's backward needs preact");
  }
  if (!is_aligned(inputs, 16) || !is_aligned(preact, 16) || !is_aligned(grad_output, 16) ||
      !is_aligned(grad_residual, 16) || !is_aligned(grad_input, 16) || !is_aligned(d_weight, 16) ||
      !is_aligned(d_bias, 16))
    return set_error(KT_RAWINT4_EINVAL, "tensors must be 16-byte aligned");
  if (checkpoint && (!is_aligned(checkpoint->codes, 4) || !is_aligned(checkpoint->scales, 4)))
    return set_error(KT_RAWINT4_EINVAL, "codes and scales must be 4-byte aligned");
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (T == 0) {
    begin_launches();
    if (!accumulate && d_weight) launch_fill_zero_f32(d_weight, N * K, st);
    if (!accumulate && d_bias) launch_fill_zero_f32(d_bias, N, st);
    return finish_launches();
  }
  const LinearBwdPlan p = plan_linear_bwd(linear, T, checkpoint != nullptr);
  rc = check_caller_workspace(workspace, workspace_bytes, p.total);
  if (rc) return rc;
  begin_launches();
  // a bf16 grad_output without activation is dz itself
  const bool direct = !act && grad_output_type == KT_TYPE_BF16;
  const uint16_t* dz = static_cast<const uint16_t*>(grad_output);
  if (!direct || d_bias) {
    DzArgs a{};
    a.dy = grad_output;
    a.dy_f32 = grad_output_type == KT_TYPE_F32;
    a.z = preact;
    a.act = linear->activation;
    a.T = T;
    a.N = N;
    a.hi = direct ? nullptr : ws_ptr<uint16_t>(workspace, p.hi);
    a.lo = direct || !d_weight ? nullptr : ws_ptr<uint16_t>(workspace, p.lo);
    a.part = d_bias ? ws_ptr<float>(workspace, p.part) : nullptr;
    k_linear_dz<<<dim3((unsigned)((N + 63) / 64), (unsigned)p.nb), 256, 0, st>>>(a);
    note_launch();
    if (!direct) dz = a.hi;
    if (d_bias) {
      k_linear_db<<<(unsigned)((N + 255) / 256), 256, 0, st>>>(a.part, p.nb, N, d_bias, accumulate, grad_scale);
      note_launch();
    }
  }
  LinearGemm g{};
  if (grad_input) {
    g.a = dz;
    g.am = N;
    g.ak = 1;
    g.b = linear->weight;
    g.bn = 1;
    g.bk = K;
    g.M = T;
    g.N = K;
    g.K = N;
    g.planes = 1;
    g.residual = grad_residual;
    g.out = grad_input;
    launch_linear<kLinDx>(g, st);
  }
  if (d_weight) {
    const uint16_t* x = inputs;
    if (checkpoint) {
      uint16_t* rows = ws_ptr<uint16_t>(workspace, p.x);
      launch_ckpt8_unpack(checkpoint->codes, checkpoint->scales, T, K, checkpoint->format, rows, st);
      x = rows;
    }
    g = LinearGemm{};
    g.a = dz;
    g.am = 1;
    g.ak = N;
    g.b = x;
    g.bn = 1;
    g.bk = K;
    g.M = N;
    g.N = K;
    g.K = T;
    g.planes = direct ? 1 : 2;
    g.a_plane = (int64_t)(p.lo - p.hi) / 2;
    g.out = d_weight;
    g.accumulate = accumulate;
    g.scale = grad_scale;
    launch_linear<kLinDw>(g, st);
  }
  return finish_launches();
}

}  // extern "C"
