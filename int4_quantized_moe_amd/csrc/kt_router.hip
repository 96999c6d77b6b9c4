// Routing of tokens to experts: scores, the choice of top_k experts (bias for
// balance, groups), their weights, the gradient with respect to the logits, the
// load per expert and the bias's balance rule.
//
// The choice is made on c = s + b to 64 bits, ties to the lower index, so that
// it is the formula's choice and not one of fp32 roundings: with a few hundred
// experts some tokens of every long batch have two candidates whose c differ
// by less than an fp32 rounding.
#include <math.h>

#include "kt_common.hpp"
#include "kt_internal.hpp"

namespace kt {

struct RouterArgs {
  int E, k, G, per, top_groups, group_top;
  int renorm;
  float scale;
  const void* logits;
  const float* bias;
  const uint8_t* mask;
  int64_t* ids;
  float* w;
};

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if (BF16) return bf16_to_float(static_cast<const uint16_t*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }
__device__ __forceinline__ bool is_nan(float v) { return v != v; }

// Whether a logit makes its row undefined (NaN scores).
template <int SCORE>
__device__ __forceinline__ bool bad_logit(float l) {
  return is_nan(l) || (SCORE == KT_SCORE_SOFTMAX && l == INFINITY);
}

// ---------------------------------------------------------------- any size

constexpr int kAnyThreads = 256;

// (value, index) pairs in the order of choice: larger value, then lower index.
__device__ __forceinline__ bool better(double a, int ia, double b, int ib) { return a > b || (a == b && ia < ib); }

__device__ __forceinline__ void wave_best(double& v, int& i) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const double ov = __shfl_xor(v, off);
    const int oi = __shfl_xor(i, off);
    if (better(ov, oi, v, i)) {
      v = ov;
      i = oi;
    }
  }
}

// One block per token, c of every expert in LDS, top_k rounds of the block's
// best.  Takes any E, k and group shape.
template <int SCORE, bool BF16>
__global__ __launch_bounds__(kAnyThreads) void k_route_any(RouterArgs a) {
  __shared__ double c[KT_RAWINT4_MAX_EXPERTS];
  __shared__ double red_v[4];
  __shared__ int red_i[4];
  __shared__ double gscore[KT_ROUTER_MAX_GROUPS];
  __shared__ uint8_t gkeep[KT_ROUTER_MAX_GROUPS];
  __shared__ double sum_s;
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int64_t* ids = a.ids + t * a.k;
  float* w = a.w + t * a.k;
  if (a.mask && !a.mask[t]) {
    for (int j = tid; j < a.k; j += kAnyThreads) {
      ids[j] = -1;
      w[j] = 0.f;
    }
    return;
  }
  const int64_t base = t * a.E;
  int bad = 0;
  float mx = -INFINITY;
  for (int e = tid; e < a.E; e += kAnyThreads) {
    const float l = load_logit<BF16>(a.logits, base + e);
    const float b = a.bias ? a.bias[e] : 0.f;
    bad |= bad_logit<SCORE>(l) || is_nan(b) || b == INFINITY;
    mx = fmaxf(mx, l);
  }
  if (__syncthreads_or(bad)) {
    for (int j = tid; j < a.k; j += kAnyThreads) {
      ids[j] = j;
      w[j] = __uint_as_float(0x7fc00000u);
    }
    return;
  }
  double z = 1.0, m = 0.0;
  if (SCORE == KT_SCORE_SOFTMAX) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
    if (lane == 0) red_v[wave] = mx;
    __syncthreads();
    m = fmax(fmax(red_v[0], red_v[1]), fmax(red_v[2], red_v[3]));
    __syncthreads();
    if (m == -INFINITY) m = 0.0;  // no expert left: every s is 0
    double part = 0.0;
    for (int e = tid; e < a.E; e += kAnyThreads) part += exp((double)load_logit<BF16>(a.logits, base + e) - m);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) part += __shfl_xor(part, off);
    if (lane == 0) red_v[wave] = part;
    __syncthreads();
    z = (red_v[0] + red_v[1]) + (red_v[2] + red_v[3]);
    __syncthreads();
  }
  auto score = [&](float l) { return SCORE == KT_SCORE_SOFTMAX ? exp((double)l - m) / z : sigmoid64((double)l); };
  for (int e = tid; e < a.E; e += kAnyThreads) {
    const float l = load_logit<BF16>(a.logits, base + e);
    const float b = a.bias ? a.bias[e] : 0.f;
    c[e] = l == -INFINITY || b == -INFINITY ? -INFINITY : score(l) + (double)b;
  }
  if (tid == 0) sum_s = 0.0;
  __syncthreads();
  if (a.G > 1) {
    for (int g = wave; g < a.G; g += 4) {
      double v1 = -INFINITY, v2 = -INFINITY;
      for (int e = g * a.per + lane; e < (g + 1) * a.per; e += 64) {
        const double v = c[e];
        v2 = fmax(v2, fmin(v1, v));
        v1 = fmax(v1, v);
      }
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const double o1 = __shfl_xor(v1, off), o2 = __shfl_xor(v2, off);
        v2 = fmax(fmin(v1, o1), fmax(v2, o2));
        v1 = fmax(v1, o1);
      }
      if (lane == 0) gscore[g] = a.group_top == 2 ? v1 + v2 : v1;
    }
    __syncthreads();
    if (tid < a.G) {
      int rank = 0;
      for (int g = 0; g < a.G; ++g) rank += better(gscore[g], g, gscore[tid], tid);
      gkeep[tid] = rank < a.top_groups;
    }
    __syncthreads();
    for (int e = tid; e < a.E; e += kAnyThreads)
      if (!gkeep[e / a.per]) c[e] = -INFINITY;
    __syncthreads();
  }
  // each thread keeps the best of its experts tid, tid + 256, ...
  double bv = -INFINITY;
  int bi = a.E;
  auto rescan = [&] {
    bv = -INFINITY;
    bi = a.E;
    for (int e = tid; e < a.E; e += kAnyThreads)
      if (better(c[e], e, bv, bi) && c[e] > -INFINITY) {
        bv = c[e];
        bi = e;
      }
  };
  rescan();
  int j = 0;
  for (; j < a.k; ++j) {
    double v = bv;
    int i = bi;
    wave_best(v, i);
    if (lane == 0) {
      red_v[wave] = v;
      red_i[wave] = i;
    }
    __syncthreads();
    v = red_v[0];
    i = red_i[0];
    for (int q = 1; q < 4; ++q)
      if (better(red_v[q], red_i[q], v, i)) {
        v = red_v[q];
        i = red_i[q];
      }
    __syncthreads();
    if (i >= a.E) break;  // nothing left to choose (the same in every thread)
    if (i == bi) {
      const double s = score(load_logit<BF16>(a.logits, base + i));
      ids[j] = i;
      w[j] = (float)s;
      sum_s += s;
      c[i] = -INFINITY;
      rescan();
    }
    __syncthreads();  // before the next round's owner adds to sum_s
  }
  const float mul = a.renorm ? (float)((double)a.scale / (sum_s + 1e-20)) : a.scale;
  for (int q = tid; q < a.k; q += kAnyThreads) {
    if (q < j) {
      w[q] *= mul;
    } else {
      ids[q] = -1;
      w[q] = 0.f;
    }
  }
}

// ---------------------------------------------------------------- gradient, any size

struct RouterBwdArgs {
  int E, k;
  int renorm;
  float scale;
  const void* logits;
  const int64_t* ids;
  const float* g;
  void* out;
};

template <bool BF16>
__device__ __forceinline__ void store_grad(void* p, int64_t i, float v) {
  if (BF16)
    static_cast<uint16_t*>(p)[i] = float_to_bf16(v);
  else
    static_cast<float*>(p)[i] = v;
}

// Sigmoid and softmax in fp32 with the library's exponential (about one rounding).
__device__ __forceinline__ float sigmoid32(float l) { return 1.f / (1.f + expf(-l)); }

// With p = s / S the gradient of the chosen scores is ds = scale (g - d) / S,
// and the softmax's sum ds s is scale d (1 - sum s / S) / S = scale d 1e-20 / S^2:
// written so, the tiny term keeps its value instead of a difference of roundings.
struct RowGrad {
  float m, zinv;       // softmax: maximum and 1 / sum of exponentials
  float inv, d, dot;   // 1 / S (1 without renormalisation), d, sum ds s
};

// ds of a chosen expert with score gradient g
__device__ __forceinline__ float chosen_ds(const RouterBwdArgs& a, const RowGrad& r, float g) {
  return a.renorm ? a.scale * (g - r.d) * r.inv : a.scale * g;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off);
  return v;
}

// One block per token; ds of every expert in LDS.  Each thread owns the experts
// tid, tid + 256, ... and adds their slots in slot order.
template <int SCORE, bool BF16>
__global__ __launch_bounds__(kAnyThreads) void k_route_bwd_any(RouterBwdArgs a) {
  __shared__ float ds[KT_RAWINT4_MAX_EXPERTS];
  __shared__ float red[4], red2[4], red3[4];
  __shared__ int sid[kAnyThreads];
  __shared__ float sg[kAnyThreads];
  const int64_t t = blockIdx.x, base = t * a.E;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t* ids = a.ids + t * a.k;
  const float* g = a.g + t * a.k;
  int bad = 0;
  float mx = -INFINITY;
  for (int e = tid; e < a.E; e += kAnyThreads) {
    const float l = load_logit<BF16>(a.logits, base + e);
    bad |= bad_logit<SCORE>(l);
    mx = fmaxf(mx, l);
    ds[e] = 0.f;
  }
  bad = __syncthreads_or(bad);
  auto block_sum = [&](float v, float* buf) {
    v = wave_sum(v);
    if (lane == 0) buf[wave] = v;
    __syncthreads();
    return (buf[0] + buf[1]) + (buf[2] + buf[3]);
  };
  RowGrad r{0.f, 1.f, 1.f, 0.f, 0.f};
  if (SCORE == KT_SCORE_SOFTMAX) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
    if (lane == 0) red[wave] = mx;
    __syncthreads();
    r.m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    if (r.m == -INFINITY) r.m = 0.f;
    float part = 0.f;
    for (int e = tid; e < a.E; e += kAnyThreads) part += expf(load_logit<BF16>(a.logits, base + e) - r.m);
    const float z = block_sum(part, red2);
    r.zinv = z > 0.f ? 1.f / z : 0.f;
    __syncthreads();
  }
  auto score = [&](float l) { return SCORE == KT_SCORE_SOFTMAX ? expf(l - r.m) * r.zinv : sigmoid32(l); };
  float ssum = 0.f, gsum = 0.f, used = 0.f;
  for (int j = tid; j < a.k; j += kAnyThreads) {
    const int64_t id = ids[j];
    if (id >= 0 && id < a.E) {
      const float s = score(load_logit<BF16>(a.logits, base + id));
      ssum += s;
      gsum += g[j] * s;
      used = 1.f;
    }
  }
  ssum = block_sum(ssum, red);
  gsum = block_sum(gsum, red2);
  used = block_sum(used, red3);
  if (used == 0.f) bad = 0;
  if (a.renorm) {
    const float S = ssum + 1e-20f;
    r.inv = 1.f / S;
    r.d = gsum * r.inv;
    r.dot = a.scale * r.d * (1e-20f * r.inv);
  } else {
    r.dot = a.scale * gsum;
  }
  for (int j0 = 0; j0 < a.k; j0 += kAnyThreads) {
    __syncthreads();
    const int64_t id = j0 + tid < a.k ? ids[j0 + tid] : -1;
    sid[tid] = id >= 0 && id < a.E ? (int)id : -1;
    sg[tid] = j0 + tid < a.k ? g[j0 + tid] : 0.f;
    __syncthreads();
    const int n = min(kAnyThreads, a.k - j0);
    for (int j = 0; j < n; ++j)
      if (sid[j] >= 0 && (sid[j] & (kAnyThreads - 1)) == tid) ds[sid[j]] += chosen_ds(a, r, sg[j]);
  }
  for (int e = tid; e < a.E; e += kAnyThreads) {
    const float s = score(load_logit<BF16>(a.logits, base + e));
    float v = SCORE == KT_SCORE_SOFTMAX ? s * (ds[e] - (used == 0.f ? 0.f : r.dot)) : ds[e] * s * (1.f - s);
    if (used == 0.f) v = 0.f;
    if (bad) v = __uint_as_float(0x7fc00000u);
    store_grad<BF16>(a.out, base + e, v);
  }
}

// ---------------------------------------------------------------- load and bias

// One block: load = (accumulate ? load : 0) + slots per expert, counted in LDS.
__global__ __launch_bounds__(1024) void k_route_load_one(const int64_t* __restrict__ ids, int64_t n, int E,
                                                         int accumulate, int32_t* __restrict__ load) {
  __shared__ int32_t hist[KT_RAWINT4_MAX_EXPERTS];
  for (int e = threadIdx.x; e < E; e += 1024) hist[e] = 0;
  __syncthreads();
  for (int64_t i = threadIdx.x; i < n; i += 1024) {
    const int64_t e = ids[i];
    if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 1024) load[e] = (accumulate ? load[e] : 0) + hist[e];
}

__global__ __launch_bounds__(256) void k_zero_i32(int32_t* p, int n) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0;
}

// Several blocks (whole numbers: the order of the atomic sums does not matter).
__global__ __launch_bounds__(256) void k_route_load(const int64_t* __restrict__ ids, int64_t n, int E,
                                                    int32_t* __restrict__ load) {
  __shared__ int32_t hist[KT_RAWINT4_MAX_EXPERTS];
  for (int e = threadIdx.x; e < E; e += 256) hist[e] = 0;
  __syncthreads();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t e = ids[i];
    if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 256)
    if (hist[e]) atomicAdd(&load[e], hist[e]);
}

__global__ __launch_bounds__(1024) void k_route_bias(float* __restrict__ bias, const int32_t* __restrict__ load,
                                                     int E, float rate) {
  __shared__ int64_t part[16];
  int64_t sum = 0;
  for (int e = threadIdx.x; e < E; e += 1024) sum += load[e];
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) sum += __shfl_xor(sum, off);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  sum = 0;
  for (int q = 0; q < 16; ++q) sum += part[q];
  for (int e = threadIdx.x; e < E; e += 1024) {
    const int64_t mine = (int64_t)load[e] * E;
    if (mine < sum) bias[e] += rate;
    if (mine > sum) bias[e] -= rate;
  }
}

// ---------------------------------------------------------------- host

static int check_router(const kt_router* r, int32_t tokens) {
  if (!r) return set_error(KT_RAWINT4_EINVAL, "router is NULL");
  if (r->num_experts < 1 || r->num_experts > KT_RAWINT4_MAX_EXPERTS)
    return set_error(KT_RAWINT4_EINVAL, "num_experts must be in [1, 8192]");
  if (r->top_k < 1 || r->top_k > r->num_experts)
    return set_error(KT_RAWINT4_EINVAL, "top_k must be in [1, num_experts]");
  if (r->num_groups < 1 || r->num_groups > KT_ROUTER_MAX_GROUPS || r->num_experts % r->num_groups)
    return set_error(KT_RAWINT4_EINVAL, "num_groups must be in [1, 64] and divide num_experts");
  const int per = r->num_experts / r->num_groups;
  if (r->top_groups < 1 || r->top_groups > r->num_groups)
    return set_error(KT_RAWINT4_EINVAL, "top_groups must be in [1, num_groups]");
  if (r->group_top < 1 || r->group_top > 2 || r->group_top > per)
    return set_error(KT_RAWINT4_EINVAL, "group_top must be 1 or 2 and at most the experts of a group");
  if (r->top_k > r->top_groups * per)
    return set_error(KT_RAWINT4_EINVAL, "top_k must be at most the experts of top_groups groups");
  if (r->score != KT_SCORE_SOFTMAX && r->score != KT_SCORE_SIGMOID)
    return set_error(KT_RAWINT4_EINVAL, "score must be KT_SCORE_SOFTMAX or KT_SCORE_SIGMOID");
  if (r->logits_type != KT_TYPE_F32 && r->logits_type != KT_TYPE_BF16)
    return set_error(KT_RAWINT4_EINVAL, "logits_type must be KT_TYPE_F32 or KT_TYPE_BF16");
  if (!isfinite(r->scale)) return set_error(KT_RAWINT4_EINVAL, "scale must be finite");
  if (tokens < 0) return set_error(KT_RAWINT4_EINVAL, "tokens must be non-negative");
  if (tokens > (1 << 23)) return set_error(KT_RAWINT4_EINVAL, "tokens must be at most 2^23 a call");
  return KT_RAWINT4_OK;
}

template <int SCORE, bool BF16>
static void launch_route(const RouterArgs& a, int tokens, hipStream_t st) {
  k_route_any<SCORE, BF16><<<(unsigned)tokens, kAnyThreads, 0, st>>>(a);
  note_launch();
}

template <int SCORE, bool BF16>
static void launch_route_bwd(const RouterBwdArgs& a, int tokens, hipStream_t st) {
  k_route_bwd_any<SCORE, BF16><<<(unsigned)tokens, kAnyThreads, 0, st>>>(a);
  note_launch();
}

static void launch_load(const int64_t* ids, int64_t n, int E, int accumulate, int32_t* load, hipStream_t st) {
  if (n <= 16384) {
    k_route_load_one<<<1, 1024, 0, st>>>(ids, n, E, accumulate, load);
    note_launch();
    return;
  }
  if (!accumulate) {
    k_zero_i32<<<(unsigned)((E + 255) / 256), 256, 0, st>>>(load, E);
    note_launch();
  }
  const int64_t blocks = (n + 4095) / 4096;
  k_route_load<<<(unsigned)(blocks < 256 ? blocks : 256), 256, 0, st>>>(ids, n, E, load);
  note_launch();
}

}  // namespace kt

using namespace kt;

extern "C" {

int kt_router_fwd(const kt_router* router, int32_t tokens, const void* logits, const float* bias,
                  const uint8_t* token_mask, int64_t* expert_ids, float* route_weights, int32_t* load,
                  int32_t accumulate, void* stream) {
  const int rc = check_router(router, tokens);
  if (rc) return rc;
  if (tokens > 0 && (!logits || !expert_ids || !route_weights))
    return set_error(KT_RAWINT4_EINVAL, "logits, expert_ids and route_weights must be non-NULL");
  if (!is_aligned(logits, 16) || !is_aligned(bias, 4) || !is_aligned(expert_ids, 8) || !is_aligned(route_weights, 4) ||
      !is_aligned(load, 4))
    return set_error(KT_RAWINT4_EINVAL, "logits must be 16-byte aligned, expert_ids 8-byte aligned");
  hipStream_t st = static_cast<hipStream_t>(stream);
  RouterArgs a{router->num_experts, router->top_k,     router->num_groups, router->num_experts / router->num_groups,
               router->top_groups,  router->group_top, router->renormalize != 0, router->scale,
               logits,              bias,              token_mask,         expert_ids,
               route_weights};
  if (a.top_groups == a.G) a.G = 1;  // every group stays
  begin_launches();
  if (tokens > 0) {
    const bool bf = router->logits_type == KT_TYPE_BF16, soft = router->score == KT_SCORE_SOFTMAX;
    if (soft && bf)
      launch_route<KT_SCORE_SOFTMAX, true>(a, tokens, st);
    else if (soft)
      launch_route<KT_SCORE_SOFTMAX, false>(a, tokens, st);
    else if (bf)
      launch_route<KT_SCORE_SIGMOID, true>(a, tokens, st);
    else
      launch_route<KT_SCORE_SIGMOID, false>(a, tokens, st);
  }
  if (load) launch_load(expert_ids, (int64_t)tokens * a.k, a.E, accumulate, load, st);
  return finish_launches();
}

int kt_router_bwd(const kt_router* router, int32_t tokens, const void* logits, const int64_t* expert_ids,
                  const float* grad_route, void* grad_logits, void* stream) {
  const int rc = check_router(router, tokens);
  if (rc) return rc;
  if (tokens > 0 && (!logits || !expert_ids || !grad_route || !grad_logits))
    return set_error(KT_RAWINT4_EINVAL, "logits, expert_ids, grad_route and grad_logits must be non-NULL");
  if (!is_aligned(logits, 16) || !is_aligned(grad_logits, 16) || !is_aligned(expert_ids, 8) ||
      !is_aligned(grad_route, 4))
    return set_error(KT_RAWINT4_EINVAL, "logits and grad_logits must be 16-byte aligned, expert_ids 8-byte aligned");
  hipStream_t st = static_cast<hipStream_t>(stream);
  const RouterBwdArgs a{router->num_experts, router->top_k, router->renormalize != 0, router->scale,
                        logits,              expert_ids,    grad_route,               grad_logits};
  begin_launches();
  if (tokens > 0) {
    const bool bf = router->logits_type == KT_TYPE_BF16, soft = router->score == KT_SCORE_SOFTMAX;
    if (soft && bf)
      launch_route_bwd<KT_SCORE_SOFTMAX, true>(a, tokens, st);
    else if (soft)
      launch_route_bwd<KT_SCORE_SOFTMAX, false>(a, tokens, st);
    else if (bf)
      launch_route_bwd<KT_SCORE_SIGMOID, true>(a, tokens, st);
    else
      launch_route_bwd<KT_SCORE_SIGMOID, false>(a, tokens, st);
  }
  return finish_launches();
}

int kt_router_update_bias(float* bias, const int32_t* load, int32_t num_experts, float rate, void* stream) {
  if (num_experts < 1 || num_experts > KT_RAWINT4_MAX_EXPERTS)
    return set_error(KT_RAWINT4_EINVAL, "num_experts must be in [1, 8192]");
  if (!bias || !load) return set_error(KT_RAWINT4_EINVAL, "bias and load must be non-NULL");
  if (!is_aligned(bias, 4) || !is_aligned(load, 4))
    return set_error(KT_RAWINT4_EINVAL, "bias and load must be 4-byte aligned");
  if (!isfinite(rate)) return set_error(KT_RAWINT4_EINVAL, "rate must be finite");
  begin_launches();
  k_route_bias<<<1, 1024, 0, static_cast<hipStream_t>(stream)>>>(bias, load, num_experts, rate);
  return finish_launches();
}

}  // extern "C"
