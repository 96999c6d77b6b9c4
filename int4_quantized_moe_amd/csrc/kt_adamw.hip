// AdamW over many tensors at once, with states in 32 bits or in 8, and the
// gradients' global norm.
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,  p = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Bound by memory: a value's parameter, gradient and states are read and written once, 28
// bytes in fp32, 16 with 8-bit states, 30 for a bf16 parameter with a master; clipping reads the gradients once
// before.  So one launch takes the chunks of up to 32 tensors, whatever their sizes, a wave has all its
// loads in flight before the first is used, and what the whole step shares (the steps made, the
// clipping, both bias corrections) is worked out once, by a kernel of one workgroup.
// 170 million values: fp32 with clipping 1012 us, 5.4 TB/s of 32 bytes a value; 8-bit states 492 us, 5.5
// TB/s, where instructions bind as well (vector ones about 90% busy; on bf16 parameters and gradients 392 us, 4.4
// TB/s); 47 million bf16 ones with masters 265 us, 5.3 TB/s (a copy of 1 GiB: 4.9 to 5.1).
// Six small tensors: 10 to 11 us, 7.4 of them on the GPU (2.4 for what is shared, 5.0); 360 of them 141 us, which is
// the host's, 86 in a graph (13 kernels; floor 58).
#include "kt_step_common.hpp"

#include <math.h>

// Products and sums are rounded one by one, as written.
#pragma clang fp contract(off)

namespace kt {

constexpr int kAdamPerLaunch = 32;  // tensors in a launch's arguments
constexpr int kAdamUnits = 4;       // blocks of 256 values a wave takes
constexpr int kAdamChunk = 4 * kAdamUnits * KT_ADAMW_BLOCK;  // values of a workgroup
constexpr int kNormBlocks = 1024;  // of the norm, a launch
constexpr int64_t kAdamLaunch = 1 << 20;  // chunks a launch of the update takes: more of them in several (a launch has fewer than 2^32 threads)
static_assert(kAdamLaunch * 256 < (int64_t)1 << 32, "threads of a launch");
constexpr float kTiny = 0x1p-100f;

struct AdamTensor {
  void* p;
  float* master;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t n;
  int64_t first;  // its first chunk
  uint8_t p_f32, g_f32, decay;
};

// What a step's kernels read, made by k_adamw_begin at the head of the workspace.
struct AdamControl {
  float grad_mult, step_size, inv_root_c2, decay;
  int32_t skip;
};

struct AdamArgs {
  const AdamControl* ctl;
  int64_t chunks;
  int64_t from;  // the launch's first chunk
  int count;
  float b1, b1c, b2, b2c, eps;
  double* part;
  AdamTensor t[kAdamPerLaunch];
};

// The tensor of a chunk, by a lane a tensor (one after another, a load each would wait for the last).
__device__ __forceinline__ int find_tensor(const AdamArgs& a, int64_t chunk) {
  const int lane = threadIdx.x & 63, last = a.count - 1;
  const bool before = a.t[lane < last ? lane : last].first <= chunk && lane <= last;
  return __popcll(__ballot(before)) - 1;
}

// four values from i on; those behind n are 0
__device__ __forceinline__ float4 load4(const void* p, bool f32, int64_t i, int64_t n) {
  float4 r = {0, 0, 0, 0};
  if (i + 4 <= n) {
    if (f32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const u32pair w = *reinterpret_cast<const u32pair*>(static_cast<const uint16_t*>(p) + i);
    return float4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                  __uint_as_float(w.y & 0xffff0000u)};
  }
  float* f = &r.x;
  for (int j = 0; j < 4; ++j)
    if (i + j < n) f[j] = f32 ? static_cast<const float*>(p)[i + j] : bf16_to_float(static_cast<const uint16_t*>(p)[i + j]);
  return r;
}
__device__ __forceinline__ void store4(void* p, bool f32, int64_t i, int64_t n, float4 v) {
  if (i + 4 <= n) {
    if (f32)
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = v;
    else
      *reinterpret_cast<u32pair*>(static_cast<uint16_t*>(p) + i) =
          u32pair{bf16_pair(v.x, v.y), bf16_pair(v.z, v.w)};
    return;
  }
  const float f[4] = {v.x, v.y, v.z, v.w};
  for (int j = 0; j < 4; ++j)
    if (i + j < n) {
      if (f32)
        static_cast<float*>(p)[i + j] = f[j];
      else
        static_cast<uint16_t*>(p)[i + j] = float_to_bf16(f[j]);
    }
}

__device__ __forceinline__ uint32_t load_codes(const void* p, int64_t i, int64_t n) {
  const uint8_t* b = static_cast<const uint8_t*>(p) + i;
  if (i + 4 <= n) return *reinterpret_cast<const uint32_t*>(b);
  uint32_t w = 0;
  for (int j = 0; j < 4; ++j)
    if (i + j < n) w |= (uint32_t)b[j] << (8 * j);
  return w;
}
__device__ __forceinline__ void store_codes(void* p, int64_t i, int64_t n, uint32_t w) {
  uint8_t* b = static_cast<uint8_t*>(p) + i;
  if (i + 4 <= n) {
    *reinterpret_cast<uint32_t*>(b) = w;
    return;
  }
  for (int j = 0; j < 4; ++j)
    if (i + j < n) b[j] = (uint8_t)(w >> (8 * j));
}

__device__ __forceinline__ float4 decode4(uint32_t w) {
  const float2_t a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  return float4{a.x, a.y, b.x, b.y};
}
__device__ __forceinline__ uint32_t codes4(const float* f) {
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w, true);
}
__device__ __forceinline__ float most4(const float* f) {
  return wave_max(fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3]))));
}

// Codes of a block's values and their scale; ROOT: not negative, and positive ones keep a code that is not 0.
template <bool ROOT>
__device__ __forceinline__ uint32_t encode4(const float* v, float& scale) {
  const float amax = most4(v);
  const bool some = !(amax < kTiny);
  const float inv = some ? 448.f * (1.f / amax) : 0.f;
  scale = some ? amax * (1.f / 448.f) : 0.f;
  float f[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float w = v[j] * inv;
    if (ROOT && some && v[j] > 0.f) w = fmaxf(w, 0x1p-9f);
    // (a NaN keeps its place: comparisons with it are false)
    f[j] = w > 448.f ? 448.f : w < -448.f ? -448.f : w;
  }
  return codes4(f);
}

// A lane's four values of a block as they lie in memory; the types are known where
// it is compiled, so that loads in flight are (fp32 with clipping 1042 -> 1010 us, bf16 with masters 273 -> 262).  P: the parameter is 0: bf16, 1: fp32, 2: bf16 with an fp32 master.
template <int P, bool GF32, bool E8, bool WHOLE>
struct AdamValues {
  float4 g, p, m, v;
  u32pair gw, pw;
  uint32_t mw, vw;
  float ms, vs;
  __device__ __forceinline__ void load(const AdamTensor& t, int64_t block, int64_t i) {
    const int64_t n = WHOLE ? INT64_MAX : t.n;
    if (!WHOLE) {
      g = load4(t.g, GF32, i, n);
      p = load4(P == 2 ? t.master : t.p, P != 0, i, n);
    } else {
      if (GF32) g = *reinterpret_cast<const float4*>(static_cast<const float*>(t.g) + i);
      if (!GF32) gw = *reinterpret_cast<const u32pair*>(static_cast<const uint16_t*>(t.g) + i);
      if (P != 0) p = *reinterpret_cast<const float4*>(static_cast<const float*>(P == 2 ? t.master : t.p) + i);
      if (P == 0) pw = *reinterpret_cast<const u32pair*>(static_cast<const uint16_t*>(t.p) + i);
    }
    if (E8) {
      const int64_t s = block / KT_ADAMW_BLOCK;
      mw = load_codes(t.m, i, n), ms = t.ms[s];
      vw = load_codes(t.v, i, n), vs = t.vs[s];
    } else {
      m = load4(t.m, true, i, n);
      v = load4(t.v, true, i, n);
    }
  }
  __device__ __forceinline__ void widen() {
    if (WHOLE && !GF32) g = wide(gw);
    if (WHOLE && P == 0) p = wide(pw);
    if (E8) m = decode4(mw), v = decode4(vw);
  }
  static __device__ __forceinline__ float4 wide(u32pair w) {
    return float4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u)};
  }
};

template <int P, bool GF32, bool E8, bool WHOLE>
__device__ __forceinline__ void adam_block(const AdamArgs& a, const AdamControl& ctl, const AdamTensor& t, float decay, int64_t block,
                                           int64_t i, AdamValues<P, GF32, E8, WHOLE>& x) {
  const int64_t n = WHOLE ? INT64_MAX : t.n;
  x.widen();
  float *pf = &x.p.x, *mf = &x.m.x, *vf = &x.v.x, root[4];
  const float* gf = &x.g.x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float g = gf[j] * ctl.grad_mult;
    if (E8) {
      mf[j] = mf[j] * x.ms;
      vf[j] = vf[j] * x.vs;
      vf[j] = vf[j] * vf[j];
    }
    mf[j] = a.b1 * mf[j] + a.b1c * g;
    vf[j] = a.b2 * vf[j] + a.b2c * (g * g);
    root[j] = sqrtf(vf[j]);
    pf[j] = pf[j] * decay - ctl.step_size * mf[j] / (root[j] * ctl.inv_root_c2 + a.eps);
  }
  if (P == 2) store4(t.master, true, i, n, x.p);
  store4(t.p, P == 1, i, n, x.p);
  if (E8) {
    float ms, vs;
    store_codes(t.m, i, n, encode4<false>(mf, ms));
    store_codes(t.v, i, n, encode4<true>(root, vs));
    const int64_t s = block / KT_ADAMW_BLOCK;
    if ((threadIdx.x & 63) == 0) t.ms[s] = ms, t.vs[s] = vs;
  } else {
    store4(t.m, true, i, n, x.m);
    store4(t.v, true, i, n, x.v);
  }
}

// A wave's blocks of a chunk: all loads of whole ones first.
template <int P, bool GF32, bool E8>
__device__ __forceinline__ void adam_chunk(const AdamArgs& a, const AdamControl& ctl, const AdamTensor& t, int64_t base) {
  const int lane = threadIdx.x & 63;
  const float decay = t.decay ? ctl.decay : 1.f;
  constexpr int64_t kStep = 4 * KT_ADAMW_BLOCK;
  if (base + (kAdamUnits - 1) * kStep + KT_ADAMW_BLOCK <= t.n) {
    AdamValues<P, GF32, E8, true> x[kAdamUnits];
#pragma unroll
    for (int u = 0; u < kAdamUnits; ++u) x[u].load(t, base + u * kStep, base + u * kStep + lane * 4);
#pragma unroll
    for (int u = 0; u < kAdamUnits; ++u) {
      __builtin_amdgcn_sched_barrier(0);
      adam_block(a, ctl, t, decay, base + u * kStep, base + u * kStep + lane * 4, x[u]);
    }
    return;
  }
#pragma unroll 1
  for (int64_t block = base; block < t.n && block < base + kAdamUnits * kStep; block += kStep) {
    AdamValues<P, GF32, E8, false> x;
    x.load(t, block, block + lane * 4);
    adam_block(a, ctl, t, decay, block, block + lane * 4, x);
  }
}

// (Three waves a SIMD: with more, reads and writes of more places are mixed in memory; 8-bit states, fp32
// parameters and gradients: 491 us, with 4 506, with 6 527, with 2 525; both bf16 398, 393, 380, 463.)
template <bool E8>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(3, 3))) void k_adamw(AdamArgs a) {
  const AdamControl ctl = *a.ctl;
  const int64_t chunk = a.from + blockIdx.x;
  const AdamTensor& t = a.t[find_tensor(a, chunk)];
  if (ctl.skip) return;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t base = (chunk - t.first) * kAdamChunk + wave * KT_ADAMW_BLOCK;
  if (t.p_f32)
    t.g_f32 ? adam_chunk<1, true, E8>(a, ctl, t, base) : adam_chunk<1, false, E8>(a, ctl, t, base);
  else if (t.master)
    t.g_f32 ? adam_chunk<2, true, E8>(a, ctl, t, base) : adam_chunk<2, false, E8>(a, ctl, t, base);
  else
    t.g_f32 ? adam_chunk<0, true, E8>(a, ctl, t, base) : adam_chunk<0, false, E8>(a, ctl, t, base);
}

// Sums of squares of the gradients in 64 bits: a partial sum a block, each over
// chunks a grid apart, joined by k_adamw_begin in the blocks' order.
__global__ __launch_bounds__(256) void k_grad_squares(AdamArgs a) {
  __shared__ double red[4];
  double s = 0.0;
  for (int64_t chunk = blockIdx.x; chunk < a.chunks; chunk += gridDim.x) {
    const AdamTensor& t = a.t[find_tensor(a, chunk)];
    const int64_t base = (chunk - t.first) * kAdamChunk + threadIdx.x * 4;
#pragma unroll
    for (int u = 0; u < kAdamUnits; ++u) {
      const float4 g = load4(t.g, t.g_f32, base + u * 1024, t.n);
      s += (double)g.x * g.x;
      s += (double)g.y * g.y;
      s += (double)g.z * g.z;
      s += (double)g.w * g.w;
    }
  }
  for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) a.part[blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

struct AdamBegin {
  AdamControl* ctl;
  const double* part;
  int parts;
  int64_t* step;
  float* norm;
  const float* lr_ptr;
  double lr, beta1, beta2, decay, max_norm, grad_scale;
};
__global__ __launch_bounds__(256) void k_adamw_begin(AdamBegin a) {
  __shared__ double red[256];
  double s = 0.0;
  for (int i = threadIdx.x; i < a.parts; i += 256) s += a.part[i];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int d = 128; d > 0; d >>= 1) {
    if ((int)threadIdx.x < d) red[threadIdx.x] += red[threadIdx.x + d];
    __syncthreads();
  }
  if (threadIdx.x) return;
  double mult = a.grad_scale;
  bool skip = false;
  if (a.norm) {
    const double norm = sqrt(red[0]) * fabs(a.grad_scale);
    *a.norm = (float)norm;
    skip = !isfinite(*a.norm);  // (as the caller sees it)
    if (a.max_norm > 0.0) mult *= fmin(1.0, a.max_norm / (norm + 1e-6));
  }
  AdamControl c;
  c.skip = skip;
  const int64_t t = *a.step + 1;
  if (!skip) *a.step = t;
  double p1 = 1.0, p2 = 1.0, b1 = a.beta1, b2 = a.beta2;
  for (int64_t n = t; n > 0; n >>= 1) {
    if (n & 1) p1 *= b1, p2 *= b2;
    b1 *= b1, b2 *= b2;
  }
  const double lr = a.lr_ptr ? (double)*a.lr_ptr : a.lr;
  c.grad_mult = (float)mult;
  c.step_size = (float)(lr / (1.0 - p1));
  c.inv_root_c2 = (float)(1.0 / sqrt(1.0 - p2));
  c.decay = (float)(1.0 - lr * a.decay);
  *a.ctl = c;
}

// ---------------------------------------------------------------- host

static size_t adamw_workspace(int64_t tensors) {
  const int64_t launches = (tensors + kAdamPerLaunch - 1) / kAdamPerLaunch;
  return 256 + round256((size_t)launches * kNormBlocks * 8);
}

static int check_adamw(const kt_adamw* h) {
  if (!h) return set_error(KT_RAWINT4_EINVAL, "hyper is NULL");
  if (!isfinite(h->lr) || !isfinite(h->weight_decay) || !isfinite(h->grad_scale))
    return set_error(KT_RAWINT4_EINVAL, "lr, weight_decay and grad_scale must be finite");
  if (!(h->beta1 >= 0.0 && h->beta1 < 1.0) || !(h->beta2 >= 0.0 && h->beta2 < 1.0))
    return set_error(KT_RAWINT4_EINVAL, "beta1 and beta2 must be in [0, 1)");
  if (!(h->eps >= 0.0) || !isfinite(h->eps)) return set_error(KT_RAWINT4_EINVAL, "eps must be finite and non-negative");
  if (!(h->max_norm >= 0.0) || !isfinite(h->max_norm))
    return set_error(KT_RAWINT4_EINVAL, "max_norm must be finite and non-negative");
  if (h->state_format != KT_ADAMW_STATES_F32 && h->state_format != KT_ADAMW_STATES_E4M3)
    return set_error(KT_RAWINT4_EINVAL, "state_format must be KT_ADAMW_STATES_F32 or KT_ADAMW_STATES_E4M3");
  return KT_RAWINT4_OK;
}

static int check_adamw_tensor(const kt_adamw_tensor& t, int format) {
  // (a list's chunks are then at most 2^40)
  if (t.count < 0 || t.count > ((int64_t)1 << 36)) return set_error(KT_RAWINT4_EINVAL, "a tensor's count must be in [0, 2^36]");
  if ((t.param_type != KT_TYPE_BF16 && t.param_type != KT_TYPE_F32) ||
      (t.grad_type != KT_TYPE_BF16 && t.grad_type != KT_TYPE_F32))
    return set_error(KT_RAWINT4_EINVAL, "param_type and grad_type must be KT_TYPE_BF16 or KT_TYPE_F32");
  if (t.decay != 0 && t.decay != 1) return set_error(KT_RAWINT4_EINVAL, "decay must be 0 or 1");
  if (t.master && t.param_type != KT_TYPE_BF16) return set_error(KT_RAWINT4_EINVAL, "a master needs a bf16 param");
  const bool e8 = format == KT_ADAMW_STATES_E4M3;
  if (!e8 && (t.m_scale || t.v_scale)) return set_error(KT_RAWINT4_EINVAL, "m_scale and v_scale must be NULL with fp32 states");
  if (t.count == 0) return KT_RAWINT4_OK;
  if (!t.param || !t.grad || !t.m || !t.v) return set_error(KT_RAWINT4_EINVAL, "param, grad, m and v must be non-NULL");
  if (e8 && (!t.m_scale || !t.v_scale)) return set_error(KT_RAWINT4_EINVAL, "8-bit states need m_scale and v_scale");
  const void* ptrs[] = {t.param, t.master, t.grad, t.m, t.v, t.m_scale, t.v_scale};
  for (const void* p : ptrs)
    if (!is_aligned(p, 16)) return set_error(KT_RAWINT4_EINVAL, "tensors must be 16-byte aligned");
  return KT_RAWINT4_OK;
}

}  // namespace kt

using namespace kt;

extern "C" {

size_t kt_adamw_workspace_bytes(int32_t num_tensors) {
  if (num_tensors < 0 || num_tensors > KT_ADAMW_MAX_TENSORS) {
    set_error(KT_RAWINT4_EINVAL, "num_tensors must be in [0, 65536]");
    return 0;
  }
  set_error(KT_RAWINT4_OK, "");
  return adamw_workspace(num_tensors);
}

int kt_adamw_step(const kt_adamw* hyper, const kt_adamw_tensor* tensors, int32_t num_tensors, int64_t* step,
                  float* grad_norm, const float* lr, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_adamw(hyper);
  if (rc) return rc;
  if (num_tensors < 0 || num_tensors > KT_ADAMW_MAX_TENSORS)
    return set_error(KT_RAWINT4_EINVAL, "num_tensors must be in [0, 65536]");
  if (!tensors && num_tensors) return set_error(KT_RAWINT4_EINVAL, "tensors must be non-NULL");
  if (!step) return set_error(KT_RAWINT4_EINVAL, "step must be non-NULL");
  if (!is_aligned(step, 8) || !is_aligned(grad_norm, 4) || !is_aligned(lr, 4))
    return set_error(KT_RAWINT4_EINVAL, "step must be 8-byte aligned, grad_norm and lr 4-byte aligned");
  if (hyper->max_norm > 0.0 && !grad_norm) return set_error(KT_RAWINT4_EINVAL, "max_norm needs grad_norm");
  for (int i = 0; i < num_tensors; ++i)
    if ((rc = check_adamw_tensor(tensors[i], hyper->state_format))) return rc;
  rc = check_caller_workspace(workspace, workspace_bytes, adamw_workspace(num_tensors));
  if (rc) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  AdamArgs a{};
  a.ctl = static_cast<const AdamControl*>(workspace);
  a.b1 = (float)hyper->beta1;
  a.b1c = (float)(1.0 - hyper->beta1);
  a.b2 = (float)hyper->beta2;
  a.b2c = (float)(1.0 - hyper->beta2);
  a.eps = (float)hyper->eps;
  double* part = ws_ptr<double>(workspace, 256);
  int parts = 0;
  begin_launches();
  // pass 0: the norm's partial sums; 1: the updates
  for (int pass = grad_norm ? 0 : 1; pass < 2; ++pass) {
    if (pass == 1) {
      const AdamBegin b{static_cast<AdamControl*>(workspace), part, parts, step, grad_norm, lr, hyper->lr, hyper->beta1,
                        hyper->beta2, hyper->weight_decay, hyper->max_norm, hyper->grad_scale};
      k_adamw_begin<<<1, 256, 0, st>>>(b);
      note_launch();
    }
    for (int i = 0; i < num_tensors;) {
      a.count = 0;
      a.chunks = 0;
      for (; i < num_tensors && a.count < kAdamPerLaunch; ++i) {
        const kt_adamw_tensor& t = tensors[i];
        if (t.count == 0) continue;
        const int64_t chunks = (t.count + kAdamChunk - 1) / kAdamChunk;
        a.t[a.count++] = {t.param, t.master, t.grad, t.m, t.v, t.m_scale, t.v_scale, t.count, a.chunks,
                          t.param_type == KT_TYPE_F32, t.grad_type == KT_TYPE_F32, (uint8_t)t.decay};
        a.chunks += chunks;
      }
      if (!a.count) break;
      if (pass == 0) {
        const int blocks = (int)(a.chunks < kNormBlocks ? a.chunks : kNormBlocks);
        a.part = part + parts;
        parts += blocks;
        k_grad_squares<<<blocks, 256, 0, st>>>(a);
        note_launch();
        continue;
      }
      for (a.from = 0; a.from < a.chunks; a.from += kAdamLaunch) {
        const unsigned blocks = (unsigned)(a.chunks - a.from < kAdamLaunch ? a.chunks - a.from : kAdamLaunch);
        if (hyper->state_format == KT_ADAMW_STATES_E4M3)
          k_adamw<true><<<blocks, 256, 0, st>>>(a);
        else
          k_adamw<false><<<blocks, 256, 0, st>>>(a);
        note_launch();
      }
    }
  }
  return finish_launches();
}

}  // extern "C"
