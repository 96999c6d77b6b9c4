// Norms before and after a block, fused with its gate, scale and the residual
// stream, and their gradients.
#include "kt_step_common.hpp"

#include <math.h>

namespace kt {

constexpr int kNormMaxWaves = 16;

struct NormArgs {
  int64_t T;
  int H, kind;
  float eps, scale, inv_h;
  const void* x;  // backward: h
  const uint16_t* b;
  const float* tg;
  const float *w, *c, *bw, *bc, *gate;
  void* h;  // backward: grad_x
  uint16_t* y;
  // backward
  const void* gh;
  const uint16_t* gy;
  uint16_t* gb;
  float* gtg;
  float* part;  // [groups][5][H]: d_weight, d_bias, d_branch_weight, d_branch_bias, d_gate
  int nvec;     // backward: bit i, vector i is wanted; forward: whether the branch is normalised
};

// A thread's columns: chunks of 8 neighbours (VEC: rows of whole 16 bytes), or
// single ones a row's threads apart.
template <bool VEC>
struct Cols {
  int tid, nt, H;
  __device__ __forceinline__ int at(int j) const { return VEC ? 8 * (tid + (j >> 3) * nt) + (j & 7) : tid + j * nt; }
  __device__ __forceinline__ bool has(int j) const { return VEC ? 8 * (tid + (j >> 3) * nt) < H : tid + j * nt < H; }
};

template <bool VEC, int N>
__device__ __forceinline__ void load_row(const float* p, const Cols<VEC>& c, float* v) {
  if (VEC) {
#pragma unroll
    for (int j = 0; j < N; j += 8) {
      float4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
      if (c.has(j)) {
        a = *reinterpret_cast<const float4*>(p + c.at(j));
        b = *reinterpret_cast<const float4*>(p + c.at(j) + 4);
      }
      v[j] = a.x, v[j + 1] = a.y, v[j + 2] = a.z, v[j + 3] = a.w;
      v[j + 4] = b.x, v[j + 5] = b.y, v[j + 6] = b.z, v[j + 7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = c.has(j) ? p[c.at(j)] : 0.f;
  }
}

template <bool VEC, int N>
__device__ __forceinline__ void load_row(const uint16_t* p, const Cols<VEC>& c, float* v) {
  if (VEC) {
#pragma unroll
    for (int j = 0; j < N; j += 8) {
      u32x4 a = {0, 0, 0, 0};
      if (c.has(j)) a = *reinterpret_cast<const u32x4*>(p + c.at(j));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[j + 2 * i] = __uint_as_float(a[i] << 16);
        v[j + 2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = c.has(j) ? bf16_to_float(p[c.at(j)]) : 0.f;
  }
}

template <bool VEC, int N>
__device__ __forceinline__ void store_row(float* p, const Cols<VEC>& c, const float* v) {
  if (VEC) {
#pragma unroll
    for (int j = 0; j < N; j += 8) {
      if (!c.has(j)) continue;
      *reinterpret_cast<float4*>(p + c.at(j)) = float4{v[j], v[j + 1], v[j + 2], v[j + 3]};
      *reinterpret_cast<float4*>(p + c.at(j) + 4) = float4{v[j + 4], v[j + 5], v[j + 6], v[j + 7]};
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (c.has(j)) p[c.at(j)] = v[j];
  }
}

template <bool VEC, int N>
__device__ __forceinline__ void store_row(uint16_t* p, const Cols<VEC>& c, const float* v) {
  if (VEC) {
#pragma unroll
    for (int j = 0; j < N; j += 8) {
      if (!c.has(j)) continue;
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = pack2(float_to_bf16(v[j + 2 * i]), float_to_bf16(v[j + 2 * i + 1]));
      *reinterpret_cast<u32x4*>(p + c.at(j)) = o;
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (c.has(j)) p[c.at(j)] = float_to_bf16(v[j]);
  }
}

// Sums of M values over a row's threads, the same bits in all of them: in a
// wave by lanes, between waves through LDS in the waves' order.  Two buffers in
// turn: one barrier a sum.
template <bool ONE, int M>
struct RowSums {
  float (*buf)[M][kNormMaxWaves];
  int waves, turn;
  __device__ __forceinline__ void operator()(float* s) {
#pragma unroll
    for (int i = 0; i < M; ++i) s[i] = wave_sum(s[i]);
    if (ONE) return;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < M; ++i) buf[turn][i][wave] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < M; ++i) {
      float t = buf[turn][i][0];
      for (int w = 1; w < waves; ++w) t += buf[turn][i][w];
      s[i] = t;
    }
    turn ^= 1;
  }
};

// v normalised in place
template <bool VEC, int N, typename Sums>
__device__ __forceinline__ void normalise(const NormArgs& a, const Cols<VEC>& c, Sums& sums, float* v) {
  float s = 0.f, mean = 0.f;
  if (a.kind == KT_NORM_LAYER) {
#pragma unroll
    for (int j = 0; j < N; ++j) s += v[j];
    sums(&s);
    mean = s * a.inv_h;
    s = 0.f;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    v[j] = c.has(j) ? v[j] - mean : 0.f;
    s = fmaf(v[j], v[j], s);
  }
  sums(&s);
  const float r = 1.f / sqrtf(s * a.inv_h + a.eps);
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] *= r;
}

template <bool VEC, int N>
__device__ __forceinline__ void affine(const Cols<VEC>& c, const float* w, const float* bias, float* v) {
  float t[N];
  if (w) {
    load_row<VEC, N>(w, c, t);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] *= t[j];
  }
  if (bias) {
    load_row<VEC, N>(bias, c, t);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] += t[j];
  }
}

template <typename S, bool VEC, int VPT, bool ONE>
__global__ __launch_bounds__(ONE ? 256 : 1024) void k_norm_fwd(NormArgs a) {
  constexpr int N = 8 * VPT;
  __shared__ float buf[2][1][kNormMaxWaves];
  RowSums<ONE, 1> sums{buf, (int)(blockDim.x >> 6), 0};
  const Cols<VEC> c{ONE ? (int)threadIdx.x & 63 : (int)threadIdx.x, ONE ? 64 : (int)blockDim.x, a.H};
  const int64_t first = ONE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const int64_t step = ONE ? (int64_t)gridDim.x * 4 : gridDim.x;
  for (int64_t row = first; row < a.T; row += step) {
    float v[N];
    load_row<VEC, N>(static_cast<const S*>(a.x) + row * a.H, c, v);
    if (a.b) {
      float b[N];
      load_row<VEC, N>(a.b + row * a.H, c, b);
      if (a.nvec) normalise<VEC, N>(a, c, sums, b);
      affine<VEC, N>(c, a.bw, a.bc, b);
      const float s = a.tg ? a.scale * a.tg[row] : a.scale;
      affine<VEC, N>(c, a.gate, nullptr, b);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = fmaf(s, b[j], v[j]);
      if (a.h) store_row<VEC, N>(static_cast<S*>(a.h) + row * a.H, c, v);
    }
    if (a.y) {
      normalise<VEC, N>(a, c, sums, v);
      affine<VEC, N>(c, a.w, a.c, v);
      store_row<VEC, N>(a.y + row * a.H, c, v);
    }
  }
}

// POST: the norm behind the block; BR: a block's output; NEXT: grad_y.
template <typename S, bool VEC, int VPT, bool ONE, bool BR, bool POST, bool NEXT>
__global__ __launch_bounds__(ONE ? 256 : 1024) void k_norm_bwd(NormArgs a) {
  constexpr int N = 8 * VPT;
  __shared__ float buf[2][3][kNormMaxWaves];
  RowSums<ONE, 3> sums{buf, (int)(blockDim.x >> 6), 0};
  const Cols<VEC> c{ONE ? (int)threadIdx.x & 63 : (int)threadIdx.x, ONE ? 64 : (int)blockDim.x, a.H};
  const int64_t group = ONE ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x;
  const int64_t step = ONE ? (int64_t)gridDim.x * 4 : gridDim.x;
  const bool layer = a.kind == KT_NORM_LAYER;
  float dw[N], dc[N], dbw[N], dbc[N], dg[N];
#pragma unroll
  for (int j = 0; j < N; ++j) dw[j] = dc[j] = dbw[j] = dbc[j] = dg[j] = 0.f;
  for (int64_t row = group; row < a.T; row += step) {
    float v[N], d[N], b[N], e[N];
    float s[3] = {0.f, 0.f, 0.f};
    if (NEXT) {
      load_row<VEC, N>(static_cast<const S*>(a.x) + row * a.H, c, v);
      load_row<VEC, N>(a.gy + row * a.H, c, e);
      if (a.w) {
        load_row<VEC, N>(a.w, c, d);
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) d[j] = 1.f;
      }
    }
    if (BR) load_row<VEC, N>(a.b + row * a.H, c, b);
    // means and deviations of h and b; d = grad_y * weight
    float r1 = 0.f, r2 = 0.f, m1 = 0.f, m2 = 0.f;
    if (NEXT) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        dc[j] += e[j];
        d[j] *= e[j];
      }
    }
    if (layer && (NEXT || POST)) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (NEXT) s[0] += v[j], s[1] += d[j];
        if (POST) s[2] += b[j];
      }
      sums(s);
      m1 = s[1] * a.inv_h;
      const float mv = s[0] * a.inv_h, mb = s[2] * a.inv_h;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (NEXT) v[j] = c.has(j) ? v[j] - mv : 0.f;
        if (POST) b[j] = c.has(j) ? b[j] - mb : 0.f;
      }
      s[0] = s[1] = s[2] = 0.f;
    }
    if (NEXT || POST) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (NEXT) s[0] = fmaf(v[j], v[j], s[0]), s[1] = fmaf(d[j], v[j], s[1]);
        if (POST) s[2] = fmaf(b[j], b[j], s[2]);
      }
      sums(s);
      if (NEXT) {
        r1 = 1.f / sqrtf(s[0] * a.inv_h + a.eps);
        m2 = s[1] * a.inv_h * r1;
      }
      if (POST) r2 = 1.f / sqrtf(s[2] * a.inv_h + a.eps);
    }
    // d = grad of h
    if (NEXT) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        v[j] *= r1;
        dw[j] = fmaf(e[j], v[j], dw[j]);
        d[j] = r1 * (d[j] - m1 - v[j] * m2);
      }
    }
    if (a.gh) {
      if (NEXT) {
        load_row<VEC, N>(static_cast<const S*>(a.gh) + row * a.H, c, e);
#pragma unroll
        for (int j = 0; j < N; ++j) d[j] += e[j];
      } else {
        load_row<VEC, N>(static_cast<const S*>(a.gh) + row * a.H, c, d);
      }
    }
    if (a.h) store_row<VEC, N>(static_cast<S*>(a.h) + row * a.H, c, d);
    if (!BR) continue;
    // e = n, the block's output behind its norm
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (POST) b[j] *= r2;
      e[j] = b[j];
    }
    if (POST) affine<VEC, N>(c, a.bw, a.bc, e);
    s[0] = s[1] = s[2] = 0.f;
    const float sc = a.tg ? a.scale * a.tg[row] : a.scale;
    // the token gate's gradient is without it, the channel gate's with it
#pragma unroll
    for (int j = 0; j < N; ++j) {
      e[j] = c.has(j) ? e[j] * d[j] : 0.f;
      dg[j] = fmaf(sc, e[j], dg[j]);
    }
    affine<VEC, N>(c, a.gate, nullptr, d);
    if (a.gtg) {
      affine<VEC, N>(c, a.gate, nullptr, e);
#pragma unroll
      for (int j = 0; j < N; ++j) s[2] += e[j];
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      d[j] *= sc;
      if (POST) {
        dbw[j] = fmaf(d[j], b[j], dbw[j]);
        dbc[j] += d[j];
      }
    }
    if (POST) {
      affine<VEC, N>(c, a.bw, nullptr, d);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        d[j] = c.has(j) ? d[j] : 0.f;
        s[0] += d[j];
        s[1] = fmaf(d[j], b[j], s[1]);
      }
    }
    if (POST || a.gtg) sums(s);
    if (a.gtg && (ONE ? (threadIdx.x & 63) == 0 : threadIdx.x == 0)) a.gtg[row] = a.scale * s[2];
    if (!a.gb) continue;
    if (POST) {
      const float k1 = layer ? s[0] * a.inv_h : 0.f, k2 = s[1] * a.inv_h;
#pragma unroll
      for (int j = 0; j < N; ++j) d[j] = r2 * (d[j] - k1 - b[j] * k2);
    }
    store_row<VEC, N>(a.gb + row * a.H, c, d);
  }
  float* part = a.part + group * 5 * a.H;
  if (a.nvec & 1) store_row<VEC, N>(part, c, dw);
  if (a.nvec & 2) store_row<VEC, N>(part + a.H, c, dc);
  if (a.nvec & 4) store_row<VEC, N>(part + 2 * (int64_t)a.H, c, dbw);
  if (a.nvec & 8) store_row<VEC, N>(part + 3 * (int64_t)a.H, c, dbc);
  if (a.nvec & 16) store_row<VEC, N>(part + 4 * (int64_t)a.H, c, dg);
}

// The parameters' gradients from the groups' partial sums: 64 columns by 16
// runs of groups a block, joined in the runs' order.
struct NormJoin {
  const float* part;
  int64_t groups;
  int H, accumulate;
  float scale;
  float* out[5];
};
__global__ __launch_bounds__(1024) void k_norm_join(NormJoin a) {
  __shared__ float red[16][64];
  const int lane = threadIdx.x & 63, run = threadIdx.x >> 6, col = blockIdx.x * 64 + lane, vec = blockIdx.y;
  float* out = a.out[vec];
  if (!out) return;
  float s = 0.f;
  if (col < a.H) {
    const int64_t per = (a.groups + 15) / 16, end = min(a.groups, (run + 1) * per);
    for (int64_t g = run * per; g < end; ++g) s += a.part[(g * 5 + vec) * a.H + col];
  }
  red[run][lane] = s;
  __syncthreads();
  if (run || col >= a.H) return;
  for (int r = 1; r < 16; ++r) s += red[r][lane];
  out[col] = (a.accumulate ? out[col] : 0.f) + a.scale * s;
}

// ---------------------------------------------------------------- host

struct NormShape {
  bool vec, one;
  int vpt, threads;
};
static NormShape norm_shape(int H) {
  NormShape s;
  s.vec = H % 8 == 0;
  const int units = (H + 7) / 8;
  s.one = units <= 64;
  s.vpt = units <= 1024 ? 1 : 2;
  s.threads = s.one ? 256 : (units + 64 * s.vpt - 1) / (64 * s.vpt) * 64;
  return s;
}
constexpr int64_t kNormGroups = 512;  // blocks of a backward (waves where a row is one wave's)

// groups of rows that have a partial sum of their own
static int64_t norm_groups(const NormShape& s, int64_t T) {
  if (s.one) return (T < 4 * kNormGroups ? (T + 3) / 4 : kNormGroups) * 4;
  return T < kNormGroups ? T : kNormGroups;
}

static int check_norm(const kt_norm* n, int32_t tokens) {
  if (!n) return set_error(KT_RAWINT4_EINVAL, "norm is NULL");
  if (n->hidden < 1 || n->hidden > KT_NORM_MAX_HIDDEN)
    return set_error(KT_RAWINT4_EINVAL, "hidden must be in [1, 16384]");
  if (n->kind != KT_NORM_RMS && n->kind != KT_NORM_LAYER)
    return set_error(KT_RAWINT4_EINVAL, "kind must be KT_NORM_RMS or KT_NORM_LAYER");
  if (n->stream_type != KT_TYPE_BF16 && n->stream_type != KT_TYPE_F32)
    return set_error(KT_RAWINT4_EINVAL, "stream_type must be KT_TYPE_BF16 or KT_TYPE_F32");
  if (n->branch_norm != 0 && n->branch_norm != 1) return set_error(KT_RAWINT4_EINVAL, "branch_norm must be 0 or 1");
  if (!isfinite(n->eps) || n->eps < 0.f) return set_error(KT_RAWINT4_EINVAL, "eps must be finite and non-negative");
  if (!isfinite(n->scale)) return set_error(KT_RAWINT4_EINVAL, "scale must be finite");
  if (!n->branch_norm && (n->branch_weight || n->branch_bias))
    return set_error(KT_RAWINT4_EINVAL, "branch_weight and branch_bias need branch_norm");
  const float* v[] = {n->weight, n->bias, n->branch_weight, n->branch_bias, n->gate};
  for (const float* p : v)
    if (!is_aligned(p, 16)) return set_error(KT_RAWINT4_EINVAL, "vectors must be 16-byte aligned");
  if (tokens < 0 || tokens > (1 << 23)) return set_error(KT_RAWINT4_EINVAL, "tokens must be in [0, 2^23]");
  return KT_RAWINT4_OK;
}

static NormArgs norm_args(const kt_norm* n, int64_t T) {
  NormArgs a{};
  a.T = T;
  a.H = n->hidden;
  a.kind = n->kind;
  a.eps = n->eps;
  a.scale = n->scale;
  a.inv_h = 1.f / (float)n->hidden;
  a.w = n->weight;
  a.c = n->bias;
  a.bw = n->branch_weight;
  a.bc = n->branch_bias;
  a.gate = n->gate;
  return a;
}

template <typename S, bool VEC>
static void launch_norm_fwd(const NormArgs& a, const NormShape& s, hipStream_t st) {
  const int64_t rows = s.one ? (a.T + 3) / 4 : a.T;
  const unsigned grid = (unsigned)(rows < 4096 ? rows : 4096);
  if (s.one)
    k_norm_fwd<S, VEC, 1, true><<<grid, 256, 0, st>>>(a);
  else if (s.vpt == 1)
    k_norm_fwd<S, VEC, 1, false><<<grid, s.threads, 0, st>>>(a);
  else
    k_norm_fwd<S, VEC, 2, false><<<grid, s.threads, 0, st>>>(a);
  note_launch();
}

template <typename S, bool VEC, bool BR, bool POST, bool NEXT>
static void launch_norm_bwd(const NormArgs& a, const NormShape& s, hipStream_t st) {
  const int64_t groups = norm_groups(s, a.T);
  if (s.one)
    k_norm_bwd<S, VEC, 1, true, BR, POST, NEXT><<<(unsigned)(groups / 4), 256, 0, st>>>(a);
  else if (s.vpt == 1)
    k_norm_bwd<S, VEC, 1, false, BR, POST, NEXT><<<(unsigned)groups, s.threads, 0, st>>>(a);
  else
    k_norm_bwd<S, VEC, 2, false, BR, POST, NEXT><<<(unsigned)groups, s.threads, 0, st>>>(a);
  note_launch();
}

template <typename S, bool VEC>
static void launch_norm_bwd_parts(const NormArgs& a, const NormShape& s, bool post, hipStream_t st) {
  if (!a.b)
    a.gy ? launch_norm_bwd<S, VEC, false, false, true>(a, s, st) : launch_norm_bwd<S, VEC, false, false, false>(a, s, st);
  else if (post)
    a.gy ? launch_norm_bwd<S, VEC, true, true, true>(a, s, st) : launch_norm_bwd<S, VEC, true, true, false>(a, s, st);
  else
    a.gy ? launch_norm_bwd<S, VEC, true, false, true>(a, s, st) : launch_norm_bwd<S, VEC, true, false, false>(a, s, st);
}

}  // namespace kt

using namespace kt;

extern "C" {

int kt_norm_fwd(const kt_norm* norm, int32_t tokens, const void* x, const uint16_t* branch, const float* token_gate,
                void* h, uint16_t* y, void* stream) {
  const int rc = check_norm(norm, tokens);
  if (rc) return rc;
  if (tokens == 0) return set_error(KT_RAWINT4_OK, "");
  if (!x) return set_error(KT_RAWINT4_EINVAL, "x must be non-NULL");
  if (!branch && (h || token_gate))
    return set_error(KT_RAWINT4_EINVAL, "h and token_gate must be NULL without a branch (h is x)");
  if (!h && !y) return set_error(KT_RAWINT4_EINVAL, "one of h and y must be non-NULL");
  if (!is_aligned(x, 16) || !is_aligned(branch, 16) || !is_aligned(h, 16) || !is_aligned(y, 16) ||
      !is_aligned(token_gate, 4))
    return set_error(KT_RAWINT4_EINVAL, "tensors must be 16-byte aligned, token_gate 4-byte aligned");
  NormArgs a = norm_args(norm, tokens);
  a.x = x;
  a.b = branch;
  a.tg = token_gate;
  a.h = h;
  a.y = y;
  a.nvec = norm->branch_norm;
  const NormShape s = norm_shape(a.H);
  hipStream_t st = static_cast<hipStream_t>(stream);
  begin_launches();
  if (norm->stream_type == KT_TYPE_BF16)
    s.vec ? launch_norm_fwd<uint16_t, true>(a, s, st) : launch_norm_fwd<uint16_t, false>(a, s, st);
  else
    s.vec ? launch_norm_fwd<float, true>(a, s, st) : launch_norm_fwd<float, false>(a, s, st);
  return finish_launches();
}

size_t kt_norm_bwd_workspace_bytes(const kt_norm* norm, int32_t tokens) {
  if (check_norm(norm, tokens)) return 0;
  set_error(KT_RAWINT4_OK, "");
  return round256((size_t)norm_groups(norm_shape(norm->hidden), tokens) * 5 * (size_t)norm->hidden * 4);
}

int kt_norm_bwd(const kt_norm* norm, int32_t tokens, const void* h, const uint16_t* branch, const float* token_gate,
                const void* grad_h, const uint16_t* grad_y, void* grad_x, uint16_t* grad_branch,
                float* grad_token_gate, float* d_weight, float* d_bias, float* d_branch_weight, float* d_branch_bias,
                float* d_gate, int32_t accumulate, float grad_scale, void* workspace, size_t workspace_bytes,
                void* stream) {
  int rc = check_norm(norm, tokens);
  if (rc) return rc;
  if (accumulate != 0 && accumulate != 1) return set_error(KT_RAWINT4_EINVAL, "accumulate must be 0 or 1");
  if (!isfinite(grad_scale)) return set_error(KT_RAWINT4_EINVAL, "grad_scale must be finite");
  const void* params[] = {d_weight, d_bias, d_branch_weight, d_branch_bias, d_gate};
  for (const void* p : params)
    if (!is_aligned(p, 16)) return set_error(KT_RAWINT4_EINVAL, "tensors must be 16-byte aligned");
  if ((d_branch_weight || d_branch_bias) && !norm->branch_norm)
    return set_error(KT_RAWINT4_EINVAL, "d_branch_weight and d_branch_bias need branch_norm");
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int H = norm->hidden;
  if (tokens == 0) {
    begin_launches();
    if (!accumulate)
      for (void* p : {(void*)d_weight, (void*)d_bias, (void*)d_branch_weight, (void*)d_branch_bias, (void*)d_gate})
        if (p) launch_fill_zero_f32(static_cast<float*>(p), H, st);
    return finish_launches();
  }
  if (!h) return set_error(KT_RAWINT4_EINVAL, "h must be non-NULL");
  if (!grad_h && !grad_y) return set_error(KT_RAWINT4_EINVAL, "one of grad_h and grad_y must be non-NULL");
  if (!grad_y && (d_weight || d_bias)) return set_error(KT_RAWINT4_EINVAL, "d_weight and d_bias need grad_y");
  if (!branch && (token_gate || grad_branch || d_branch_weight || d_branch_bias || d_gate))
    return set_error(KT_RAWINT4_EINVAL, "token_gate, grad_branch, d_branch_weight, d_branch_bias and d_gate need a branch");
  if (!token_gate && grad_token_gate) return set_error(KT_RAWINT4_EINVAL, "grad_token_gate needs token_gate");
  for (const void* p : {h, (const void*)branch, grad_h, (const void*)grad_y, (const void*)grad_x, (const void*)grad_branch})
    if (!is_aligned(p, 16)) return set_error(KT_RAWINT4_EINVAL, "tensors must be 16-byte aligned");
  if (!is_aligned(token_gate, 4) || !is_aligned(grad_token_gate, 4))
    return set_error(KT_RAWINT4_EINVAL, "token_gate must be 4-byte aligned");
  rc = check_caller_workspace(workspace, workspace_bytes, kt_norm_bwd_workspace_bytes(norm, tokens));
  if (rc) return rc;
  NormArgs a = norm_args(norm, tokens);
  a.x = h;
  a.b = branch;
  a.tg = token_gate;
  a.h = grad_x;
  a.gh = grad_h;
  a.gy = grad_y;
  a.gb = grad_branch;
  a.gtg = grad_token_gate;
  a.part = static_cast<float*>(workspace);
  for (int i = 0; i < 5; ++i) a.nvec |= (params[i] != nullptr) << i;
  const NormShape s = norm_shape(H);
  const bool post = norm->branch_norm != 0;
  begin_launches();
  if (norm->stream_type == KT_TYPE_BF16)
    s.vec ? launch_norm_bwd_parts<uint16_t, true>(a, s, post, st) : launch_norm_bwd_parts<uint16_t, false>(a, s, post, st);
  else
    s.vec ? launch_norm_bwd_parts<float, true>(a, s, post, st) : launch_norm_bwd_parts<float, false>(a, s, post, st);
  if (a.nvec) {
    NormJoin j{a.part, norm_groups(s, tokens), H, accumulate, grad_scale, {d_weight, d_bias, d_branch_weight, d_branch_bias, d_gate}};
    k_norm_join<<<dim3((unsigned)((H + 63) / 64), 5), 1024, 0, st>>>(j);
    note_launch();
  }
  return finish_launches();
}

}  // extern "C"
