// Routing of tokens to experts: scores, the choice of top_k experts (bias for
// balance, groups), their weights, the gradient with respect to the logits, the
// load per expert and the bias's balance rule.
//
// The choice is made on c = s + b to 64 bits, ties to the lower index, so that
// it is the formula's choice and not one of fp32 roundings: with a few hundred
// experts some tokens of every long batch have two candidates whose c differ
// by less than an fp32 rounding.
#include <math.h>

#include <type_traits>

#include "kt_common.hpp"
#include "kt_internal.hpp"

namespace kt {

struct RouterArgs {
  int E, k, G, per, top_groups, group_top;  // G = 1 (per = E) where every group stays
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

// ---------------------------------------------------------------- 16 lanes a token

// Up to 512 experts and 16 choices: a block routes 16 tokens, 16 lanes each.
// A token's logits are staged in LDS.  Of G groups of `per` experts, lg = 16 / G
// (rounded down) lanes share one: lane q has group q / lg and its experts q %
// lg, q % lg + lg, ..., at most VPL of them (without groups: G = 1, lg = 16).
//
// The choice.  With fp32 keys (the logit itself without a bias, which orders as
// s does; else s + b to within tol / 2) let t be the k-th largest of the 16
// lanes' two largest keys each.  At least k keys reach t, so no expert below
// t - tol is among the k best.  The few above it (8 to 10 of 384 for k = 8) are
// listed, valued in 64 bits, one per lane, and ranked against each other; equal
// values rank by index.  Where over kList experts reach t - tol (rows of equal
// scores, say), k rounds of the 16 lanes' best 64-bit value choose instead.
//
// Groups (whole lanes each) are kept by their fp32 scores, and by scores to 64
// bits where the border between kept and dropped lies within the fp32 error.
//
// Bound by instructions (1425 vector, 360 scalar and 100 LDS ones a wave of four
// tokens), then by latency where one block a unit is all there is: 16384 tokens of 384 experts in 8 groups 18 us
// (reading the logits alone: 5), 4096 tokens 11 us, one token 8 us.  Choosing
// by k rounds of a block's best instead took 434 us.
constexpr int kLanes = 16, kTokens = 16, kList = 48, kMaxVpl = 32;

template <int CTRL>
__device__ __forceinline__ int dpp_i(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xf, 0xf, true);
}
__device__ __forceinline__ int row16_or(int v) {
  v |= dpp_i<0xB1>(v);
  v |= dpp_i<0x4E>(v);
  v |= dpp_i<0x141>(v);
  return v | dpp_i<0x140>(v);
}
__device__ __forceinline__ float row16_min(float v) { return -row16_max(-v); }

// counts the other lanes' b1 and b2 (b1 >= b2) above this lane's b1 and above its b2
__device__ __forceinline__ void row16_above(float b1, float b2, int& n1, int& n2) {
  // row_ror 1 .. 15
#define KT_ABOVE(r)                                                     \
  {                                                                     \
    const float o1 = dpp_f<0x120 + r>(b1), o2 = dpp_f<0x120 + r>(b2);   \
    n1 += (o1 > b1) + (o2 > b1);                                        \
    n2 += (o1 > b2) + (o2 > b2);                                        \
  }
  KT_ABOVE(1) KT_ABOVE(2) KT_ABOVE(3) KT_ABOVE(4) KT_ABOVE(5) KT_ABOVE(6) KT_ABOVE(7) KT_ABOVE(8)
  KT_ABOVE(9) KT_ABOVE(10) KT_ABOVE(11) KT_ABOVE(12) KT_ABOVE(13) KT_ABOVE(14) KT_ABOVE(15)
#undef KT_ABOVE
}

// sum of the lower lanes' v (whole numbers)
__device__ __forceinline__ int row16_before(int v) {
  int s = v;
  s += dpp_i<0x111>(s);  // row_shr 1, 2, 4, 8 (zeros shift in)
  s += dpp_i<0x112>(s);
  s += dpp_i<0x114>(s);
  s += dpp_i<0x118>(s);
  return s - v;
}

// The sigmoid in fp32 with the library's exponential (about one rounding), from
// the exponential of -|l|: it keeps a small score's digits down to fp32's
// lowest numbers, and 1 - s is sigmoid32(-l).
__device__ __forceinline__ float sigmoid32(float l) {
  const float e = expf(-fabsf(l));
  return (l < 0.f ? e : 1.f) / (1.f + e);
}

// exp for arguments up to 0 from the hardware's exp2 (relative error below 2^-23 (2 + 1.5 |x|))
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.4426950408889634f); }

// (value, index) pairs in the order of choice: larger value, then lower index.
__device__ __forceinline__ bool better(double a, int ia, double b, int ib) { return a > b || (a == b && ia < ib); }

// A token's logits to LDS, widened to fp32, by its 16 lanes: 16-byte pieces
// where rows start at 16 bytes.
template <bool BF16>
__device__ __forceinline__ void stage_row(const void* src, int64_t first, int E, int q, float* dst) {
  constexpr int kPiece = BF16 ? 8 : 4;
  if (E % kPiece == 0) {
    for (int i = q * kPiece; i < E; i += kLanes * kPiece) {
      const u32x4 p = *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(src) + (first + i) * (16 / kPiece));
      if (BF16) {
        floatx4* d = reinterpret_cast<floatx4*>(dst + i);
        d[0] = floatx4{__uint_as_float(p.x << 16), __uint_as_float(p.x & 0xffff0000u), __uint_as_float(p.y << 16),
                       __uint_as_float(p.y & 0xffff0000u)};
        d[1] = floatx4{__uint_as_float(p.z << 16), __uint_as_float(p.z & 0xffff0000u), __uint_as_float(p.w << 16),
                       __uint_as_float(p.w & 0xffff0000u)};
      } else {
        *reinterpret_cast<u32x4*>(dst + i) = p;
      }
    }
  } else {
    for (int i = q; i < E; i += kLanes) dst[i] = load_logit<BF16>(src, first + i);
  }
}

// Rows in LDS lie kRowPad values more than the largest row apart: the four
// tokens of a wave start at different banks.
constexpr int kRowPad = 16;

template <int SCORE, bool BF16, int VPL>
__global__ __launch_bounds__(256) void k_route(RouterArgs a, int64_t tokens, int32_t* __restrict__ load) {
  __shared__ __align__(16) float rows[kTokens][kLanes * VPL + kRowPad];
  __shared__ float bias[kLanes * VPL];
  __shared__ double val[kTokens][kList];  // before that, the groups' two best of each lane
  __shared__ uint16_t list[kTokens][kList];
  __shared__ int sel[kTokens][kLanes];
  __shared__ int hist[kLanes * VPL];
  const int64_t t0 = (int64_t)blockIdx.x * kTokens;
  const int E = a.E, k = a.k;
  const int q = threadIdx.x & 15, tok = threadIdx.x >> 4;
  const int64_t t = t0 + tok;
  float* row = rows[tok];
  stage_row<BF16>(a.logits, min(t, tokens - 1) * E, E, q, row);  // (past the end: the last token again)
  int bad_bias = 0;
  for (int e = threadIdx.x; e < E; e += 256) {
    const float b = a.bias ? a.bias[e] : 0.f;
    bad_bias |= is_nan(b) || b == INFINITY;
    bias[e] = b;
    hist[e] = 0;
  }
  bad_bias = __syncthreads_or(bad_bias);
  const int lg = kLanes / a.G, g = q / lg;  // lanes per group, this lane's group (from G on: none)
  // this lane's experts are e0 + lg i, i < own.  With per <= lg VPL, e0 + lg i stays below 16 VPL for every i < VPL.
  const int e0 = g < a.G ? g * a.per + q % lg : 0, own = g < a.G ? max(0, (a.per - q % lg + lg - 1) / lg) : 0;
  const bool exact = a.bias == nullptr;

  // (reads past a token's logits stay inside the array; the fp32 keys use the hardware's exponential and
  // reciprocal, whose error tol covers; a few loops stay rolled to keep the code short: a single token's time
  // is mostly that of fetching it)
  float l[VPL];
  float mx = -INFINITY;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float x = row[e0 + lg * i];
    l[i] = i < own ? x : -INFINITY;
    odd |= bad_logit<SCORE>(l[i]);
    mx = fmaxf(mx, l[i]);
  }
  const int bad = row16_or(odd) | bad_bias;
  float m = 0.f, zinv = 1.f;
  double m64 = 0.0, zinv64 = 1.0;
  if (SCORE == KT_SCORE_SOFTMAX) {
    m = row16_max(mx);
    if (!(fabsf(m) < INFINITY)) m = 0.f;  // nobody left (s is 0), or an undefined row
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) z += fast_exp(l[i] - m);
    z = row16_sum(z);
    zinv = z > 0.f ? 1.f / z : 0.f;
    if (!exact) {  // s + b to 64 bits needs the sum to 64 bits
      m64 = (double)m;
      double z64 = 0.0;
#pragma unroll 1
      for (int i = 0; i < own; ++i) z64 += exp((double)row[e0 + lg * i] - m64);
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) z64 += __shfl_xor(z64, off);
      zinv64 = z64 > 0.0 ? z64 : 1.0;
    }
  }
  auto score32 = [&](float x) { return SCORE == KT_SCORE_SOFTMAX ? expf(x - m) * zinv : sigmoid32(x); };
  auto score_key = [&](float x) { return SCORE == KT_SCORE_SOFTMAX ? fast_exp(x - m) * zinv : sigmoid_f(x); };
  // c to 64 bits (without a bias: of what orders alike)
  auto value64 = [&](int e) {
    if (exact) return (double)row[e];
    const double s = SCORE == KT_SCORE_SOFTMAX ? exp((double)row[e] - m64) / zinv64 : sigmoid64((double)row[e]);
    return s + (double)bias[e];
  };

  float key[VPL];
  float big = 0.f;  // largest |key|
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    key[i] = l[i];
    if (!exact) {
      const float c = score_key(l[i]) + bias[e0 + lg * i];
      key[i] = l[i] == -INFINITY ? -INFINITY : c;
      big = fmaxf(big, key[i] > -INFINITY ? fabsf(c) : 0.f);
    }
  }
  // twice the error of a key: s within 2^-18 (softmax: some forty roundings of s and of s |l - m| <= 0.37;
  // sigmoid: far less), and the rounding of the sum with b
  const float tol = exact ? 0.f : 0x1p-17f + 0x1p-22f * row16_max(big);

  float best = -INFINITY, second = -INFINITY;  // of this lane
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    second = fmaxf(second, fminf(best, key[i]));
    best = fmaxf(best, key[i]);
  }
  if (a.G > 1) {
    const bool used = g < a.G;
    // keys whose sums the groups compare: c, or s where there is no bias
    float b1 = best, b2 = second;
    const bool sums = a.group_top == 2;
    const float reach2 = b2 - tol;  // a lane's two best to 64 bits are among its experts with such a key
    if (exact && sums) {
      b1 = b1 == -INFINITY ? b1 : score_key(b1);
      b2 = b2 == -INFINITY ? b2 : score_key(b2);
    }
    // one group's two best over its lanes, then the group's rank
    auto group_rank = [&](double x1, double x2, double& mine) {
      val[tok][2 * q] = x1;
      val[tok][2 * q + 1] = x2;
      wave_fence();
      double y1 = -INFINITY, y2 = -INFINITY;
      if (used)
        for (int j = 0; j < lg; ++j) {
          const double o1 = val[tok][2 * (g * lg + j)], o2 = val[tok][2 * (g * lg + j) + 1];
          y2 = fmax(fmin(y1, o1), fmax(y2, o2));
          y1 = fmax(y1, o1);
        }
      mine = sums ? y1 + y2 : y1;
      wave_fence();
      val[tok][2 * q] = mine;
      wave_fence();
      int rank = 0;
      for (int j = 0; j < a.G; ++j) rank += better(val[tok][2 * j * lg], j, mine, g);
      wave_fence();
      return rank;
    };
    double mine;
    bool keep = group_rank((double)b1, (double)b2, mine) < a.top_groups && used;
    if (!exact || sums) {
      const float lo = row16_min(keep ? (float)mine : INFINITY), hi = row16_max(keep || !used ? -INFINITY : (float)mine);
      const float err = exact ? 0x1p-16f : 2.f * tol;  // twice the error of a sum of two
      // (rows of the same wave may differ; all of them run the exact form where one needs it)
      if (__any(hi > -INFINITY && !(lo - hi > err))) {
        uint32_t left = 0;
#pragma unroll
        for (int i = 0; i < VPL; ++i) left |= key[i] >= reach2 && key[i] > -INFINITY ? 1u << i : 0u;
        double c1 = -INFINITY, c2 = -INFINITY;
        for (; left; left &= left - 1) {
          const int e = e0 + lg * (__ffs(left) - 1);
          double c;
          if (SCORE == KT_SCORE_SOFTMAX)  // without a bias the common divisor changes no order
            c = exp((double)row[e] - (double)m) / zinv64 + (double)bias[e];
          else
            c = sigmoid64((double)row[e]) + (double)bias[e];
          c2 = fmax(c2, fmin(c1, c));
          c1 = fmax(c1, c);
        }
        keep = group_rank(c1, c2, mine) < a.top_groups && used;
      }
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) key[i] = keep ? key[i] : -INFINITY;
    best = keep ? best : -INFINITY;
    second = keep ? second : -INFINITY;
  }

  int above1 = 0, above2 = second < best;
  row16_above(best, second, above1, above2);
  const float t_k = row16_min(above2 < k ? second : above1 < k ? best : INFINITY);
  const float floor_key = t_k - tol;
  uint32_t reach = 0;  // this lane's experts that reach it
#pragma unroll
  for (int i = 0; i < VPL; ++i) reach |= key[i] >= floor_key && key[i] > -INFINITY ? 1u << i : 0u;
  const int count = __popc(reach), at = row16_before(count);
  const int n = (int)row16_max((float)(at + count));  // of the token: the last lane's end
  const bool few = n <= kList;
  if (few) {
    int w = at;
    for (uint32_t left = reach; left; left &= left - 1) list[tok][w++] = (uint16_t)(e0 + lg * (__ffs(left) - 1));
  }
  if (q < k) sel[tok][q] = -1;
  wave_fence();
  if (few) {
    for (int c = q; c < n; c += kLanes) val[tok][c] = value64(list[tok][c]);
    wave_fence();
    for (int c = q; c < n; c += kLanes) {
      const double x = val[tok][c];
      const int e = list[tok][c];
      int rank = 0;
#pragma unroll 4
      for (int o = 0; o < n; ++o) rank += better(val[tok][o], list[tok][o], x, e);
      if (rank < k) sel[tok][rank] = e;
    }
  }
  if (__any(!few)) {
    // k rounds; a lane's experts are taken in descending order, so it keeps the last one taken
    double last = INFINITY;
    int last_e = -1;
    for (int j = 0; j < k; ++j) {
      double x = -INFINITY;
      int e = E;
      for (uint32_t left = few ? 0u : reach; left; left &= left - 1) {
        const int f = e0 + lg * (__ffs(left) - 1);
        const double c = value64(f);
        if (better(last, last_e, c, f) && better(c, f, x, e)) {
          x = c;
          e = f;
        }
      }
      double y = x;
      int f = e;
#pragma unroll
      for (int off = 1; off < 16; off <<= 1) {
        const double oy = __shfl_xor(y, off);
        const int of = __shfl_xor(f, off);
        if (better(oy, of, y, f)) {
          y = oy;
          f = of;
        }
      }
      if (f == e && e < E) {
        last = x;
        last_e = e;
      }
      if (!few && q == j && f < E) sel[tok][j] = f;
    }
  }
  wave_fence();
  int id = q < k ? sel[tok][q] : -1;
  float s = id >= 0 ? score32(row[id]) : 0.f;
  const float total = row16_sum(s);
  float w = id >= 0 ? (a.renorm ? s / (total + 1e-20f) : s) * a.scale : 0.f;
  if (bad) {
    id = q;
    w = __uint_as_float(0x7fc00000u);
  }
  if (t < tokens && q < k) {
    if (a.mask && !a.mask[t]) {
      id = -1;
      w = 0.f;
    }
    a.ids[t * k + q] = id;
    a.w[t * k + q] = w;
    if (load && id >= 0) atomicAdd(&hist[id], 1);
  }
  if (load) {  // whole numbers: the order of the sums does not matter
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 256)
      if (hist[e]) atomicAdd(&load[e], hist[e]);
  }
}

// ---------------------------------------------------------------- any size

constexpr int kAnyThreads = 256;

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

// One block per token, c of every expert in LDS to 64 bits, top_k rounds of the
// block's best.  Takes any E, k and group shape; 384 experts by top 8: 26 ns a token.
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
    // without a bias the logit itself, which orders as s does
    c[e] = l == -INFINITY || b == -INFINITY ? -INFINITY : a.bias ? score(l) + (double)b : (double)l;
  }
  if (tid == 0) sum_s = 0.0;
  __syncthreads();
  if (a.G > 1) {
    for (int g = wave; g < a.G; g += 4) {
      double v1 = -INFINITY, v2 = -INFINITY;
      for (int e = g * a.per + lane; e < (g + 1) * a.per; e += 64) {
        const double v = a.bias || a.group_top == 1 || c[e] == -INFINITY ? c[e] : score((float)c[e]);
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
  const double mul = a.renorm ? (double)a.scale / (sum_s + 1e-20) : (double)a.scale;
  for (int q = tid; q < a.k; q += kAnyThreads) {
    if (q < j) {
      w[q] = (float)(w[q] * mul);
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

// Of the chosen scores the gradient is scale (g - d) / S (scale g without
// renormalisation), and the softmax's sum ds s is scale d (1 - sum s / S) / S =
// scale d 1e-20 / S^2: written so, the tiny term keeps its value instead of a
// difference of roundings.  Scores are multiplied with 1 / S (up to 1e20) first
// and with the scale last, so that nothing overflows on the way to a result that does not.
struct RowGrad {
  float m, zinv;     // softmax: maximum and 1 / sum of exponentials
  float inv, d;      // 1 / S (1 without renormalisation), d (0 without)
  float c;           // sum ds s / scale: 1e-20 / S d (renormalised), sum g s
};

// d, c and 1 / S from the sums of the chosen s and of their g s
__device__ __forceinline__ void finish_row(const RouterBwdArgs& a, RowGrad& r, float ssum, float gsum) {
  r.c = gsum;
  if (a.renorm) {
    r.inv = 1.f / (ssum + 1e-20f);
    r.d = gsum * r.inv;
    r.c = 1e-20f * r.inv * r.d;
  }
}

// dl of an expert with logit l and score s whose slots' g - d add up to gd
// (1 - s from the logit: the difference would lose its digits where s is close to 1)
template <int SCORE>
__device__ __forceinline__ float chosen_grad(const RouterBwdArgs& a, const RowGrad& r, float l, float s, float gd) {
  if (SCORE == KT_SCORE_SIGMOID) return s * r.inv * sigmoid32(-l) * gd * a.scale;
  return (a.renorm ? s * r.inv * gd - s * r.c : s * (gd - r.c)) * a.scale;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off);
  return v;
}

// Up to 512 experts and 16 slots: 16 tokens a block, 16 lanes each.  A token's
// logits are staged in LDS and turned into -s sum ds s in place, the chosen
// experts' values are put over those, and the row is written back whole.  16384
// tokens of 384 experts in bf16 by softmax take 11 us (25 MB; a plain copy of them:
// 5), 4096 in fp32 6.6 us, of which launch and latency are most.
template <int SCORE, bool BF16, int VPL>
__global__ __launch_bounds__(256) void k_route_bwd(RouterBwdArgs a, int64_t tokens) {
  __shared__ __align__(16) float rows[kTokens][kLanes * VPL + kRowPad];
  const int E = a.E, k = a.k, v = (E + kLanes - 1) / kLanes;
  const int q = threadIdx.x & 15, tok = threadIdx.x >> 4;
  const int64_t t = (int64_t)blockIdx.x * kTokens + tok, tc = min(t, tokens - 1);
  float* row = rows[tok];
  stage_row<BF16>(a.logits, tc * E, E, q, row);
  wave_fence();
  const int64_t slot = tc * k + q;
  int id = -1;
  float g = 0.f;
  if (q < k) {
    const int64_t given = a.ids[slot];
    if (given >= 0 && given < E) {
      id = (int)given;
      g = a.g[slot];
    }
  }
  // lane q: experts q, q + 16, ... (neighbouring lanes, neighbouring banks)
  float s[VPL], mx = -INFINITY;
  int bad = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = q + kLanes * i;
    s[i] = i < v && e < E ? row[e] : -INFINITY;
    bad |= bad_logit<SCORE>(s[i]);
    mx = fmaxf(mx, s[i]);
  }
  bad = row16_or(bad);
  const int used = row16_or(id >= 0);
  RowGrad r{0.f, 1.f, 1.f, 0.f, 0.f};
  if (SCORE == KT_SCORE_SOFTMAX) {
    r.m = row16_max(mx);
    if (!(fabsf(r.m) < INFINITY)) r.m = 0.f;
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i < v) {
        s[i] = fast_exp(s[i] - r.m);
        z += s[i];
      }
    z = row16_sum(z);
    r.zinv = z > 0.f ? 1.f / z : 0.f;
  }
  const float lc = id >= 0 ? row[id] : -INFINITY;
  const float sc = id < 0 ? 0.f : SCORE == KT_SCORE_SOFTMAX ? expf(lc - r.m) * r.zinv : sigmoid32(lc);
  const float ssum = row16_sum(sc), gsum = row16_sum(g * sc);
  finish_row(a, r, ssum, gsum);
  // an expert in several slots: every one of its lanes has the sum, in slot order
  float gd = 0.f;
  const float own = id >= 0 ? g - r.d : 0.f;
  for (int j = 0; j < k; ++j) {
    const int oi = __shfl(id, j, kLanes);
    const float od = __shfl(own, j, kLanes);
    if (oi == id) gd += od;
  }
  const float rest = bad && used ? __uint_as_float(0x7fc00000u) : SCORE == KT_SCORE_SOFTMAX && used ? -r.c * r.zinv : 0.f;
  wave_fence();
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = q + kLanes * i;
    if (i < v && e < E) row[e] = bad || !used || SCORE == KT_SCORE_SIGMOID ? rest : s[i] * rest * a.scale;
  }
  wave_fence();
  if (id >= 0 && !bad) row[id] = chosen_grad<SCORE>(a, r, lc, sc, gd);
  wave_fence();
  if (t >= tokens) return;
  if (BF16) {
    uint16_t* p = static_cast<uint16_t*>(a.out) + t * E;
    if (E % 8 == 0) {
      for (int i = q * 8; i < E; i += kLanes * 8) {
        u32x4 o;
#pragma unroll
        for (int h = 0; h < 4; ++h) o[h] = pack2(float_to_bf16(row[i + 2 * h]), float_to_bf16(row[i + 2 * h + 1]));
        *reinterpret_cast<u32x4*>(p + i) = o;
      }
    } else {
      for (int i = q; i < E; i += kLanes) p[i] = float_to_bf16(row[i]);
    }
  } else {
    float* p = static_cast<float*>(a.out) + t * E;
    if (E % 4 == 0) {
      for (int i = q * 4; i < E; i += kLanes * 4)
        *reinterpret_cast<floatx4*>(p + i) = *reinterpret_cast<const floatx4*>(row + i);
    } else {
      for (int i = q; i < E; i += kLanes) p[i] = row[i];
    }
  }
}

// One block per token; the slots' g - d by expert in LDS.  Each thread owns the
// experts tid, tid + 256, ... and adds their slots in slot order.
template <int SCORE, bool BF16>
__global__ __launch_bounds__(kAnyThreads) void k_route_bwd_any(RouterBwdArgs a) {
  __shared__ float gd[KT_RAWINT4_MAX_EXPERTS];
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
    gd[e] = 0.f;
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
  finish_row(a, r, ssum, gsum);
  for (int j0 = 0; j0 < a.k; j0 += kAnyThreads) {
    __syncthreads();
    const int64_t id = j0 + tid < a.k ? ids[j0 + tid] : -1;
    sid[tid] = id >= 0 && id < a.E ? (int)id : -1;
    sg[tid] = j0 + tid < a.k ? g[j0 + tid] : 0.f;
    __syncthreads();
    const int n = min(kAnyThreads, a.k - j0);
    for (int j = 0; j < n; ++j)
      if (sid[j] >= 0 && (sid[j] & (kAnyThreads - 1)) == tid) gd[sid[j]] += sg[j] - r.d;
  }
  for (int e = tid; e < a.E; e += kAnyThreads) {
    const float l = load_logit<BF16>(a.logits, base + e);
    float v = used == 0.f ? 0.f : chosen_grad<SCORE>(a, r, l, score(l), gd[e]);
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

static void launch_zero_i32(int32_t* p, int n, hipStream_t st) {
  k_zero_i32<<<(unsigned)((n + 255) / 256), 256, 0, st>>>(p, n);
  note_launch();
}

static void launch_load(const int64_t* ids, int64_t n, int E, int accumulate, int32_t* load, hipStream_t st) {
  if (n <= 16384) {
    k_route_load_one<<<1, 1024, 0, st>>>(ids, n, E, accumulate, load);
    note_launch();
    return;
  }
  if (!accumulate) launch_zero_i32(load, E, st);
  const int64_t blocks = (n + 4095) / 4096;
  k_route_load<<<(unsigned)(blocks < 256 ? blocks : 256), 256, 0, st>>>(ids, n, E, load);
  note_launch();
}

// body(VPL as a constant) for the experts of a lane
template <typename F>
static void with_vpl(int v, F body) {
  if (v <= 4)
    body(std::integral_constant<int, 4>());
  else if (v <= 8)
    body(std::integral_constant<int, 8>());
  else if (v <= 16)
    body(std::integral_constant<int, 16>());
  else if (v <= 24)
    body(std::integral_constant<int, 24>());
  else
    body(std::integral_constant<int, kMaxVpl>());
}

// 16 lanes a token where they serve, else a block a token.
template <int SCORE, bool BF16>
static void launch_route(const RouterArgs& a, int64_t tokens, int32_t* load, int accumulate, hipStream_t st) {
  const int lg = a.G <= kLanes ? kLanes / a.G : 0, v = lg ? (a.per + lg - 1) / lg : kMaxVpl + 1;
  if (v <= kMaxVpl && a.k <= kLanes) {
    if (load && !accumulate) launch_zero_i32(load, a.E, st);
    with_vpl(v, [&](auto vpl) {
      k_route<SCORE, BF16, decltype(vpl)::value>
          <<<(unsigned)((tokens + kTokens - 1) / kTokens), 256, 0, st>>>(a, tokens, load);
    });
    note_launch();
    return;
  }
  k_route_any<SCORE, BF16><<<(unsigned)tokens, kAnyThreads, 0, st>>>(a);
  note_launch();
  if (load) launch_load(a.ids, tokens * a.k, a.E, accumulate, load, st);
}

template <int SCORE, bool BF16>
static void launch_route_bwd(const RouterBwdArgs& a, int64_t tokens, hipStream_t st) {
  if (a.E <= kLanes * kMaxVpl && a.k <= kLanes) {
    with_vpl((a.E + kLanes - 1) / kLanes, [&](auto vpl) {
      k_route_bwd<SCORE, BF16, decltype(vpl)::value>
          <<<(unsigned)((tokens + kTokens - 1) / kTokens), 256, 0, st>>>(a, tokens);
    });
  } else {
    k_route_bwd_any<SCORE, BF16><<<(unsigned)tokens, kAnyThreads, 0, st>>>(a);
  }
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
  if (a.top_groups == a.G) {  // every group stays
    a.G = 1;
    a.per = a.E;
  }
  if (tokens == 0 && (!load || accumulate)) return set_error(KT_RAWINT4_OK, "");
  begin_launches();
  if (tokens > 0) {
    const bool bf = router->logits_type == KT_TYPE_BF16, soft = router->score == KT_SCORE_SOFTMAX;
    if (soft && bf)
      launch_route<KT_SCORE_SOFTMAX, true>(a, tokens, load, accumulate, st);
    else if (soft)
      launch_route<KT_SCORE_SOFTMAX, false>(a, tokens, load, accumulate, st);
    else if (bf)
      launch_route<KT_SCORE_SIGMOID, true>(a, tokens, load, accumulate, st);
    else
      launch_route<KT_SCORE_SIGMOID, false>(a, tokens, load, accumulate, st);
  }
  if (tokens == 0 && load && !accumulate) launch_zero_i32(load, a.E, st);
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
  if (tokens == 0) return set_error(KT_RAWINT4_OK, "");
  hipStream_t st = static_cast<hipStream_t>(stream);
  const RouterBwdArgs a{router->num_experts, router->top_k, router->renormalize != 0, router->scale,
                        logits,              expert_ids,    grad_route,               grad_logits};
  begin_launches();
  const bool bf = router->logits_type == KT_TYPE_BF16, soft = router->score == KT_SCORE_SOFTMAX;
  if (soft && bf)
    launch_route_bwd<KT_SCORE_SOFTMAX, true>(a, tokens, st);
  else if (soft)
    launch_route_bwd<KT_SCORE_SOFTMAX, false>(a, tokens, st);
  else if (bf)
    launch_route_bwd<KT_SCORE_SIGMOID, true>(a, tokens, st);
  else
    launch_route_bwd<KT_SCORE_SIGMOID, false>(a, tokens, st);
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
