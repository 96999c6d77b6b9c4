// Norms before and after a block, fused with its gate, scale and the residual
// stream, and their gradients.
//
//   h = x + t n,  t = scale * gate * token_gate,  n = N(b) w2 + c2 or b,  y = N(h) w + c
//   with u = grad_y w and q = N(h), 1/s its deviation's inverse:
//   grad_x = grad_h + (u - [mean u] - q mean(u q)) / s      ([..]: layer norm alone)
//   and the same once more from t grad_x to b.
//
// Both directions are bound by memory: every row is read once and stays in registers between
// its statistics and its outputs (deviations from the mean are squared, not
// differences of squares), so that the bytes are those of the inputs and outputs.  Reached with
// bf16 (a copy of 1 GiB: 4.9 to 5.1 TB/s): forward with a block's output, 16384 x 7168,
// 184 us, 5.1 TB/s; backward without a norm behind the block, 16384 x 7168, 258 us, 5.5 TB/s.
// Statistics, sums and the parameters' gradients are fp32; each output is rounded once.
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

// A thread's columns: chunks of 8 neighbours, a row's threads apart.  MODE 0: rows
// are whole chunks.  MODE 1: they are not; the last chunk then is the row's
// last 8 columns, some of which another thread has too: sums over the row count them
// there, and both store the same values.  Not so in a call in place over several waves: there
// a wave may have changed them before another reads them, so that only the one that they belong to
// stores them.  Rows start at any multiple
// of their type (the hardware's unaligned accesses serve as well).  MODE 2: a row
// has fewer than 8 columns, which one thread takes one by one.
// Loads are issued whatever the thread (one without a chunk loads the row's last 8
// columns and takes zeros instead), so that how many are in flight is known
// where one is waited for.
template <int MODE>
struct Cols {
  int tid, nt, H;
  bool in_place;  // over several waves
  __device__ __forceinline__ int own(int chunk) const { return 8 * (tid + chunk * nt); }
  __device__ __forceinline__ int at(int chunk) const { return MODE == 2 ? 0 : min(own(chunk), H - 8); }
  // columns of a chunk that the one before has too
  __device__ __forceinline__ int shared(int chunk) const { return own(chunk) - at(chunk); }
  // (a 32-bit offset in bytes to a row's scalar address)
  template <typename T>
  __device__ __forceinline__ T* column(T* row, int chunk) const {
    return (T*)((char*)row + (uint32_t)at(chunk) * (uint32_t)sizeof(T));
  }
  __device__ __forceinline__ bool on(int chunk) const { return own(chunk) < H; }
  // 0 for what does not exist
  template <int N>
  __device__ __forceinline__ void mask(float* v) const {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = on(j >> 3) && (MODE < 2 || (j & 7) < H) ? v[j] : 0.f;
  }
  // a thread's part of a sum over the row: without what another thread counts
  __device__ __forceinline__ float once(int j, float v) const { return (j & 7) >= shared(j >> 3) ? v : 0.f; }
  template <int N>
  __device__ __forceinline__ float sum(const float* v) const {
    float s = 0.f;
    if (MODE != 1) {
#pragma unroll
      for (int j = 0; j < N; ++j) s += v[j];
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) s += once(j, v[j]);
    }
    return s;
  }
  template <int N>
  __device__ __forceinline__ float dot(const float* u, const float* v) const {
    float s = 0.f;
    if (MODE != 1) {
#pragma unroll
      for (int j = 0; j < N; ++j) s = fmaf(u[j], v[j], s);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) s = fmaf(once(j, u[j]), once(j, v[j]), s);
    }
    return s;
  }
};

typedef u32x4 u32x4_u2 __attribute__((aligned(2)));
typedef float f32x4_u4 __attribute__((ext_vector_type(4), aligned(4)));

// A chunk as it lies in memory, and as numbers.
template <typename T>
struct Raw;
template <>
struct Raw<uint16_t> {
  u32x4 w;
  template <int MODE>
  __device__ __forceinline__ void load(const uint16_t* row, const Cols<MODE>& c, int chunk) {
    const uint16_t* p = c.column(row, chunk);
    if (MODE == 0) w = *reinterpret_cast<const u32x4*>(p);
    if (MODE == 1) w = *reinterpret_cast<const u32x4_u2*>(p);
    if (MODE == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)p[min(2 * i, c.H - 1)] | (uint32_t)p[min(2 * i + 1, c.H - 1)] << 16;
    }
  }
  __device__ __forceinline__ void numbers(float* v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
};
template <>
struct Raw<float> {
  floatx4 lo, hi;
  template <int MODE>
  __device__ __forceinline__ void load(const float* row, const Cols<MODE>& c, int chunk) {
    const float* p = c.column(row, chunk);
    if (MODE == 0) lo = *reinterpret_cast<const floatx4*>(p), hi = *reinterpret_cast<const floatx4*>(p + 4);
    if (MODE == 1) lo = *reinterpret_cast<const f32x4_u4*>(p), hi = *reinterpret_cast<const f32x4_u4*>(p + 4);
    if (MODE == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) lo[i] = p[min(i, c.H - 1)], hi[i] = p[min(4 + i, c.H - 1)];
    }
  }
  __device__ __forceinline__ void numbers(float* v) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
  }
};

template <int N, typename T, int MODE>
__device__ __forceinline__ void load_row(const T* p, const Cols<MODE>& c, float* v) {
#pragma unroll
  for (int j = 0; j < N; j += 8) {
    Raw<T> r;
    r.load(p, c, j >> 3);
    r.numbers(v + j);
  }
  c.template mask<N>(v);
}

template <int N, int MODE>
__device__ __forceinline__ void store_row(float* p, const Cols<MODE>& c, const float* v) {
#pragma unroll
  for (int j = 0; j < N; j += 8) {
    float* at = c.column(p, j >> 3);
    if (!c.on(j >> 3)) continue;
    if (MODE == 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < c.H) p[i] = v[j + i];
    } else if (MODE == 1 && c.in_place && c.shared(j >> 3) > 0) {
#pragma unroll
      for (int i = 1; i < 8; ++i)
        if (i >= c.shared(j >> 3)) at[i] = v[j + i];
    } else {
      const floatx4 lo = {v[j], v[j + 1], v[j + 2], v[j + 3]}, hi = {v[j + 4], v[j + 5], v[j + 6], v[j + 7]};
      if (MODE == 0) {
        *reinterpret_cast<floatx4*>(at) = lo;
        *reinterpret_cast<floatx4*>(at + 4) = hi;
      } else {
        *reinterpret_cast<f32x4_u4*>(at) = lo;
        *reinterpret_cast<f32x4_u4*>(at + 4) = hi;
      }
    }
  }
}

template <int N, int MODE>
__device__ __forceinline__ void store_row(uint16_t* p, const Cols<MODE>& c, const float* v) {
#pragma unroll
  for (int j = 0; j < N; j += 8) {
    uint16_t* at = c.column(p, j >> 3);
    if (!c.on(j >> 3)) continue;
    if (MODE == 2) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < c.H) p[i] = float_to_bf16(v[j + i]);
    } else if (MODE == 1 && c.in_place && c.shared(j >> 3) > 0) {
#pragma unroll
      for (int i = 1; i < 8; ++i)
        if (i >= c.shared(j >> 3)) at[i] = float_to_bf16(v[j + i]);
    } else {
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = bf16_pair(v[j + 2 * i], v[j + 2 * i + 1]);
      if (MODE == 0)
        *reinterpret_cast<u32x4*>(at) = o;
      else
        *reinterpret_cast<u32x4_u2*>(at) = o;
    }
  }
}

// Sums of M values over a row's threads (the waves first .. first + waves - 1
// of a workgroup), the same bits in all of them: in a wave by lanes, between
// waves through LDS, a wave's sum to each of 16 lanes and by lanes again.  Two buffers in turn: one barrier a sum.
template <bool ONE, int M>
struct RowSums {
  float (*buf)[M][kNormMaxWaves];
  int first, waves, turn;
  __device__ __forceinline__ void operator()(float* s) {
#pragma unroll
    for (int i = 0; i < M; ++i) s[i] = wave_sum(s[i]);
    if (ONE) return;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < M; ++i) buf[turn][i][threadIdx.x >> 6] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const int w = threadIdx.x & 15;
      s[i] = row16_sum(w < waves ? buf[turn][i][first + w] : 0.f);
    }
    turn ^= 1;
  }
};

// v normalised in place
template <int N, typename Sums, int MODE>
__device__ __forceinline__ void normalise(const NormArgs& a, const Cols<MODE>& c, Sums& sums, float* v) {
  float s, mean;
  if (a.kind == KT_NORM_LAYER) {
    s = c.template sum<N>(v);
    sums(&s);
    mean = s * a.inv_h;
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] -= mean;
    c.template mask<N>(v);
  }
  s = c.template dot<N>(v, v);
  sums(&s);
  const float r = 1.f / sqrtf(s * a.inv_h + a.eps);
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] *= r;
}

// The vectors into LDS as the threads' chunks read them: the first four columns of every
// chunk, then the last four, so that neighbours' reads meet in no bank.  All loads first.
template <int MODE>
__device__ __forceinline__ void spread(const float* const* v, int H, float* out) {
  const int chunks = (H + 7) / 8;
  for (int chunk = threadIdx.x; chunk < chunks; chunk += blockDim.x) {
    const Cols<MODE> c{chunk, 0, H, false};
    Raw<float> r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (v[i]) r[i].load(v[i], c, 0);
    float* to = out + 4 * chunk;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!v[i]) continue;
      *reinterpret_cast<floatx4*>(to) = r[i].lo;
      *reinterpret_cast<floatx4*>(to + 4 * chunks) = r[i].hi;
      to += 8 * chunks;
    }
  }
}
template <int N, int MODE>
__device__ __forceinline__ void load_spread(const float* p, const Cols<MODE>& c, float* v) {
  const int chunks = (c.H + 7) / 8;
#pragma unroll
  for (int j = 0; j < N; j += 8) {
    const int chunk = min(c.tid + (j >> 3) * c.nt, chunks - 1);
    const floatx4 lo = *reinterpret_cast<const floatx4*>(p + 4 * chunk);
    const floatx4 hi = *reinterpret_cast<const floatx4*>(p + 4 * (chunks + chunk));
#pragma unroll
    for (int i = 0; i < 4; ++i) v[j + i] = lo[i], v[j + 4 + i] = hi[i];
  }
  c.template mask<N>(v);
}

// The thread's own sums of one of two vectors kept there, in the same order.
template <int N, int MODE, typename Value>
__device__ __forceinline__ void add_spread(float* p, const Cols<MODE>& c, Value value) {
  const int chunks = (c.H + 7) / 8;
#pragma unroll
  for (int j = 0; j < N; j += 8) {
    if (!c.on(j >> 3)) continue;
    floatx4* lo = reinterpret_cast<floatx4*>(p + 4 * (c.tid + (j >> 3) * c.nt));
    floatx4* hi = lo + chunks;
    floatx4 s = *lo, t = *hi;
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = value(j + i, s[i]), t[i] = value(j + 4 + i, t[i]);
    *lo = s, *hi = t;
  }
}

// (SPREAD: the vectors are as spread() leaves them)
template <int N, bool SPREAD = false, int MODE>
__device__ __forceinline__ void affine(const Cols<MODE>& c, const float* w, const float* bias, float* v) {
  float t[N];
  if (w) {
    SPREAD ? load_spread<N>(w, c, t) : load_row<N>(w, c, t);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] *= t[j];
  }
  if (bias) {
    SPREAD ? load_spread<N>(bias, c, t) : load_row<N>(bias, c, t);
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] += t[j];
  }
}

// (IN_PLACE: h is x, in rows of several waves that are no whole chunks)
template <typename S, int MODE, int VPT, bool ONE, bool IN_PLACE>
__global__ __launch_bounds__(ONE ? 256 : 1024) void k_norm_fwd(NormArgs a) {
  constexpr int N = 8 * VPT;
  __shared__ float buf[2][1][kNormMaxWaves];
  RowSums<ONE, 1> sums{buf, 0, (int)(blockDim.x >> 6), 0};
  Cols<MODE> c{ONE ? (int)threadIdx.x & 63 : (int)threadIdx.x, ONE ? 64 : (int)blockDim.x, a.H, IN_PLACE};
  const int64_t first = ONE ? (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : blockIdx.x;
  const int64_t step = ONE ? (int64_t)gridDim.x * 4 : gridDim.x;
  for (int64_t row = first; row < a.T; row += step) {
    float v[N];
    load_row<N>(static_cast<const S*>(a.x) + row * a.H, c, v);
    if (a.b) {
      float b[N];
      load_row<N>(a.b + row * a.H, c, b);
      if (a.nvec) normalise<N>(a, c, sums, b);
      affine<N>(c, a.bw, a.bc, b);
      const float s = a.tg ? a.scale * a.tg[row] : a.scale;
      affine<N>(c, a.gate, nullptr, b);
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = fmaf(s, b[j], v[j]);
      if (a.h) store_row<N>(static_cast<S*>(a.h) + row * a.H, c, v);
    }
    if (a.y) {
      normalise<N>(a, c, sums, v);
      affine<N>(c, a.w, a.c, v);
      store_row<N>(a.y + row * a.H, c, v);
    }
  }
}

// A row of the backward's inputs as it lies in memory.
template <typename S, int MODE, int VPT, bool BR, bool NEXT>
struct BwdRow {
  Raw<S> h[VPT];
  Raw<uint16_t> y[VPT], b[VPT];
  float tg;
  __device__ __forceinline__ void load(const NormArgs& a, const Cols<MODE>& c, int64_t row) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (NEXT) h[i].load(static_cast<const S*>(a.x) + row * a.H, c, i);
      if (NEXT) y[i].load(a.gy + row * a.H, c, i);
      if (BR) b[i].load(a.b + row * a.H, c, i);
    }
    if (BR) tg = a.tg ? a.tg[row] : 1.f;
  }
};

// The backward.  Teams of waves take a row each, a workgroup has as many teams
// as fit; a thread keeps its columns and their parts of the parameters'
// gradients over all rows, which the teams join in LDS at the end: one partial
// sum a workgroup.  The next row's inputs are on their way while one is worked on,
// and the vectors lie in LDS (they would have to come from the L2 four times a
// row, with every wave waiting).
// What is the same in a wave (rows' addresses) is in scalar registers, or the
// addresses kept over the rows are spilled, and their loads wait for all others (4001 x 2049:
// 68 -> 58 us).  4096 x 7168, fp32 stream, everything on: 116 us, 4.6 TB/s, the partial sums (37 MB both
// ways) not counted.  Rows that are no whole chunks are bound by what a row costs whatever
// its length (three exchanges, 15 waves of which one in five has one chunk): 4001 x 2049
// 56 us, 1.8 TB/s.  MOST: threads, from which the compiler has 256 or 128 registers.
// BR: a block's output; POST: the norm behind it; NEXT: grad_y; BIAS: d_bias or d_branch_bias.
template <typename S, int MODE, int VPT, int MOST, bool ONE, bool BR, bool POST, bool NEXT, bool BIAS>
__global__ __launch_bounds__(MOST) void k_norm_bwd(NormArgs a, int waves) {
  constexpr int N = 8 * VPT;
  constexpr bool AHEAD = VPT == 1 || MOST == 512;
  __shared__ float buf[2][3][kNormMaxWaves];
  extern __shared__ __align__(16) float lds[];  // the vectors in use (up to 8192 columns), [teams][H]
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // (rows' addresses in scalar registers)
  const int team = wave / waves, teams = (blockDim.x >> 6) / waves;
  RowSums<ONE, 3> sums{buf, team * waves, waves, 0};
  Cols<MODE> c{(int)threadIdx.x - team * waves * 64, waves * 64, a.H, !ONE && a.h && a.h == a.gh};
  const bool layer = a.kind == KT_NORM_LAYER;
  float dw[N], dc[N], dbw[N], dbc[N], dg[N];
#pragma unroll
  for (int j = 0; j < N; ++j) dw[j] = dc[j] = dbw[j] = dbc[j] = dg[j] = 0.f;
  // (rows above 8192 columns: 16 waves' registers do not hold all of them)
  float* const dg_lds = lds;
  float* const dbw_lds = lds + ((a.H + 7) & ~7);
  if (!AHEAD) {
    if (BR) add_spread<N>(dg_lds, c, [](int, float) { return 0.f; });
    if (POST) add_spread<N>(dbw_lds, c, [](int, float) { return 0.f; });
  }
  // weight, branch_weight, branch_bias, gate
  const float* vec[4] = {NEXT ? a.w : nullptr, POST ? a.bw : nullptr, POST ? a.bc : nullptr, BR ? a.gate : nullptr};
  float* join = lds;
  if (AHEAD) {
    spread<MODE>(vec, a.H, lds);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!vec[i]) continue;
      vec[i] = join;
      join += (a.H + 7) & ~7;
    }
    __syncthreads();
  }
  const int64_t step = (int64_t)gridDim.x * teams;
  int64_t row = (int64_t)blockIdx.x * teams + team;
  BwdRow<S, MODE, VPT, BR, NEXT> in;
  if (AHEAD) in.load(a, c, min(row, a.T - 1));
  // (all teams make the same number of rounds; one without a row works on the last and keeps nothing)
  for (int64_t base = (int64_t)blockIdx.x * teams; base < a.T; base += step, row += step) {
    const bool mine = row < a.T;
    const int64_t here = min(row, a.T - 1);
    asm volatile("" : "+v"(c.tid));  // (no addresses kept in registers from row to row)
    if (!AHEAD) in.load(a, c, here);
    float v[N], d[N], b[N], e[N];
    Raw<S> gh[VPT];
    float s[3] = {0.f, 0.f, 0.f};
    const float sc = BR ? a.scale * in.tg : 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (NEXT) in.h[i].numbers(v + 8 * i), in.y[i].numbers(e + 8 * i);
      if (BR) in.b[i].numbers(b + 8 * i);
      // (wanted late in the row, which hides its way; without grad_h: not used)
      gh[i].load(static_cast<const S*>(a.gh ? a.gh : a.x) + here * a.H, c, i);
    }
    if (AHEAD) in.load(a, c, min(row + step, a.T - 1));
    if (NEXT) c.template mask<N>(v), c.template mask<N>(e);
    if (BR) c.template mask<N>(b);
    // means and deviations of h and b; d = grad_y * weight
    float r1 = 0.f, r2 = 0.f, m1 = 0.f, m2 = 0.f;
    if (NEXT) {
#pragma unroll
      for (int j = 0; j < N; ++j) d[j] = e[j];
      affine<N, AHEAD>(c, vec[0], nullptr, d);
    }
    if (layer && (NEXT || POST)) {
      if (NEXT) s[0] = c.template sum<N>(v), s[1] = c.template sum<N>(d);
      if (POST) s[2] = c.template sum<N>(b);
      sums(s);
      m1 = s[1] * a.inv_h;
      const float mv = s[0] * a.inv_h, mb = s[2] * a.inv_h;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (NEXT) v[j] -= mv;
        if (POST) b[j] -= mb;
      }
      if (NEXT) c.template mask<N>(v);
      if (POST) c.template mask<N>(b);
    }
    if (NEXT || POST) {
      if (NEXT) s[0] = c.template dot<N>(v, v), s[1] = c.template dot<N>(d, v);
      if (POST) s[2] = c.template dot<N>(b, b);
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
      for (int j = 0; j < N; ++j) v[j] *= r1;
      if (mine) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          dw[j] = fmaf(e[j], v[j], dw[j]);
          if (BIAS) dc[j] += e[j];
        }
      }
#pragma unroll
      for (int j = 0; j < N; ++j) d[j] = r1 * (d[j] - m1 - v[j] * m2);
    }
    if (a.gh) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) gh[i].numbers(e + 8 * i);
#pragma unroll
      for (int j = 0; j < N; ++j) d[j] = NEXT ? d[j] + e[j] : e[j];
    }
    if (a.h && mine) store_row<N>(static_cast<S*>(a.h) + here * a.H, c, d);
    if (!BR) continue;
    // e = n, the block's output behind its norm
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (POST) b[j] *= r2;
      e[j] = b[j];
    }
    if (POST) affine<N, AHEAD>(c, vec[1], vec[2], e);
    // the token gate's gradient is without it, the channel gate's with it
#pragma unroll
    for (int j = 0; j < N; ++j) {
      e[j] *= d[j];
      if (AHEAD && mine) dg[j] = fmaf(sc, e[j], dg[j]);
    }
    if (!AHEAD) add_spread<N>(dg_lds, c, [&](int j, float s) { return fmaf(sc, e[j], s); });
    c.template mask<N>(e);
    if (vec[3]) {
      float g[N];
      AHEAD ? load_spread<N>(vec[3], c, g) : load_row<N>(vec[3], c, g);
#pragma unroll
      for (int j = 0; j < N; ++j) d[j] *= g[j], e[j] *= g[j];
    }
    s[0] = s[1] = 0.f;
    s[2] = c.template sum<N>(e);
#pragma unroll
    for (int j = 0; j < N; ++j) d[j] *= sc;
    if (POST) {
      if (mine) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          if (AHEAD) dbw[j] = fmaf(d[j], b[j], dbw[j]);
          if (BIAS) dbc[j] += d[j];
        }
      }
      if (!AHEAD) add_spread<N>(dbw_lds, c, [&](int j, float s) { return fmaf(d[j], b[j], s); });
      affine<N, AHEAD>(c, vec[1], nullptr, d);
      c.template mask<N>(d);
      s[0] = c.template sum<N>(d);
      s[1] = c.template dot<N>(d, b);
    }
    if (POST || a.gtg) sums(s);
    if (a.gtg && mine && c.tid == 0) a.gtg[here] = a.scale * s[2];
    if (!a.gb) continue;
    if (POST) {
      const float k1 = layer ? s[0] * a.inv_h : 0.f, k2 = s[1] * a.inv_h;
#pragma unroll
      for (int j = 0; j < N; ++j) d[j] = r2 * (d[j] - k1 - b[j] * k2);
    }
    if (mine) store_row<N>(a.gb + here * a.H, c, d);
  }
  float* part = a.part + (int64_t)blockIdx.x * 5 * a.H;
  auto give = [&](int i, const float* v) {
    if (!(a.nvec >> i & 1)) return;
    float* out = part + (int64_t)i * a.H;
    if (teams == 1) {
      store_row<N>(out, c, v);
      return;
    }
    __syncthreads();
    store_row<N>(join + team * a.H, c, v);
    __syncthreads();
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
      float s = join[j];
      for (int t = 1; t < teams; ++t) s += join[t * a.H + j];
      out[j] = s;
    }
  };
  if (!AHEAD) {
    if (BR) load_spread<N>(dg_lds, c, dg);
    if (POST) load_spread<N>(dbw_lds, c, dbw);
  }
  give(0, dw);
  give(1, dc);
  give(2, dbw);
  give(3, dbc);
  give(4, dg);
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
#pragma unroll 8
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
  bool one;    // a row is one wave's
  int vpt, waves, threads;
};
static NormShape norm_shape(int H) {
  NormShape s;
  const int units = (H + 7) / 8;
  s.one = units <= 64;
  s.vpt = units <= 1024 ? 1 : 2;
  s.waves = (units + 64 * s.vpt - 1) / (64 * s.vpt);
  s.threads = s.one ? 256 : s.waves * 64;
  return s;
}

// The backward's workgroups, one a unit of the chip, and their teams: as many as fit
// in 16 waves, unless fewer give every unit a row.  Rows of 4097 to 8192 columns take 16
// columns a thread and 8 waves, whose 256 registers each hold the parameters' gradients
// and the next row (4096 rows, everything on: of 7168 116 us, as 8 columns a thread in 14 waves
// of 128 registers; of 8192, bf16, 93 against 97; 2000 of 4097 66 against 61).  Shorter rows take 8 columns a
// thread, in as many teams as fit in 16 waves (4001 of 2049: 56 us; in 8 waves 73; but 8192 of
// 4096 126 against 118, 16384 of 1024 68 against 64).  Longer ones take 16 columns a thread in 16 waves, without the next
// row and the vectors ahead and with two of the gradients in LDS (2048 rows of 16384: 197 us; with all
// in registers, that is spilled, 288).
constexpr int64_t kNormGroups = 256;
struct NormTeams {
  int vpt, waves, teams;
  int64_t groups;
};
static NormTeams norm_teams(int H, int64_t T) {
  NormTeams t;
  const int units = (H + 7) / 8;
  t.vpt = units <= 512 ? 1 : 2;
  t.waves = (units + 64 * t.vpt - 1) / (64 * t.vpt);
  const int64_t most = t.vpt == 2 ? 1 : 16 / t.waves, want = (T + kNormGroups - 1) / kNormGroups;
  t.teams = (int)(want < most ? want : most);
  const int64_t groups = (T + t.teams - 1) / t.teams;
  t.groups = groups < kNormGroups ? groups : kNormGroups;
  return t;
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

template <typename S, bool WHOLE>
static void launch_norm_fwd(const NormArgs& a, const NormShape& s, hipStream_t st) {
  const int64_t rows = s.one ? (a.T + 3) / 4 : a.T;
  const unsigned grid = (unsigned)(rows < 4096 ? rows : 4096);
  const bool in_place = !WHOLE && !s.one && a.h == a.x;
  if (a.H < 8)
    k_norm_fwd<S, 2, 1, true, false><<<grid, 256, 0, st>>>(a);
  else if (s.one)
    k_norm_fwd<S, WHOLE ? 0 : 1, 1, true, false><<<grid, 256, 0, st>>>(a);
  else if (s.vpt == 1)
    in_place ? k_norm_fwd<S, WHOLE ? 0 : 1, 1, false, !WHOLE><<<grid, s.threads, 0, st>>>(a)
             : k_norm_fwd<S, WHOLE ? 0 : 1, 1, false, false><<<grid, s.threads, 0, st>>>(a);
  else
    in_place ? k_norm_fwd<S, WHOLE ? 0 : 1, 2, false, !WHOLE><<<grid, s.threads, 0, st>>>(a)
             : k_norm_fwd<S, WHOLE ? 0 : 1, 2, false, false><<<grid, s.threads, 0, st>>>(a);
  note_launch();
}

template <typename S, bool WHOLE, bool BR, bool POST, bool NEXT, bool BIAS>
static void launch_norm_bwd(const NormArgs& a, hipStream_t st) {
  const NormTeams t = norm_teams(a.H, a.T);
  const unsigned grid = (unsigned)t.groups, threads = (unsigned)(t.teams * t.waves * 64);
  const int vectors = (NEXT && a.w) + (POST && a.bw) + (POST && a.bc) + (BR && a.gate);
  const size_t lds = (t.teams > 1 ? (size_t)t.teams * a.H * 4 : 0) + (size_t)(a.H <= 8192 ? vectors : (int)BR + (int)POST) * ((a.H + 7) & ~7) * 4;
  if (a.H < 8)
    k_norm_bwd<S, 2, 1, 1024, true, BR, POST, NEXT, BIAS><<<grid, threads, lds, st>>>(a, t.waves);
  else if (t.waves == 1)
    k_norm_bwd<S, WHOLE ? 0 : 1, 1, 1024, true, BR, POST, NEXT, BIAS><<<grid, threads, lds, st>>>(a, t.waves);
  else if (t.vpt == 1)
    k_norm_bwd<S, WHOLE ? 0 : 1, 1, 1024, false, BR, POST, NEXT, BIAS><<<grid, threads, lds, st>>>(a, t.waves);
  else if (t.waves <= 8)
    k_norm_bwd<S, WHOLE ? 0 : 1, 2, 512, false, BR, POST, NEXT, BIAS><<<grid, threads, lds, st>>>(a, t.waves);
  else
    k_norm_bwd<S, WHOLE ? 0 : 1, 2, 1024, false, BR, POST, NEXT, BIAS><<<grid, threads, lds, st>>>(a, t.waves);
  note_launch();
}

template <typename S, bool WHOLE, bool BIAS>
static void launch_norm_bwd_parts(const NormArgs& a, bool post, hipStream_t st) {
  if (!a.b)
    a.gy ? launch_norm_bwd<S, WHOLE, false, false, true, BIAS>(a, st) : launch_norm_bwd<S, WHOLE, false, false, false, false>(a, st);
  else if (post)
    a.gy ? launch_norm_bwd<S, WHOLE, true, true, true, BIAS>(a, st) : launch_norm_bwd<S, WHOLE, true, true, false, BIAS>(a, st);
  else
    a.gy ? launch_norm_bwd<S, WHOLE, true, false, true, BIAS>(a, st) : launch_norm_bwd<S, WHOLE, true, false, false, false>(a, st);
}

template <typename S>
static void launch_norm_bwd_type(const NormArgs& a, bool post, bool bias, hipStream_t st) {
  if (a.H % 8 == 0)
    bias ? launch_norm_bwd_parts<S, true, true>(a, post, st) : launch_norm_bwd_parts<S, true, false>(a, post, st);
  else
    bias ? launch_norm_bwd_parts<S, false, true>(a, post, st) : launch_norm_bwd_parts<S, false, false>(a, post, st);
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
  const bool whole = a.H % 8 == 0;
  if (norm->stream_type == KT_TYPE_BF16)
    whole ? launch_norm_fwd<uint16_t, true>(a, s, st) : launch_norm_fwd<uint16_t, false>(a, s, st);
  else
    whole ? launch_norm_fwd<float, true>(a, s, st) : launch_norm_fwd<float, false>(a, s, st);
  return finish_launches();
}

size_t kt_norm_bwd_workspace_bytes(const kt_norm* norm, int32_t tokens) {
  if (check_norm(norm, tokens)) return 0;
  set_error(KT_RAWINT4_OK, "");
  // (more teams a group may make fewer groups of more tokens: the most over all numbers up to this one)
  const int64_t groups = tokens < kNormGroups ? tokens : kNormGroups;
  return round256((size_t)groups * 5 * (size_t)norm->hidden * 4);
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
  const bool post = norm->branch_norm != 0, bias = d_bias || d_branch_bias;
  begin_launches();
  if (norm->stream_type == KT_TYPE_BF16)
    launch_norm_bwd_type<uint16_t>(a, post, bias, st);
  else
    launch_norm_bwd_type<float>(a, post, bias, st);
  if (a.nvec) {
    NormJoin j{a.part, norm_teams(H, tokens).groups, H, accumulate, grad_scale, {d_weight, d_bias, d_branch_weight, d_branch_bias, d_gate}};
    k_norm_join<<<dim3((unsigned)((H + 63) / 64), 5), 1024, 0, st>>>(j);
    note_launch();
  }
  return finish_launches();
}

}  // extern "C"
